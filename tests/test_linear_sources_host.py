"""Checks of the matrix products' sources on the host, without a GPU."""
from deterministic_residual_add_gb300 import build as drbuild


def test_products_compile_without_warnings():
    drbuild.build()
    logs = sorted(drbuild.BUILD.glob("dradd_linear_*.ptxas.txt"))
    assert len(logs) == 6
    for log in logs:
        assert "warning" not in log.read_text(), log.name
