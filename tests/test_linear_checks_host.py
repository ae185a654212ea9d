"""Checks of the matrix products' sources on the host, without a GPU."""
import subprocess
from pathlib import Path

from deterministic_residual_add_gb300 import build as drbuild


def test_products_compile_without_warnings():
    drbuild.build()
    logs = sorted(drbuild.BUILD.glob("dradd_linear_*.ptxas.txt"))
    assert len(logs) == 6
    for log in logs:
        assert "warning" not in log.read_text(), log.name


def test_a_box_s_copies_are_waited_for(tmp_path):
    """Also where a wait has given up: shared memory is not left while a copy into it may be in flight."""
    exe = tmp_path / "staging_check"
    src = Path(__file__).with_name("staging_check.cpp")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-I", drbuild.CSRC, src, "-o", exe], check=True)
    assert subprocess.run([exe], capture_output=True, text=True, check=True).stdout == "ok\n"
