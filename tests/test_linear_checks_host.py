"""Checks of the matrix products on the host, without a GPU: their sources, and how calls are planned."""
import subprocess
from pathlib import Path

import pytest

from deterministic_residual_add_gb300 import build as drbuild
from test_linear_host import L  # noqa: F401


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


@pytest.mark.parametrize("rows,inner,cols,tiles", [
    (16, 4096, 4096, False), (16, 5120, 4096, False), (16, 5128, 4096, True), (9, 8192, 2048, True), (17, 4096, 4096, True),
    (8, 8192, 4096, False), (8, 10240, 4096, True), (1, 5120, 8192, False)])
def test_few_rows_that_take_split_tiles(L, rows, inner, cols, tiles):
    """Where the few rows' kernel is the slower one a product takes tiles, which these sizes split: a workspace."""
    assert (L.linear_act_add_fwd_workspace_bytes(rows, inner, cols) > 0) == tiles
