"""The in-tree build, on the host: what the library and the binding need, and
when they are built again.  A small library stands in for libdradd.so."""
import subprocess
import sys

import pytest

import deterministic_residual_add_gb300 as dr
from deterministic_residual_add_gb300 import build as drbuild
from deterministic_residual_add_gb300 import train


@pytest.fixture
def small(tmp_path, monkeypatch):
    """One source and no binding yet, in a folder of their own."""
    src = tmp_path / "one.cu"
    src.write_text('extern "C" int answer() { return 42; }\n')
    for name, value in (("LIB", tmp_path / "libdradd.so"), ("BINDING", tmp_path / "_binding.so"),
                        ("BUILD", tmp_path / "_build"), ("BINDING_SRC", tmp_path / "binding.cpp"),
                        ("_sources", lambda: [src])):
        monkeypatch.setattr(drbuild, name, value)
    (tmp_path / "binding.cpp").write_text('extern "C" int more() { return 1; }\n')
    return tmp_path


def test_library_is_there_where_the_binding_fails(small):
    (small / "binding.cpp").write_text("#error not today\n")
    with pytest.raises(RuntimeError, match="not today"):
        drbuild.build()
    assert (small / "libdradd.so").exists() and not (small / "_binding.so").exists()


@pytest.mark.parametrize("lacking", ["g++", "Python's headers", "torch"])
def test_library_needs_nvcc_alone(small, monkeypatch, lacking):
    if lacking == "g++":
        which = drbuild.shutil.which
        monkeypatch.setattr(drbuild.shutil, "which", lambda n: None if n == "g++" else which(n))
    elif lacking == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)  # its import fails
    else:
        monkeypatch.setattr(drbuild.sysconfig, "get_paths", lambda: {"include": str(small)})
    with pytest.warns(UserWarning, match=lacking.replace("+", r"\+")):
        assert drbuild.build() == small / "libdradd.so"
    assert (small / "libdradd.so").exists() and not (small / "_binding.so").exists()


def test_binding_follows_its_python_and_torch(small, monkeypatch):
    import torch
    drbuild.build()
    assert (small / "_binding.so").exists() and not drbuild.stale()
    made = (small / "libdradd.so").stat().st_mtime_ns
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert drbuild.stale()
    drbuild.build()
    assert not drbuild.stale() and (small / "libdradd.so").stat().st_mtime_ns == made
    monkeypatch.setattr(sys, "version", "another")
    assert drbuild.stale()


def test_calls_say_that_the_binding_is_missing(monkeypatch):
    drbuild.build()
    monkeypatch.setattr(train, "_C", None)
    monkeypatch.setitem(sys.modules, "deterministic_residual_add_gb300._binding", None)
    monkeypatch.delattr(dr, "_binding", raising=False)
    with pytest.raises(RuntimeError, match="binding does not load"):
        dr.dropout_fwd(None, 0.1, seed=1)
    assert dr.abi_version() == 1  # the other calls do without it


def test_package_and_library_without_torch():
    """Configurations and the C ABI are there where torch is not."""
    drbuild.build()
    code = ("import sys; sys.modules['torch'] = None\n"
            "import deterministic_residual_add_gb300 as dr\n"
            "from deterministic_residual_add_gb300 import build\n"
            "print(dr.abi_version(), dr.resolve_config(4096, 4096).threads_per_row, build.binding_lacks())")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=drbuild.ROOT)
    assert r.returncode == 0 and r.stdout.split() == ["1", "128", "torch"], r.stderr


def test_command_line():
    r = subprocess.run([sys.executable, "-m", "deterministic_residual_add_gb300.build"], capture_output=True, text=True,
                       cwd=drbuild.ROOT)
    assert r.returncode == 0 and r.stdout.strip().endswith("libdradd.so"), r.stderr
