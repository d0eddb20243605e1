"""Building and loading the binding of the paged calls: the C library needs no torch, a binding of another torch or
Python counts as stale, and one that does not load says why (CPU only)."""
import os
import shutil
import subprocess
import sys

import pytest

from column_sparse_masked_b200 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(code, *args):
    return subprocess.run([sys.executable, "-c", code, *args], capture_output=True, text=True, cwd=ROOT, timeout=300)


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def test_the_library_is_built_without_torch():
    r = run("import sys, runpy; sys.modules['torch'] = None; sys.argv = ['build.py'];"
            "runpy.run_path('column_sparse_masked_b200/build.py', run_name='__main__')")
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip().endswith("libflashmask.so") and "torch" in r.stderr


def test_a_binding_of_another_torch_is_stale(monkeypatch, tmp_path):
    assert not build.binding_stale()
    import torch

    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "0.0.0")
        assert build.binding_stale()
    with monkeypatch.context() as m:
        m.setattr(build, "BINDING", str(tmp_path / "_paged_binding.so"))
        assert build.binding_stale()
        (tmp_path / "_paged_binding.so").write_bytes(b"no key in here")
        assert build.binding_stale()
    os.utime(build.BINDING, (1, 1))
    assert build.binding_stale()
    os.utime(build.BINDING)


def _package(tmp_path, binding):
    pkg = tmp_path / "column_sparse_masked_b200"
    pkg.mkdir()
    src = os.path.join(ROOT, "column_sparse_masked_b200")
    for n in os.listdir(src):
        if n.endswith(".py"):
            shutil.copy(os.path.join(src, n), pkg / n)
    os.symlink(os.path.join(src, "libflashmask.so"), pkg / "libflashmask.so")
    if binding is not None:
        (pkg / "_paged_binding.so").write_bytes(binding)


CALL = ("import sys; sys.path.insert(0, sys.argv[1]); import column_sparse_masked_b200 as fm\n"
        "assert fm.__file__.startswith(sys.argv[1])\n"
        "fm.paged_gather(None, None, None, None, 1)")


def test_a_binding_that_does_not_load_says_why(tmp_path):
    _package(tmp_path, b"not a shared object")
    r = run(CALL, str(tmp_path))
    assert "RuntimeError: _paged_binding.so does not load" in r.stderr and "is missing" not in r.stderr
    assert "file too short" in r.stderr or "invalid ELF header" in r.stderr


def test_a_missing_binding_is_called_missing(tmp_path):
    _package(tmp_path, None)
    assert "RuntimeError: _paged_binding.so is missing" in run(CALL, str(tmp_path)).stderr


def test_a_binding_of_another_torch_is_not_used(tmp_path):
    with open(build.BINDING, "rb") as f:
        _package(tmp_path, f.read())
    r = run("import torch; torch.__version__ = '0.0.0'\n" + CALL, str(tmp_path))
    assert "RuntimeError: _paged_binding.so does not load" in r.stderr and "0.0.0" in r.stderr
