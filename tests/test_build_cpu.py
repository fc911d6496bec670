"""The build where the native calls of the torch classes cannot be compiled: the
library is there all the same, and so is everything that needs no more."""
import importlib.util
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAME = "head_heterogeneous_block_gb300"


@pytest.fixture
def copy(tmp_path):
    """A copy of the built tree (times kept, so nothing is out of date) without its
    libraries, and its build script."""
    pytest.importorskip("torch")
    import __graft_entry__
    __graft_entry__.build()
    for d in (NAME, "include", os.path.join("_build", "obj")):
        shutil.copytree(os.path.join(ROOT, d), tmp_path / d, ignore=shutil.ignore_patterns("__pycache__"))
    spec = importlib.util.spec_from_file_location("_sa_build_copy", tmp_path / NAME / "_build.py")
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    os.remove(build.LIB)
    return build


IMPORTS = f"""
import {NAME} as sa
from {NAME} import *
assert callable(sparse_attn_plan) and "PagedCache" in globals() and "Rotary" not in globals()
assert sa.PagedCache is PagedCache
for name in ("Rotary", "PagePool", "PackedAttention"):
    try:
        getattr(sa, name)
    except ImportError as e:
        assert "_calls.so" in str(e)
    else:
        raise AssertionError(name)
"""


def uses(build):
    root = os.path.dirname(build.PKG)
    r = subprocess.run([sys.executable, "-c", IMPORTS], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_without_headers_the_library_is_built_alone(copy, tmp_path, monkeypatch, capfd):
    paths = dict(copy.sysconfig.get_paths(), include=str(tmp_path / "nowhere"))
    monkeypatch.setattr(copy.sysconfig, "get_paths", lambda: paths)
    os.utime(copy.CALLS, (1, 1))                 # calls of an older library are not left beside the new one
    assert copy.build() == copy.LIB and os.path.exists(copy.LIB)
    assert not os.path.exists(copy.CALLS) and "Python.h is missing" in capfd.readouterr().err
    uses(copy)


def test_calls_that_do_not_compile_leave_the_library(copy):
    with open(copy.CALLS_SRC, "w") as f:
        f.write("#error not to be compiled\n")
    with pytest.raises(RuntimeError, match="calls.cpp"):
        copy.build()
    assert os.path.exists(copy.LIB) and not os.path.exists(copy.CALLS)
    uses(copy)


def test_both_are_built_where_they_can_be(copy):
    os.remove(copy.CALLS)
    copy.build()
    assert os.path.exists(copy.LIB) and os.path.exists(copy.CALLS)
