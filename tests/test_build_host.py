"""What build.py leaves behind for Python: a module per interpreter, and a library
that does without it."""
import importlib.machinery
import os
import sys
import sysconfig

import pytest

from test_expert_host import REFUSED as EXPERT
from test_mxfp4_host import REFUSED as MX
from tiled_dense_gemm_tma_b200 import binding, build as tg_build


def test_the_module_is_this_interpreters():
    """Another Python must not load a module that was built for this one."""
    tg_build.build()
    assert os.path.basename(tg_build.CALLS) == "_tg_calls" + sysconfig.get_config_var("EXT_SUFFIX")
    assert sysconfig.get_config_var("EXT_SUFFIX") in importlib.machinery.EXTENSION_SUFFIXES
    assert os.path.samefile(binding._calls().__file__, tg_build.CALLS)


def test_a_module_of_no_interpreter_goes(tmp_path, monkeypatch):
    """One of an older build would be found by any Python that has none of its own."""
    tg_build.build()
    for name in ("libtg_gemm.so", "_tg_calls.so"):
        (tmp_path / name).write_bytes(open(tg_build.OUT, "rb").read() if name == "libtg_gemm.so" else b"old")
    monkeypatch.setattr(tg_build, "HERE", str(tmp_path))
    monkeypatch.setattr(tg_build, "CALLS", str(tmp_path / os.path.basename(tg_build.CALLS)))
    tg_build._build_calls(False)
    assert sorted(os.listdir(tmp_path)) == sorted(["libtg_gemm.so", os.path.basename(tg_build.CALLS)])


def test_the_library_alone(tmp_path, monkeypatch, capfd):
    """Without a C compiler or Python's headers the library is built all the same, and
    the build says what is missing."""
    import shutil
    tg_build.build()
    shutil.copy(tg_build.OUT, tmp_path / "libtg_gemm.so")
    monkeypatch.setattr(tg_build, "HERE", str(tmp_path))
    monkeypatch.setattr(tg_build, "CALLS", str(tmp_path / os.path.basename(tg_build.CALLS)))
    monkeypatch.setenv("PATH", str(tmp_path))           # no gcc
    assert tg_build.build() == tg_build.OUT
    assert "_tg_calls" in capfd.readouterr().err
    assert os.listdir(tmp_path) == ["libtg_gemm.so"]
    monkeypatch.undo()
    shutil.copy(tg_build.OUT, tmp_path / "libtg_gemm.so")
    monkeypatch.setattr(tg_build, "HERE", str(tmp_path))
    monkeypatch.setattr(tg_build, "CALLS", str(tmp_path / os.path.basename(tg_build.CALLS)))
    monkeypatch.setattr(sysconfig, "get_path", lambda name: str(tmp_path))      # no Python.h
    assert tg_build.build() == tg_build.OUT
    assert "_tg_calls" in capfd.readouterr().err
    assert os.listdir(tmp_path) == ["libtg_gemm.so"]


@pytest.fixture
def without_module(monkeypatch):
    tg_build.build()
    monkeypatch.setitem(sys.modules, "tiled_dense_gemm_tma_b200._tg_calls", None)
    monkeypatch.delattr("tiled_dense_gemm_tma_b200._tg_calls", raising=False)
    return binding._calls()


@pytest.mark.parametrize("name,names,good,cases", EXPERT + MX, ids=[r[0] for r in EXPERT + MX])
def test_calls_without_the_module(without_module, name, names, good, cases):
    for change, want in cases:
        a = dict(good, **change)
        assert getattr(without_module, name)(*[a[n] for n in names]) == want, change


def test_numbers_beyond_an_int_without_the_module(without_module):
    good = (0, 8, None, 8, 2, None, 0, 2, 1, 2, 1, 1.0, None, None, None)
    assert without_module.tg_expert_route(*good) == 0
    for at in (1, 4, 6, 7, 8, 9, 10):
        for far in (1 << 32, -(1 << 32)):
            args = list(good)
            args[at] += far
            assert without_module.tg_expert_route(*args) != 0, (at, far)
