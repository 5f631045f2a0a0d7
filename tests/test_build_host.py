"""What build.py leaves behind for Python: a module per interpreter."""
import importlib.machinery
import os
import sysconfig

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
