"""Host checks of the group arithmetic of csrc/tile_sched.h, which the kernels
run on the device: row tiles and their widths, the pieces of a thin last wave,
rows of groups from arbitrary offsets."""
import ctypes
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "tiled_dense_gemm_tma_b200", "csrc")


@pytest.fixture(scope="module")
def chk(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    out = str(tmp_path_factory.mktemp("group") / "libgroup_check.so")
    subprocess.run([gxx, "-O2", "-std=c++17", "-shared", "-fPIC", "-I", CSRC,
                    os.path.join(HERE, "group_sched_check.cpp"), "-o", out], check=True)
    return ctypes.CDLL(out)


@pytest.mark.parametrize("name,args", [("check_group_tiles", (3000,)), ("check_group_large", ()),
                                       ("check_group_schedule", (200, 80)), ("check_group_rows", ())])
def test_group_arithmetic(chk, name, args):
    fn = getattr(chk, name)
    fn.restype = ctypes.c_longlong
    n = ctypes.c_longlong(0)
    bad = fn(*[ctypes.c_int(a) for a in args], ctypes.byref(n))
    assert n.value > 0 and bad == 0
