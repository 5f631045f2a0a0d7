"""Host check of how the weight gradient over groups keeps a group's last block
to the group's own rows (csrc/tile_sched.h, run on the device by the kernel)."""
import ctypes
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "tiled_dense_gemm_tma_b200", "csrc")


def test_every_row_of_a_group_enters_once(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    out = str(tmp_path / "libwindow_check.so")
    subprocess.run([gxx, "-O2", "-std=c++17", "-shared", "-fPIC", "-I", CSRC,
                    os.path.join(HERE, "group_window_check.cpp"), "-o", out], check=True)
    fn = ctypes.CDLL(out).check_windows
    fn.restype = ctypes.c_longlong
    n = ctypes.c_longlong(0)
    assert fn(ctypes.c_int(700), ctypes.byref(n)) == 0 and n.value > 0


def test_products_over_groups_signal_the_peer_by_copies_and_commits_only():
    """No thread of the grouped kernel writes operands in shared memory that
    the peer's MMA issuer then reads on the strength of a plain arrival: its
    only arrival on a barrier of the leader CTA frees an accumulator."""
    with open(os.path.join(CSRC, "gemm_group.cuh")) as f:
        text = f.read()
    arrivals = [line.strip() for line in text.splitlines() if "mbar_arrive_cluster(" in line]
    assert len(arrivals) == 1 and "tempty" in arrivals[0]
