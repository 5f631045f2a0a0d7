"""Edges of the 8-bit and experts' operators on a B200: group ends of every
kind beside foreign rows, positions outside the rows, the most groups."""
import os
import subprocess
import sys
import textwrap

import pytest
import torch

from expert_util import DTYPES, close, normal, offsets_of, product16

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def tg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import tiled_dense_gemm_tma_b200 as tg
    tg.load_library()
    return tg


def _status(tg):
    torch.cuda.synchronize()
    assert tg.last_device_status() == 0


# ------------------------------------------------- the weight gradient's groups

@pytest.mark.parametrize("K,N,dtype", [(72, 136, "bf16"), (300, 260, "f16"), (8, 520, "bf16")])
def test_every_group_end_beside_foreign_rows(tg, K, N, dtype):
    """Groups of 1 to 130 rows, one of infinities and NaN behind each, such
    rows before the matrices' first and behind their last one too: none of it
    enters a neighbour's sum, on any of many runs."""
    dt = DTYPES[dtype]
    counts = [c for n in range(1, 131) for c in (n, 3)]
    R = sum(counts)
    bufA, bufG = normal((R + 160, K), dt, 1), normal((R + 160, N), dt, 2)
    A, G = bufA[80:80 + R], bufG[80:80 + R]
    for buf, bad in ((bufA, float("nan")), (bufG, float("inf"))):
        buf[:80], buf[80 + R:] = bad, bad
    at = 0
    for i, n in enumerate(counts):
        if i % 2:
            A[at:at + n], G[at:at + n] = float("inf"), float("nan")
        at += n
    o = offsets_of(counts)
    C = tg.gemm_grouped_wgrad(A, G, o)
    _status(tg)
    at = 0
    for e, n in enumerate(counts):
        if e % 2:
            assert bool(torch.isnan(C[e]).all())
        else:
            ref, bound = product16(A[at:at + n].t(), G[at:at + n], dt)
            close(C[e], ref, bound, f"group of {n}")
        at += n
    for _ in range(50):
        again = tg.gemm_grouped_wgrad(A, G, o)
        assert torch.equal(again[::2], C[::2])
    _status(tg)


def test_long_cut_groups_repeat_themselves(tg):
    """Ordinary groups that all end inside a 16-row step, both CTAs of every
    pair at work, under load from run to run."""
    g = torch.Generator().manual_seed(4)
    counts = [int(n) | 1 for n in torch.randint(700, 1300, (16,), generator=g)]
    A, G = normal((sum(counts), 1024), torch.bfloat16, 5), normal((sum(counts), 768), torch.bfloat16, 6)
    o = offsets_of(counts)
    C = tg.gemm_grouped_wgrad(A, G, o)
    at = 0
    for e, n in enumerate(counts):
        ref, bound = product16(A[at:at + n].t(), G[at:at + n], torch.bfloat16)
        close(C[e], ref, bound, f"group of {n}")
        at += n
    for _ in range(200):
        assert torch.equal(tg.gemm_grouped_wgrad(A, G, o), C)
    _status(tg)


# ------------------------------------------------------- sums over very many k

LONG = textwrap.dedent("""
    import sys, torch
    sys.path.insert(0, %r); sys.path.insert(0, %r)
    import tiled_dense_gemm_tma_b200 as tg
    from expert_util import offsets_of
    n = 1 << 24
    one = lambda *shape: torch.ones(shape, dtype=torch.bfloat16, device="cuda")
    warm = tg.gemm_grouped(one(8, 64), offsets_of([8]), one(1, 64, 8))
    warm = tg.gemm_grouped_wgrad(one(64, 8), one(64, 8), offsets_of([64]))
    if sys.argv[1] == "product":
        A, B, o = one(8, n), one(1, n, 8), offsets_of([8])
        call = lambda: tg.gemm_grouped(A, o, B)
    else:
        A, G, o = one(n, 8), one(n, 8), offsets_of([n])
        call = lambda: tg.gemm_grouped_wgrad(A, G, o)
    torch.cuda.synchronize()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    C = call()
    b.record()
    torch.cuda.synchronize()
    # 16 ones a step: integers up to 2^24, exact
    print("RESULT", tg.last_device_status(), bool((C == n).all()), a.elapsed_time(b))
""") % (ROOT, os.path.join(ROOT, "tests"))


@pytest.mark.parametrize("what", ["product", "wgrad"])
def test_a_tile_may_take_longer_than_the_wait_limit(tg, what):
    """The limit is for waits that nothing will end.  A tile whose sum runs over
    2^24 terms makes progress for longer than the 20 ms set here (as 2^30 terms
    would for longer than the 4 s of the default) and is no time-out."""
    env = dict(os.environ, TG_DEBUG_TIMEOUT_US="20000")
    r = subprocess.run([sys.executable, "-c", LONG, what], env=env, capture_output=True, text=True, timeout=180)
    assert r.returncode == 0, r.stderr[-3000:]
    status, right, ms = [l for l in r.stdout.splitlines() if l.startswith("RESULT")][0].split()[1:]
    assert (status, right) == ("0", "True"), (status, right, ms)
    assert float(ms) > 20                                     # or the case shows nothing
