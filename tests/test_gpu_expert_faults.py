"""Bounded waits of the kernels behind the 8-bit and experts' products, without
a fault: with TG_INJECT=1 the first launch of the process leaves one ring slot
unarmed, so a wait that nothing completes runs into its limit (0.2 s here);
the call's status word reads TG_ERR_TIMEOUT, the context stays usable and the
next call is right.  A child process each: both knobs are read once."""
import os
import subprocess
import sys
import textwrap

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = textwrap.dedent("""
    import sys, time, torch
    sys.path.insert(0, %r); sys.path.insert(0, %r)
    import tiled_dense_gemm_tma_b200 as tg
    from expert_util import *

    fam = sys.argv[1]
    bf = torch.bfloat16
    if fam in ("grouped", "wgrad", "wgrad_cut"):
        counts = [600, 0, 424] if fam != "wgrad_cut" else [601, 3, 420]
        X, W, G = normal((1024, 512), bf, 1), normal((3, 512, 768), bf, 2), normal((1024, 768), bf, 3)
        o = offsets_of(counts)
        call = (lambda: tg.gemm_grouped(X, o, W)) if fam == "grouped" else (lambda: tg.gemm_grouped_wgrad(X, G, o))
        def check(C):
            at = 0
            for e, n in enumerate(counts):
                if fam == "grouped":
                    close(C[at:at + n], *product16(X[at:at + n], W[e], bf))
                else:
                    close(C[e], *product16(X[at:at + n].t(), G[at:at + n], bf))
                at += n
    else:
        M, K, N = {"i8_pair": (512, 1024, 768), "i8_skinny": (16, 4096, 2048), "i8_skinny_whole": (3, 300, 100)}[fam]
        A, W, rs, cs = ints8((M, K), 1), ints8((K, N), 2), positive((M,), 3), positive((N,), 4)
        call = lambda: tg.gemm_w8a8(A, rs, W, cs)
        check = lambda C: close(C, *product8(A, rs, W, cs, bf))
    torch.cuda.synchronize()
    t0 = time.time()
    call()                                  # the injected launch
    st = tg.last_device_status()
    dt = time.time() - t0
    st2 = tg.last_device_status()
    C = call()
    st3 = tg.last_device_status()
    check(C)
    x = (torch.ones(1024, device="cuda") * 2).sum().item()
    print("RESULT", st, st2, st3, x, round(dt, 3))
""") % (ROOT, os.path.join(ROOT, "tests"))


@pytest.mark.parametrize("family", ["grouped", "wgrad", "wgrad_cut", "i8_pair", "i8_skinny", "i8_skinny_whole"])
def test_bounded_wait_reports_timeout_then_recovers(family):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    env = dict(os.environ, TG_INJECT="1", TG_DEBUG_TIMEOUT_US="200000")
    r = subprocess.run([sys.executable, "-c", CHILD, family], env=env, capture_output=True, text=True, timeout=180)
    assert r.returncode == 0, r.stderr[-3000:]
    st, st2, st3, x, dt = [l for l in r.stdout.splitlines() if l.startswith("RESULT")][0].split()[1:]
    assert (int(st), int(st2), int(st3)) == (5, 0, 0)     # TG_ERR_TIMEOUT, cleared, a normal call
    assert float(x) == 2048.0 and float(dt) < 30.0


def test_refused_cluster_launches_are_reported():
    """With the CTA-pair kernels off the products that have no other kernel say
    so, and the weight-streaming one still runs."""
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    code = textwrap.dedent("""
        import sys, torch
        sys.path.insert(0, %r); sys.path.insert(0, %r)
        import tiled_dense_gemm_tma_b200 as tg
        from expert_util import *
        X, W, o = normal((8, 16), torch.bfloat16, 1), normal((1, 16, 16), torch.bfloat16, 2), offsets_of([8])
        A, B, s = ints8((200, 16), 1), ints8((16, 16), 2), positive((200,), 3)
        for f in (lambda: tg.gemm_grouped(X, o, W), lambda: tg.gemm_grouped_wgrad(X, X, o),
                  lambda: tg.gemm_w8a8(A, s, B, s[:16])):
            try:
                f()
                raise SystemExit("not refused")
            except tg.TgError as e:
                assert e.code == 3, e
        C = tg.gemm_w8a8(A[:4], s[:4], B, s[:16])
        close(C, *product8(A[:4], s[:4], B, s[:16], torch.bfloat16))
        print("ok", tg.last_device_status())
    """) % (ROOT, os.path.join(ROOT, "tests"))
    r = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, TG_NO_PAIR="1"), capture_output=True,
                       text=True, timeout=180)
    assert r.returncode == 0 and "ok 0" in r.stdout, r.stderr[-3000:] + r.stdout
