"""Routing and the microscaled 4-bit operators where a call meets its
surroundings: other streams, captured graphs, timeouts, refused clusters, rows far
apart in memory, offsets that no sort would write."""
import os
import subprocess
import sys
import textwrap

import pytest
import torch

import tiled_dense_gemm_tma_b200 as tg
from expert_util import close, normal, offsets_of
from mxfp4_util import product, quantised, random_blocks, values
from test_gpu_mxfp4 import guarded, untouched

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = textwrap.dedent("""
    import sys, time, torch
    sys.path.insert(0, %r); sys.path.insert(0, %r)
    import tiled_dense_gemm_tma_b200 as tg
    from expert_util import close, offsets_of
    from mxfp4_util import *

    fam = sys.argv[1]
    bf = torch.bfloat16
    if fam == "grouped":
        counts = [600, 0, 424]
        (a, sa), (w, sw), o = random_blocks((1024, 1024), 1), random_blocks((3, 768, 1024), 2), offsets_of(counts)
        call = lambda: tg.gemm_grouped_mxfp4(a, sa, o, w, sw)
        def check(C):
            at = 0
            for e, n in enumerate(counts):
                close(C[at:at + n], *product(values(a[at:at + n], sa[at:at + n]), values(w[e], sw[e]), bf))
                at += n
    else:
        M, K, N = {"pair": (512, 4096, 768), "skinny": (16, 8192, 2048), "skinny_whole": (3, 300, 100)}[fam]
        (a, sa), (w, sw) = random_blocks((M, K), 1), random_blocks((N, K), 2)
        call = lambda: tg.gemm_mxfp4(a, sa, w, sw)
        check = lambda C: close(C, *product(values(a, sa), values(w, sw), bf))
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


@pytest.mark.parametrize("family", ["grouped", "pair", "skinny", "skinny_whole"])
def test_bounded_wait_reports_timeout_then_recovers(family):
    env = dict(os.environ, TG_INJECT="1", TG_DEBUG_TIMEOUT_US="200000")
    r = subprocess.run([sys.executable, "-c", CHILD, family], env=env, capture_output=True, text=True, timeout=180)
    assert r.returncode == 0, r.stderr[-3000:]
    st, st2, st3, x, dt = [l for l in r.stdout.splitlines() if l.startswith("RESULT")][0].split()[1:]
    assert (int(st), int(st2), int(st3)) == (5, 0, 0)     # TG_ERR_TIMEOUT, cleared, a normal call
    assert float(x) == 2048.0 and float(dt) < 30.0


def test_refused_cluster_launches_are_reported():
    """With the CTA-pair kernels off the products that have no other kernel say
    so, and the weight-streaming one still runs."""
    code = textwrap.dedent("""
        import sys, torch
        sys.path.insert(0, %r); sys.path.insert(0, %r)
        import tiled_dense_gemm_tma_b200 as tg
        from expert_util import close, offsets_of
        from mxfp4_util import *
        (a, sa), (w, sw) = random_blocks((200, 64), 1), random_blocks((1, 16, 64), 2)
        for f in (lambda: tg.gemm_grouped_mxfp4(a, sa, offsets_of([200]), w, sw), lambda: tg.gemm_mxfp4(a, sa, w[0], sw[0])):
            try:
                f()
                raise SystemExit("not refused")
            except tg.TgError as e:
                assert e.code == 3, e
        C = tg.gemm_mxfp4(a[:4], sa[:4], w[0], sw[0])
        close(C, *product(values(a[:4], sa[:4]), values(w[0], sw[0]), torch.bfloat16))
        print("ok", tg.last_device_status())
    """) % (ROOT, os.path.join(ROOT, "tests"))
    r = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, TG_NO_PAIR="1"), capture_output=True,
                       text=True, timeout=180)
    assert r.returncode == 0 and "ok 0" in r.stdout, r.stderr[-3000:] + r.stdout


def layer(x, lg, w1, s1, w2, s2):
    E = lg.shape[1]
    ids, wt = tg.expert_route(lg, 2)
    plan = tg.expert_sort(ids, E)
    q, s = tg.quant_mxfp4(x, plan)
    h = tg.gemm_grouped_mxfp4(q, s, plan, w1, s1, relu=True)
    q, s = tg.quant_mxfp4(h)
    return tg.expert_combine(tg.gemm_grouped_mxfp4(q, s, plan, w2, s2), plan, wt)


def test_captured_layers_share_nothing():
    """Two captured layers of different shapes, replayed in turn and at once on
    two streams, give what the eager calls give."""
    cases = []
    for i, (T, E, D, F) in enumerate([(70, 4, 128, 320), (300, 8, 256, 96)]):
        g = torch.Generator().manual_seed(i)
        x = torch.randn((T, D), generator=g).bfloat16().cuda()
        lg = torch.randn((T, E), generator=g).cuda()
        w1, s1 = random_blocks((E, F, D), 2 + i, 120, 124)
        w2, s2 = random_blocks((E, D, F), 7 + i, 120, 124)
        cases.append([x, lg, w1, s1, w2, s2])
    graphs, outs, streams = [], [], []
    for c in cases:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            layer(*c)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            outs.append(layer(*c))
        graphs.append(graph)
        streams.append(s)
    for seed in (1, 2):
        for c in cases:
            g = torch.Generator().manual_seed(seed)
            c[0].copy_(torch.randn(c[0].shape, generator=g))
            c[1].copy_(torch.randn(c[1].shape, generator=g))
        torch.cuda.synchronize()
        for _ in range(20):
            for graph, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    graph.replay()
        torch.cuda.synchronize()
        for c, out in zip(cases, outs):
            assert torch.equal(out, layer(*c))
    assert tg.last_device_status() == 0


def test_captured_routing_step():
    """Forward and backward of the routing captured, replayed on new logits."""
    x = torch.randn((130, 16), generator=torch.Generator().manual_seed(1)).cuda().requires_grad_(True)
    dw = torch.randn((130, 3), generator=torch.Generator().manual_seed(2)).cuda()

    def step():
        x.grad = None
        ids, w = tg.expert_route(x, 3, renorm=False)
        w.backward(dw)
        return ids, w.detach()

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        ids, w = step()
    grad = x.grad
    with torch.no_grad():
        x.copy_(torch.randn((130, 16), generator=torch.Generator().manual_seed(3)))
    graph.replay()
    torch.cuda.synchronize()
    ids2, w2 = step()
    assert torch.equal(ids, ids2) and torch.equal(w, w2) and torch.equal(grad, x.grad)


@pytest.mark.parametrize("how", ["object", "handle"])
def test_another_stream(how):
    """Calls with `stream` run there, on memory of its own: work that is still
    queued on the current stream is not waited for, and its memory not reused."""
    s = torch.cuda.Stream()
    arg = s if how == "object" else s.cuda_stream
    X = normal((500, 1000), torch.bfloat16, 1)
    w, sw = random_blocks((300, 1000), 2, 120, 125)
    want = tg.gemm_mxfp4(*tg.quant_mxfp4(X), w, sw)
    back = tg.dequant_mxfp4(*tg.quant_mxfp4(X), 1000)
    s.wait_stream(torch.cuda.current_stream())
    q, qs = tg.quant_mxfp4(X, stream=arg)
    C = tg.gemm_mxfp4(q, qs, w, sw, stream=arg)
    Y = tg.dequant_mxfp4(q, qs, 1000, stream=arg)
    s.synchronize()
    assert torch.equal(C, want) and torch.equal(Y, back)
    with torch.cuda.stream(s):
        assert torch.equal(tg.gemm_mxfp4(*tg.quant_mxfp4(X), w, sw), want)
    torch.cuda.synchronize()


def test_calls_at_once():
    """The same product on several streams at the same time: nothing is shared."""
    (a, sa), (w, sw) = random_blocks((400, 2048), 1), random_blocks((2000, 2048), 2)
    want = tg.gemm_mxfp4(a, sa, w, sw)
    few = tg.gemm_mxfp4(a[:9], sa[:9], w, sw)
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append((tg.gemm_mxfp4(a, sa, w, sw), want))
                outs.append((tg.gemm_mxfp4(a[:9], sa[:9], w, sw), few))
    torch.cuda.synchronize()
    assert all(torch.equal(got, ref) for got, ref in outs)


@pytest.mark.parametrize("M", [5, 300])
def test_rows_far_apart(M):
    """Pitches of 16 MiB: the last rows lie past 4 GiB."""
    N, K, pitch = 300, 1056, 1 << 24
    big = torch.zeros(N, pitch, dtype=torch.uint8, device="cuda")
    (a, sa), (w, sw) = random_blocks((M, K), 1), random_blocks((N, K), 2)
    W, S, A, SA = big[:, :K // 2], big[:, 4096:4096 + K // 32], big[:M, 8192:8192 + K // 2], big[:M, 16384:16384 + K // 32]
    for t, v in ((W, w), (S, sw), (A, a), (SA, sa)):
        t.copy_(v)
    want = tg.gemm_mxfp4(a, sa, w, sw)
    assert torch.equal(tg.gemm_mxfp4(A, SA, W, S), want)
    far = big.view(torch.bfloat16)[:M, 1 << 20:(1 << 20) + K]
    X = normal((M, K), torch.bfloat16, 3)
    far.copy_(X)
    q, s = quantised(X)
    got = tg.quant_mxfp4(far, Q=A, scales=SA)
    assert torch.equal(got[0].cpu(), q) and torch.equal(got[1].cpu(), s)
    out = big.view(torch.bfloat16)[:M, 1 << 21:(1 << 21) + K]
    tg.dequant_mxfp4(A, SA, C=out)
    assert torch.equal(out.double().cpu(), values(q, s))
    # experts far apart
    We, Se = big[:2 * (N // 2)].view(2, N // 2, pitch)[:, :, :K // 2], big.view(2, N // 2, pitch)[:, :, 4096:4096 + K // 32]
    C = tg.gemm_grouped_mxfp4(a, sa, offsets_of([2, M - 2]), We, Se)
    assert torch.equal(C[:2], want[:2, :N // 2]) and torch.equal(C[2:], want[2:, N // 2:])


def test_logits_far_apart():
    T, E, pitch = 300, 64, 1 << 23
    big = torch.zeros(T, pitch, device="cuda")
    x = torch.randn((T, E), generator=torch.Generator().manual_seed(1)).cuda()
    far = big[:, :E]
    far.copy_(x)
    far.requires_grad_(True)
    ids, w = tg.expert_route(far, 4, renorm=False)
    want = tg.expert_route(x, 4, renorm=False)
    assert torch.equal(ids, want[0]) and torch.equal(w.detach(), want[1])
    dx, = torch.autograd.grad(w.sum(), far)
    y = x.clone().requires_grad_(True)
    dy, = torch.autograd.grad(tg.expert_route(y, 4, renorm=False)[1].sum(), y)
    assert torch.equal(dx, dy)


@pytest.mark.parametrize("offsets", [[0, 900, 30, 500], [5, 2, 2, 9], [-7, 100, 2000000000, 40], [400, 300, 200, 100],
                                     [0, -1, -1, 600], [0, 0, 0, 0], [2147483647, 0, 5, 600]])
def test_offsets_that_no_sort_writes(offsets):
    """They lead nowhere outside the matrices: what is beside C stays, the call
    ends in time, and the next one is right."""
    R, N, K = 600, 300, 640
    (a, sa), (w, sw) = random_blocks((R, K), 1), random_blocks((3, N, K), 2)
    big = torch.full((R + 4, 320), 7.0, dtype=torch.bfloat16, device="cuda")
    tg.gemm_grouped_mxfp4(a, sa, torch.tensor(offsets, dtype=torch.int32, device="cuda"), w, sw, C=big[2:-2, 8:308])
    assert tg.last_device_status() == 0
    big[2:-2, 8:308] = 7.0
    assert bool((big == 7.0).all())
    C = tg.gemm_grouped_mxfp4(a, sa, offsets_of([200, 0, 400]), w, sw)
    for e, part in ((0, slice(0, 200)), (2, slice(200, 600))):
        close(C[part], *product(values(a[part], sa[part]), values(w[e], sw[e]), torch.bfloat16))


@pytest.mark.parametrize("R,E", [(1, 1024), (700, 1024), (2000, 1023)])
def test_the_most_groups(R, E):
    counts = [0] * E
    for i in range(R):
        counts[(i * 313) % E] += 1
    a, sa = random_blocks((R, 64), 1)
    w, sw = random_blocks((E, 24, 64), 2)
    C = tg.gemm_grouped_mxfp4(a, sa, offsets_of(counts), w, sw)
    group = torch.repeat_interleave(torch.arange(E), torch.tensor(counts)).cuda()
    A, W = values(a, sa), values(w, sw)[group]
    ref = torch.einsum("rk,rnk->rn", A, W)
    mags = torch.einsum("rk,rnk->rn", A.abs(), W.abs())
    close(C, ref, ref.abs() * 2.0 ** -8 * 1.01 + 64 * 2.0 ** -23 * mags + 2.0 ** -134)


def test_long_sums():
    """A sum of 2^21 terms, whole and split over a cluster."""
    K = 1 << 21
    a, sa = random_blocks((3, K), 1, 110, 112)
    w, sw = random_blocks((130, K), 2, 110, 112)
    C = tg.gemm_mxfp4(a, sa, w, sw)
    A, W = values(a, sa), values(w, sw)
    close(C, A @ W.t(), (A @ W.t()).abs() * 2.0 ** -8 * 1.01 + K * 2.0 ** -23 * (A.abs() @ W.abs().t()))


@pytest.mark.parametrize("M,N,K", [(16, 8192, 4096), (1000, 1000, 2048), (3, 200, 8192)])
def test_repeated_calls_are_identical(M, N, K):
    (a, sa), (w, sw) = random_blocks((M, K), 1), random_blocks((N, K), 2)
    want = tg.gemm_mxfp4(a, sa, w, sw)
    assert all(torch.equal(tg.gemm_mxfp4(a, sa, w, sw), want) for _ in range(10))


def test_many_tiles_a_pair():
    """Every pair of CTAs takes several tiles, whole and in pieces, so that both
    accumulators come round with and without shared columns."""
    (a, sa), (w, sw) = random_blocks((3000, 512), 1), random_blocks((5000, 512), 2)
    C = tg.gemm_mxfp4(a, sa, w, sw)
    close(C, *product(values(a, sa), values(w, sw), torch.bfloat16))
    counts = [256, 32, 224, 240, 256, 31, 1, 255, 700, 0, 208, 256, 256, 129]
    R = sum(counts)
    (a, sa), (w, sw) = random_blocks((R, 768), 3), random_blocks((len(counts), 4000, 768), 4)
    C = tg.gemm_grouped_mxfp4(a, sa, offsets_of(counts), w, sw)
    at = 0
    for e, n in enumerate(counts):
        close(C[at:at + n], *product(values(a[at:at + n], sa[at:at + n]), values(w[e], sw[e]), torch.bfloat16), f"group {e}")
        at += n


@pytest.mark.parametrize("T,k,H", [(2400, 2, 1000), (1250, 3, 1090), (1250, 2, 1033), (1200, 2, 1279), (1200, 1, 2048),
                                   (820, 2, 2051)])
def test_quant_sorted_of_many_rows(T, k, H):
    """Enough rows for four blocks of 256 values a warp, which writes the scales of
    a place in words: whole ones, and parts of one at a row's end."""
    ids = torch.randint(-1, 9, (T, k), generator=torch.Generator().manual_seed(T)).int().cuda()
    plan = tg.expert_sort(ids, 8)
    X = normal((T, H), torch.bfloat16, seed=H)
    bq, Q = guarded(T * k, (H + 1) // 2)
    bs, S = guarded(T * k, -(-H // 32))
    tg.quant_mxfp4(X, plan, Q=Q, scales=S)
    q, s = tg.quant_mxfp4(X)
    want = quantised(X[:40])
    assert torch.equal(q[:40].cpu(), want[0]) and torch.equal(s[:40].cpu(), want[1])
    token, kept = plan.src.long() // k, int(plan.offsets[-1])
    q, s = q[token], s[token]
    q[kept:] = 0
    s[kept:] = 0
    assert 0 < kept < T * k and torch.equal(Q, q) and torch.equal(S, s)
    untouched(bq, Q)
    untouched(bs, S)


@pytest.mark.parametrize("M,most", [(1400, 1), (4000, 6)])
def test_more_items_than_a_pair_lists(M, most):
    """Items past those that a pair works out beforehand: groups of a few rows (some of
    none, rows behind the last) on enough column tiles for more than 64 a pair."""
    E, N, K = 1024, 1500, 96
    counts = torch.randint(1, most + 1, (E,), generator=torch.Generator().manual_seed(M))
    counts[::7] = 0
    counts[5] = 300
    off, live = offsets_of(counts.tolist()), int(counts.sum())
    assert live < M
    tiles = int(((counts + 255) // 256).sum()) + (M - live + 255) // 256
    assert tiles * -(-N // 256) > 65 * (torch.cuda.get_device_properties(0).multi_processor_count // 2)
    a, sa = random_blocks((M, K), 1)
    w, sw = random_blocks((E, N, K), 2)
    C = tg.gemm_grouped_mxfp4(a, sa, off, w, sw)
    assert tg.last_device_status() == 0
    group = torch.repeat_interleave(torch.arange(E), counts).cuda()
    av, wv = values(a, sa), values(w, sw)
    for r0 in range(0, live, 256):
        rows = slice(r0, min(r0 + 256, live))
        x, v = av[rows, None, :], wv[group[rows]]
        ref = (v @ x.transpose(1, 2))[..., 0]
        mags = (v.abs() @ x.abs().transpose(1, 2))[..., 0]
        close(C[rows], ref, ref.abs() * 2.0 ** -8 * 1.01 + K * 2.0 ** -23 * mags + 2.0 ** -134)
    assert not bool(C[live:].any())



def test_second_device_is_named():
    """Operands on two devices, or on the host, are refused before any launch."""
    q, s = random_blocks((4, 64), 1)
    with pytest.raises(ValueError):
        tg.gemm_mxfp4(q, s, q.cpu(), s.cpu())
    with pytest.raises(ValueError):
        tg.quant_mxfp4(normal((4, 64), torch.bfloat16, 1), Q=q.cpu())
    with pytest.raises(ValueError):
        tg.expert_route(torch.zeros(4, 8, device="cuda"), 2, bias=torch.zeros(8))


def test_nothing_to_do():
    """No rows, no columns, no tokens: results of the right shapes, no launch
    that would fail."""
    bf = torch.bfloat16
    for M, K in ((0, 64), (5, 0), (0, 0)):
        q, s = tg.quant_mxfp4(torch.zeros(M, K, dtype=bf, device="cuda"))
        assert q.shape == (M, K // 2) and s.shape == (M, K // 32)
        assert tg.dequant_mxfp4(q, s).shape == (M, K)
    ids, w = tg.expert_route(torch.zeros(0, 8, device="cuda"), 2)
    plan = tg.expert_sort(ids, 8)
    q, s = tg.quant_mxfp4(torch.zeros(0, 64, dtype=bf, device="cuda"), plan)
    W, S = random_blocks((8, 40, 64), 1)
    y = tg.gemm_grouped_mxfp4(q, s, plan, W, S)
    assert y.shape == (0, 40) and tg.expert_combine(y, plan, w).shape == (0, 40)
    # no k: zeros, groups or not
    none, nos = torch.zeros(6, 0, dtype=torch.uint8, device="cuda"), torch.zeros(6, 0, dtype=torch.uint8, device="cuda")
    W0 = torch.zeros(2, 40, 0, dtype=torch.uint8, device="cuda")
    C = tg.gemm_grouped_mxfp4(none, nos, offsets_of([2, 4]), W0, W0)
    assert C.shape == (6, 40) and not C.any()
    # every choice dropped
    plan = tg.expert_sort(torch.full((5, 2), -1, dtype=torch.int32, device="cuda"), 8)
    q, s = tg.quant_mxfp4(normal((5, 64), bf, 1), plan)
    assert not q.any() and not s.any()
    assert not tg.gemm_grouped_mxfp4(q, s, plan, W, S).any()
    assert tg.last_device_status() == 0


def test_refusals_of_the_library():
    """Limits and alignment that only the entry points check."""
    q, s = random_blocks((4, 64), 1)
    odd = torch.zeros(4 * 40 + 8, dtype=torch.uint8, device="cuda")
    for call, code in [
            (lambda: tg.expert_route(torch.zeros(4, 64, device="cuda"), 33), 3),
            (lambda: tg.expert_route(torch.zeros(4, 1025, device="cuda"), 2), 3),
            (lambda: tg.expert_route(torch.zeros(4, 64, device="cuda"), 65), 1),
            (lambda: tg.expert_route(torch.zeros(4, 64, device="cuda"), 9, groups=8, topk_groups=1), 1),
            (lambda: tg.expert_route(torch.zeros(4, 64, device="cuda"), 2, groups=5), 1),
            (lambda: tg.gemm_mxfp4(odd[8:].view(4, 40)[:, :32], s, q, s), 2),
            (lambda: tg.gemm_mxfp4(odd[:160].view(4, 40)[:, :32], s, q, s), 2),
            (lambda: tg.dequant_mxfp4(q, s, C=torch.zeros(4, 68, dtype=torch.bfloat16, device="cuda")[:, :64]), 2),
            (lambda: tg.quant_mxfp4(normal((4, 64), torch.bfloat16, 1), Q=odd[:160].view(4, 40)[:, :32]), 2)]:
        with pytest.raises(tg.TgError) as e:
            call()
        assert e.value.code == code
