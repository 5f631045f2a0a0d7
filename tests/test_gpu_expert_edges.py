"""Edges of the 8-bit and experts' operators on a B200: group ends of every
kind beside foreign rows, positions outside the rows, the most groups."""
import os
import subprocess
import sys
import textwrap

import pytest
import torch

from expert_util import DTYPES, H, TINY, close, normal, offsets_of, pitched, positive, product16
from gpu_util import SENTINEL16, check_guard, guarded_out

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


# ------------------------------------------------------ widths of any alignment

@pytest.mark.parametrize("D,F,shift", [(11, 11, 0), (8, 11, 0), (11, 8, 0), (7, 16, 0), (8, 16, 3)])
@pytest.mark.parametrize("stored", ["plain", "transposed"])
def test_layer_of_any_width(tg, D, F, shift, stored):
    """Ordinary contiguous tensors whose rows do not start on 16-byte
    boundaries, or (shift) views that start off one, through a whole layer and
    its gradients.  All values are -1, 0 or 1, the router's weights 1, D F <= 128
    and at most 22 rows: no stage's result exceeds 256, to which bfloat16 holds
    every integer, so each equals the 64-bit one."""
    E, T, k = 3, 11, 2
    g = torch.Generator().manual_seed(1)

    def small(*shape):
        flat = torch.zeros(torch.Size(shape).numel() + shift, dtype=torch.bfloat16, device="cuda")
        flat[shift:] = torch.randint(-1, 2, (flat.numel() - shift,), generator=g).to(torch.bfloat16).cuda()
        return flat[shift:].view(shape)

    x, W1, W2, gy = small(T, D), small(E, D, F), small(E, F, D), small(T, D)
    if stored == "transposed":
        W1, W2 = small(E, F, D), small(E, D, F)
    ids = torch.randint(0, E + 1, (T, k), generator=g).cuda()                 # E: dropped
    leaves = [t.requires_grad_(True) for t in (x, W1, W2, torch.ones((T, k), device="cuda"))]

    def view(w):
        return w.transpose(1, 2) if stored == "transposed" else w

    plan = tg.expert_sort(ids, E)
    h = torch.relu(tg.expert_matmul(tg.expert_gather(x, plan), view(W1), plan))
    y = tg.expert_combine(tg.expert_matmul(h.contiguous(), view(W2), plan), plan, leaves[3])
    got = torch.autograd.grad(y, leaves, gy)
    _status(tg)
    d = [t.detach().double().requires_grad_(True) for t in leaves]
    hot = torch.nn.functional.one_hot(ids, E + 1)[..., :E].double()           # T x k x E
    per = torch.einsum("td,edf->tef", d[0], view(d[1]))
    per = torch.einsum("tef,efd->ted", torch.relu(per), view(d[2]))
    out = torch.einsum("tke,tk,ted->td", hot, d[3], per)
    want = torch.autograd.grad(out, d, gy.double())
    for a, b in zip([y.detach(), *got], [out.detach(), *want]):
        assert torch.equal(a.double(), b)


def test_moves_of_any_width(tg):
    """Gather and combine on dense rows of odd widths and on views that start
    off a 16-byte boundary, 16-bit and int8, against the aligned call."""
    ids = torch.tensor([[0, 2], [1, -1], [2, 0], [7, 2], [0, 1]], device="cuda")
    plan = tg.expert_sort(ids, 3)
    for W in (1, 9, 16, 515):
        X = normal((5, W), torch.bfloat16, 1)
        Y = normal((10, W), torch.float16, 2)
        q, s = torch.randint(-128, 128, (5, W), dtype=torch.int8, device="cuda"), positive((5,), 3)
        qp = pitched((5, W), torch.int8)
        qp.copy_(q)
        w = positive((5, 2), 4)

        def off(t):                                           # the same rows one element off
            return torch.cat([t[:, :1], t], 1)[:, 1:]

        for f in (lambda t: t.contiguous(), off, lambda t: t.t().contiguous().t()):
            assert torch.equal(tg.expert_gather(f(X), plan), tg.expert_gather(X, plan))
            assert torch.equal(tg.expert_combine(f(Y), plan, w), tg.expert_combine(Y, plan, w))
            a, b = tg.expert_gather(f(q), plan, scales=s), tg.expert_gather(qp, plan, scales=s)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        one = X[:1].expand(5, W)
        assert torch.equal(tg.expert_gather(one, plan), tg.expert_gather(one.contiguous(), plan))
    _status(tg)


# ------------------------------------------------- positions outside the rows

@pytest.mark.parametrize("kept", [4, 2, 0, -7, 2147483647])
@pytest.mark.parametrize("pos", [[[0, 4], [5, -1]], [[-1, 1], [2, 4]], [[3, -3], [0, 6]], [[-2147483648, 2], [2147483647, 3]],
                                 [[0, 1], [2, 3]]])
def test_positions_outside_the_rows_write_nothing(tg, pos, kept):
    """4 rows inside a buffer of sentinels, positions just outside them: nothing
    but the rows that a position names is written, and these as they should be."""
    from tiled_dense_gemm_tma_b200 import binding
    T, k, H, n = 2, 2, 40, 4
    live = min(max(kept, 0), n)
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    o = torch.tensor([0, kept], dtype=torch.int32, device="cuda")
    X, Y, g = normal((T, H), torch.bfloat16, 1), normal((n, H), torch.bfloat16, 2), normal((T, H), torch.bfloat16, 3)
    w, s = positive((T, k), 4), positive((T,), 5)
    named = {r: (t, j) for t, row in enumerate(pos) for j, r in enumerate(row) if 0 <= r < n}

    def rows_are(big, C, want):
        """C's rows as in `want` (row -> values), all else the sentinel."""
        ref = torch.full_like(big, SENTINEL16, dtype=torch.int16).view(torch.bfloat16)
        pr, pc = 3, 8
        for r, v in want.items():
            ref[pr + r, pc:pc + H] = v
        assert torch.equal(big.view(torch.int16), ref.view(torch.int16))

    # gather, with scales
    big, C, _ = guarded_out(n, H, "bf16")
    ss = torch.full((n + 6,), -5.0, device="cuda")
    binding._launch("tg_expert_gather", X.device, None, T, k, H, 2, X.data_ptr(), X.stride(0), s.data_ptr(), p.data_ptr(),
                    o[1:].data_ptr(), C.data_ptr(), C.stride(0), ss[3:].data_ptr())
    rows_are(big, C, {r: X[t] if r < live else 0 for r, (t, _) in named.items()})
    want = torch.full_like(ss, -5.0)
    for r, (t, _) in named.items():
        want[3 + r] = s[t] if r < live else 0
    assert torch.equal(ss, want)
    # combine
    big, C, _ = guarded_out(T, H, "bf16")
    binding._launch("tg_expert_combine", X.device, None, T, k, H, 1, Y.data_ptr(), Y.stride(0), p.data_ptr(),
                    o[1:].data_ptr(), w.data_ptr(), C.data_ptr(), C.stride(0))
    check_guard(big, "bf16", T, H, (3, 8))
    counts = [[0 <= r < live for r in row] for row in pos]
    for t in range(T):
        terms = [w[t, j].double() * Y[pos[t][j]].double() for j in range(k) if counts[t][j]]
        ref = sum(terms, torch.zeros(H, dtype=torch.float64, device="cuda"))
        mags = sum((v.abs() for v in terms), torch.zeros_like(ref))
        close(C[t], ref, ref.abs() * 2.0 ** -8 * 1.01 + 3 * 2.0 ** -24 * mags + 2.0 ** -134, f"token {t}")
    # its gradient
    big, C, _ = guarded_out(n, H, "bf16")
    dw = torch.full((T * k + 6,), -5.0, device="cuda")
    binding._launch("tg_expert_combine_grad", X.device, None, T, k, H, 1, Y.data_ptr(), Y.stride(0), g.data_ptr(),
                    g.stride(0), p.data_ptr(), o[1:].data_ptr(), w.data_ptr(), C.data_ptr(), C.stride(0), dw[3:].data_ptr())
    rows_are(big, C, {r: (w[t, j] * g[t].float()).to(torch.bfloat16) if r < live else 0 for r, (t, j) in named.items()})
    assert bool((dw[:3] == -5).all()) and bool((dw[3 + T * k:] == -5).all())
    for t in range(T):
        for j in range(k):
            got = dw[3 + t * k + j].item()
            if not counts[t][j]:
                assert got == 0
                continue
            prod = Y[pos[t][j]].double() * g[t].double()
            assert abs(got - prod.sum().item()) <= H * 2.0 ** -24 * prod.abs().sum().item()
    _status(tg)


# ------------------------------------------------------------ the most groups

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("R,E", [(1, 1024), (5, 1000), (700, 1024), (3000, 1024), (2500, 1023)])
def test_gradients_of_the_most_groups(tg, R, E, dtype):
    """Every group's own weights and rows enter its results, near the limit of
    1024 groups; weights of distinct sizes, so that another group's would show."""
    dt = DTYPES[dtype]
    counts = [0] * E
    for i in range(R):
        counts[(i * 313) % E] += 1
    X = normal((R, 24), dt, 1).requires_grad_(True)
    W = normal((E, 24, 16), dt, 2)
    W *= (torch.arange(E, device="cuda") % 7 + 1)[:, None, None]
    W.requires_grad_(True)
    g = normal((R, 16), dt, 3)
    Y = tg.expert_matmul(X, W, offsets_of(counts))
    dX, dW = torch.autograd.grad(Y, (X, W), g)
    _status(tg)
    row = 0
    for e, n in enumerate(counts):
        if not n:
            assert not dW[e].any()
            continue
        part = slice(row, row + n)
        for got, a, b in ((Y.detach()[part], X.detach()[part], W.detach()[e]), (dX[part], g[part], W.detach()[e].t()),
                          (dW[e], X.detach()[part].t(), g[part])):
            close(got, *product16(a, b, dt), f"group {e}")
        row += n
    assert row == R


# -------------------------------------- combine's gradient at its variants' limits

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,k,W", [(256, 3, 520), (257, 3, 520), (300, 5, 512), (300, 2, 513), (512, 2, 2056),
                                   (513, 2, 2056), (600, 4, 2048), (513, 3, 4099), (1500, 7, 1000)])
def test_combine_gradients_of_many_tokens(tg, T, k, W, dtype):
    """Either side of where the number of threads a token changes."""
    dt = DTYPES[dtype]
    E = 11
    g0 = torch.Generator().manual_seed(T)
    ids = torch.randint(0, E + 1, (T, k), generator=g0).cuda()               # E: dropped
    plan = tg.expert_sort(ids, E)
    Y = normal((T * k, W), dt, 1).requires_grad_(True)
    w = normal((T, k), torch.float32, 2).contiguous().requires_grad_(True)
    g = normal((T, W), dt, 3)
    dY, dw = torch.autograd.grad(tg.expert_combine(Y, plan, w), (Y, w), g)
    _status(tg)
    kept = ids < E
    pos = plan.pos.long()
    wk = torch.where(kept, w.detach().double(), 0.0)
    want = torch.zeros(T * k, W, dtype=torch.float64, device="cuda")
    want[pos.reshape(-1)] = (wk[:, :, None] * g.double()[:, None, :]).reshape(T * k, W)
    close(dY, want, want.abs() * (H[dt] * 1.01 + 2.0 ** -24) + TINY[dt], "dY")
    prod = torch.where(kept[:, :, None], Y.detach().double()[pos], 0) * g.double()[:, None, :]
    close(dw, prod.sum(2), W * 2.0 ** -24 * prod.abs().sum(2) + 2.0 ** -149, "dw")


# ------------------------------------------------------- a captured backward pass

def test_captured_backward_into_grads(tg):
    """A whole step with backward() into the leaves' grads, captured as torch
    asks (a warm-up on the capture's stream, its graph gone before the capture),
    replayed on new contents: the grads of an eager step, bit for bit.  Groups end
    inside 16-row steps."""
    T, k, E, D, F = 700, 3, 6, 80, 136
    g0 = torch.Generator().manual_seed(3)
    ids = torch.randint(0, E + 1, (T, k), generator=g0).cuda()
    x, W1, W2 = (normal(s, torch.bfloat16, i, 0.1).requires_grad_(True)
                 for i, s in enumerate([(T, D), (E, D, F), (E, F, D)]))
    w = positive((T, k), 4).requires_grad_(True)
    gy = normal((T, D), torch.bfloat16, 5)
    leaves = (x, W1, W2, w)

    def step():
        for t in leaves:
            t.grad = None
        plan = tg.expert_sort(ids, E)
        h = torch.relu(tg.expert_matmul(tg.expert_gather(x, plan), W1, plan))
        tg.expert_combine(tg.expert_matmul(h, W2, plan), plan, w).backward(gy)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    kept = [t.grad for t in leaves]
    with torch.no_grad():
        ids.copy_(torch.randint(0, E + 1, (T, k), generator=g0))
        x.copy_(normal((T, D), torch.bfloat16, 9))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    step()
    _status(tg)
    for t, got in zip(leaves, kept):
        assert torch.equal(t.grad, got)
