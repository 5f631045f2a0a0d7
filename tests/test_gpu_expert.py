"""The experts' operators on a B200: sort, gather, products, combine and their
gradients against their definitions in 64 bits."""
import pytest
import torch

from expert_util import (DTYPES, H, TINY, close, ints8, normal, offsets_of, pitched, positive, product16,
                         product8)
from gpu_util import check_guard, guarded_out

pytestmark = pytest.mark.gpu


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


# ------------------------------------------------------------------- sort

def sort_ref(ids, E):
    flat = ids.reshape(-1).tolist()
    buckets = [[] for _ in range(E + 1)]
    for i, e in enumerate(flat):
        buckets[e if 0 <= e < E else E].append(i)
    offsets = [0]
    for b in buckets[:E]:
        offsets.append(offsets[-1] + len(b))
    src = [i for b in buckets for i in b]
    pos = [0] * len(flat)
    for r, i in enumerate(src):
        pos[i] = r
    return offsets, pos, src


def make_ids(T, k, E, seed, drop=0.0, dtype=torch.int64):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, E, (T, k), generator=g)
    if drop:
        gone = torch.rand((T, k), generator=g) < drop
        ids[gone] = torch.where(ids[gone] % 2 == 0, -1, E + ids[gone])
    return ids.to(dtype).cuda()


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("T,k,E,drop", [(0, 2, 4, 0), (1, 1, 1, 0), (1, 8, 8, 0.5), (16, 2, 8, 0), (33, 3, 5, 0.3),
                                        (700, 4, 64, 0.01), (1024, 8, 128, 0), (1025, 8, 129, 0.1), (2731, 3, 1024, 0),
                                        (9000, 8, 256, 0.02), (40000, 8, 1024, 0.1), (100, 2, 8, 1.0),
                                        (50000, 1, 1, 0.5), (148 * 2048 + 77, 1, 7, 0)])
def test_sort(tg, T, k, E, drop, dtype):
    ids = make_ids(T, k, E, T + E, drop, dtype)
    plan = tg.expert_sort(ids, E)
    _status(tg)
    offsets, pos, src = sort_ref(ids, E)
    assert plan.offsets.tolist() == offsets
    assert plan.src.tolist() == src
    assert plan.pos.reshape(-1).tolist() == pos and tuple(plan.pos.shape) == (T, k)


def test_sort_far_numbers_are_dropped(tg):
    """64-bit numbers whose low words name an expert."""
    ids = torch.tensor([[1, 1 << 32], [-(1 << 32), (1 << 33) + 1], [0, -1]], device="cuda")
    plan = tg.expert_sort(ids, 2)
    assert plan.offsets.tolist() == [0, 1, 2]
    assert plan.src.tolist() == [4, 0, 1, 2, 3, 5]


# -------------------------------------------------------- gather, combine

MOVES = [(1, 1, 1, 1, 0), (3, 2, 4, 7, 0), (16, 2, 8, 4096, 0), (50, 6, 16, 1030, 0.2), (257, 5, 9, 63, 0.5),
         (100, 8, 128, 2048, 0.02), (20, 33, 40, 136, 0.1), (5, 3, 8, 20001, 0.3), (12, 2, 4, 64, 1.0)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,k,E,W,drop", MOVES)
def test_gather_and_gradient(tg, T, k, E, W, drop, dtype):
    dt = DTYPES[dtype]
    ids = make_ids(T, k, E, T, drop)
    plan = tg.expert_sort(ids, E)
    X = normal((T, W), dt, 1, extra=1).requires_grad_(True)
    Xs = tg.expert_gather(X, plan)
    kept = ((ids >= 0) & (ids < E)).reshape(-1)
    pos = plan.pos.reshape(-1).long()
    ref = torch.zeros(T * k, W, dtype=dt, device="cuda")
    ref[pos[kept]] = X.detach().repeat_interleave(k, 0)[kept]
    assert torch.equal(Xs.detach(), ref)
    g = normal((T * k, W), dt, 2)
    dX, = torch.autograd.grad(Xs, X, g)
    _status(tg)
    rows = torch.where(kept[:, None], g[pos].double(), 0).view(T, k, W)
    want = rows.sum(1)
    close(dX, want, want.abs() * H[dt] * 1.01 + TINY[dt] + k * 2.0 ** -24 * rows.abs().sum(1))


def test_gather_int8_with_scales(tg):
    ids = make_ids(40, 3, 6, 1, 0.2)
    plan = tg.expert_sort(ids, 6)
    X, s = ints8((40, 515), 1), positive((40,), 2)
    Xs, ss = tg.expert_gather(X, plan, scales=s)
    _status(tg)
    n = int(plan.offsets[-1])
    tok = (plan.src // 3).long()
    assert torch.equal(Xs[:n], X[tok[:n]]) and not Xs[n:].any()
    assert torch.equal(ss[:n], s[tok[:n]]) and not ss[n:].any()
    assert torch.equal(tg.expert_gather(X, plan), Xs)


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,k,E,W,drop", MOVES)
def test_combine_and_gradients(tg, T, k, E, W, drop, dtype, weighted):
    dt = DTYPES[dtype]
    ids = make_ids(T, k, E, T + 5, drop)
    plan = tg.expert_sort(ids, E)
    Y = normal((T * k, W), dt, 1, extra=1).requires_grad_(True)
    w = normal((T, k), torch.float32, 2)[:, :].contiguous().requires_grad_(True) if weighted else None
    out = tg.expert_combine(Y, plan, w)
    kept = (ids >= 0) & (ids < E)
    wk = torch.where(kept, w.detach().double() if weighted else 1.0, 0.0)
    pos = plan.pos.long()
    rows = torch.where(kept[:, :, None], Y.detach().double()[pos], 0)
    terms = rows * wk[:, :, None]
    want = terms.sum(1)
    close(out.detach(), want, want.abs() * H[dt] * 1.01 + TINY[dt] + (k + 1) * 2.0 ** -24 * terms.abs().sum(1))
    g = normal((T, W), dt, 3)
    grads = torch.autograd.grad(out, (Y, w) if weighted else (Y,), g)
    _status(tg)
    dY = torch.zeros(T * k, W, dtype=torch.float64, device="cuda")
    dY[pos.reshape(-1)] = (wk[:, :, None] * g.double()[:, None, :]).reshape(T * k, W)
    close(grads[0], dY, dY.abs() * (H[dt] * 1.01 + 2.0 ** -24) + TINY[dt], "dY")
    if weighted:
        prod = rows * g.double()[:, None, :]
        close(grads[1], prod.sum(2), W * 2.0 ** -24 * prod.abs().sum(2) + 2.0 ** -149, "dw")


def test_infinite_rows_of_dropped_choices_do_not_count(tg):
    ids = torch.tensor([[0, -1], [1, 0]], device="cuda")
    plan = tg.expert_sort(ids, 2)
    Y = pitched((4, 16), torch.bfloat16)
    Y.fill_(1)
    Y[3] = float("nan")                                   # the dropped choice's row
    Y.requires_grad_(True)
    w = torch.full((2, 2), 2.0, device="cuda")
    w[0, 1] = float("inf")
    w.requires_grad_(True)
    out = tg.expert_combine(Y, plan, w)
    assert out.tolist() == [[2.0] * 16, [4.0] * 16]
    g = pitched((2, 16), torch.bfloat16)
    g.fill_(1)
    dY, dw = torch.autograd.grad(out, (Y, w), g)
    assert dY[:3].tolist() == [[2.0] * 16] * 3 and not dY[3].any()
    assert dw.tolist() == [[16.0, 0.0], [16.0, 16.0]]
    _status(tg)


# --------------------------------------------------------------- products

GROUPS = {
    "one": [37], "ones": [1, 1, 1, 1], "empty": [0, 0, 0], "edges": [255, 0, 256, 257, 0, 1, 31, 32, 33],
    "ends_empty": [0, 5, 0], "mixed": [300, 3, 0, 64, 129, 513], "many": [7] * 100 + [0] * 30 + [40],
}


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("groups,K,N,tail", [("one", 1, 1, 0), ("one", 64, 8, 3), ("ones", 65, 31, 0),
                                             ("empty", 16, 24, 9), ("empty", 8, 8, 0), ("edges", 130, 257, 5),
                                             ("edges", 63, 300, 0), ("ends_empty", 200, 129, 40),
                                             ("mixed", 520, 264, 11), ("many", 96, 136, 2), ("mixed", 1024, 72, 300)])
def test_product_and_gradients(tg, groups, K, N, tail, trans):
    dtype = "bf16" if (K + N) % 2 else "f16"
    dt = DTYPES[dtype]
    counts = GROUPS[groups]
    E, live = len(counts), sum(counts)
    R = live + tail
    offsets = offsets_of(counts)
    X = normal((R, K), dt, 1, extra=1).requires_grad_(True)
    S = normal((E, N, K) if trans else (E, K, N), dt, 2, K ** -0.5).requires_grad_(True)
    W = S.transpose(1, 2) if trans else S
    Y = tg.expert_matmul(X, W, offsets)
    g = normal((R, N), dt, 3, extra=1)
    if R:
        dX, dS = torch.autograd.grad(Y, (X, S), g)
    _status(tg)
    if not R:
        return
    x, w, gd = X.detach(), W.detach(), g
    at = 0
    for e, n in enumerate(counts):
        part = slice(at, at + n)
        ref, bound = product16(x[part], w[e], dt)
        close(Y.detach()[part], ref, bound, f"Y of group {e}")
        ref, bound = product16(gd[part], w[e].t(), dt)
        close(dX[part], ref, bound, f"dX of group {e}")
        ref, bound = product16(x[part].t(), gd[part], dt)
        got = dS[e].t() if trans else dS[e]
        close(got, ref, bound, f"dW of group {e}")
        at += n
    assert not Y.detach()[live:].any() and not dX[live:].any()


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("groups,K,N,tail", [("one", 1, 1, 0), ("ones", 129, 31, 2), ("edges", 256, 257, 5),
                                             ("mixed", 1000, 264, 11), ("many", 136, 136, 2), ("empty", 16, 24, 9)])
def test_product8(tg, groups, K, N, tail, trans):
    dtype = "bf16" if (K + N) % 2 else "f16"
    dt = DTYPES[dtype]
    counts = GROUPS[groups]
    E, live = len(counts), sum(counts)
    R = live + tail
    offsets = offsets_of(counts)
    A, B = ints8((R, K), 1, extra=1), ints8((E, N, K) if trans else (E, K, N), 2)
    rs, cs = positive((R,), 3, 1e-3, 2e-3), positive((E, N), 4, 1e-3, 2e-3)
    big, C, pad = guarded_out(R, N, dtype)
    tg.gemm_grouped_w8a8(A, rs, offsets, B, cs, C=C, trans_b=trans, relu=K % 2 == 0)
    _status(tg)
    at = 0
    for e, n in enumerate(counts):
        part = slice(at, at + n)
        ref, bound = product8(A[part], rs[part], B[e].t() if trans else B[e], cs[e], dt)
        close(C[part], ref.clamp(min=0) if K % 2 == 0 else ref, bound, f"group {e}")
        at += n
    assert not C[live:].any()
    check_guard(big, dtype, R, N, pad)


@pytest.mark.parametrize("N", [8, 40, 64, 200, 260])
def test_product_writes_only_its_output(tg, N):
    counts = [70, 0, 131, 3]
    A = normal((210, 100), torch.bfloat16, 1)
    B = normal((4, 100, N), torch.bfloat16, 2)
    big, C, pad = guarded_out(210, N, "bf16")
    tg.gemm_grouped(A, offsets_of(counts), B, C=C, relu=True)
    _status(tg)
    check_guard(big, "bf16", 210, N, pad)
    at = 0
    for e, n in enumerate(counts):
        ref, bound = product16(A[at:at + n], B[e], torch.bfloat16)
        close(C[at:at + n], ref.clamp(min=0), bound)
        at += n


@pytest.mark.parametrize("K,N", [(7, 9), (40, 72), (300, 65)])
def test_wgrad_writes_only_its_output(tg, K, N):
    """Into matrices with rows and columns to spare between them."""
    counts = [70, 0, 13]
    A, G = normal((90, K), torch.float16, 1), normal((90, N), torch.float16, 2)
    ld = -(-N // 8) * 8 + 8
    big = torch.full((3, K + 3, ld), 7.0, dtype=torch.float16, device="cuda")
    C = big[:, :K, :N]
    tg.gemm_grouped_wgrad(A, G, offsets_of(counts), C=C)
    _status(tg)
    assert bool((big[:, K:] == 7).all()) and bool((big[:, :, N:] == 7).all())
    at = 0
    for e, n in enumerate(counts):
        ref, bound = product16(A[at:at + n].t(), G[at:at + n], torch.float16)
        close(C[e], ref, bound)
        at += n


@pytest.mark.parametrize("n", [1, 15, 17, 63, 64, 65, 80, 100])
def test_nothing_leaks_between_groups(tg, n):
    """NaN and infinities in one group's rows and weights stay there: a group
    that ends inside a 16-row step or a 64-row block reads its neighbour's."""
    K, N = 72, 136
    counts = [n, 40, n]
    R = sum(counts) + 20
    X, g = normal((R, K), torch.bfloat16, 1), normal((R, N), torch.bfloat16, 2)
    W = normal((3, K, N), torch.bfloat16, 3)
    bad = slice(n, n + 40)
    X[bad], g[bad], W[1] = float("nan"), float("inf"), float("nan")
    X[-20:], g[-20:] = float("nan"), float("nan")         # behind the last group
    X.requires_grad_(True)
    W.requires_grad_(True)
    Y = tg.expert_matmul(X, W, offsets_of(counts))
    dX, dW = torch.autograd.grad(Y, (X, W), g)
    _status(tg)
    for got in (Y.detach(), dX):
        assert not torch.isnan(got[:n]).any() and not torch.isnan(got[n + 40:]).any()
        assert torch.isnan(got[bad]).all() and not got[-20:].any()
    assert torch.isfinite(dW[0]).all() and torch.isfinite(dW[2]).all() and torch.isnan(dW[1]).all()
    ref, bound = product16(X.detach()[:n].t(), g[:n], torch.bfloat16)
    close(dW[0], ref, bound)


def test_offsets_outside_the_rows_are_clamped(tg):
    """Bad offsets never lead outside the matrices: the calls return, report no
    time-out and write nothing outside C."""
    A, G = normal((50, 64), torch.bfloat16, 1), normal((50, 72), torch.bfloat16, 2)
    W = normal((3, 64, 72), torch.bfloat16, 3)
    for bad in ([-5, 20, 1000, 2000], [10, 5, 60, 3], [2 ** 31 - 1, -2 ** 31, 7, 2 ** 31 - 1]):
        o = torch.tensor(bad, dtype=torch.int32, device="cuda")
        big, C, pad = guarded_out(50, 72, "bf16")
        tg.gemm_grouped(A, o, W, C=C)
        wide = torch.full((4, 64, 72), 7.0, dtype=torch.bfloat16, device="cuda")
        tg.gemm_grouped_wgrad(A, G, o, C=wide[:3])
        _status(tg)
        check_guard(big, "bf16", 50, 72, pad)
        assert bool((wide[3] == 7).all())


def test_strided_weights(tg):
    """Matrices of a wider buffer, experts interleaved by row."""
    E, K, N = 3, 72, 40
    buf = normal((K, E, N + 24), torch.bfloat16, 1)
    W = buf.transpose(0, 1)[:, :, :N]                     # plane N + 24, pitch E * (N + 24)
    A = normal((60, K), torch.bfloat16, 2)
    counts = [10, 30, 20]
    C = tg.gemm_grouped(A, offsets_of(counts), W)
    _status(tg)
    at = 0
    for e, n in enumerate(counts):
        ref, bound = product16(A[at:at + n], W[e], torch.bfloat16)
        close(C[at:at + n], ref, bound)
        at += n


# ------------------------------------------------------------ as one layer

def layer(tg, x, scores, ids, W1, W2, E):
    plan = tg.expert_sort(ids, E)
    h = torch.relu(tg.expert_matmul(tg.expert_gather(x, plan), W1, plan))
    return tg.expert_combine(tg.expert_matmul(h, W2.transpose(1, 2), plan), plan, scores)


def make_layer(T=70, k=3, E=6, D=80, F=136, seed=0, drop=0.1):
    ids = make_ids(T, k, E, seed, drop)
    x = normal((T, D), torch.bfloat16, seed + 1)
    scores = positive((T, k), seed + 2, 0.1, 0.6)
    W1, W2 = normal((E, D, F), torch.bfloat16, seed + 3, D ** -0.5), normal((E, D, F), torch.bfloat16, seed + 4, F ** -0.5)
    return [t.requires_grad_(True) for t in (x, scores, W1, W2)], ids


def test_layer_against_64_bit_autograd(tg):
    """Router weights, two products and the joins, forward and backward.
    Every stage rounds once to bf16 (2^-8), forward four of them and backward
    four more; sums of at most 136 terms of alike sizes: 5 % of the largest
    value bounds them with room for the sums' growth."""
    E = 6
    leaves, ids = make_layer()
    y = layer(tg, leaves[0], leaves[1], ids, leaves[2], leaves[3], E)
    g = normal(tuple(y.shape), torch.bfloat16, 77)
    got = torch.autograd.grad(y, leaves, g)
    _status(tg)
    d = [t.detach().double().requires_grad_(True) for t in leaves]
    out = torch.zeros_like(d[0])
    for t in range(ids.shape[0]):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if 0 <= e < E:
                out = out.index_add(0, torch.tensor([t], device="cuda"),
                                    (d[1][t, j] * (torch.relu(d[0][t] @ d[2][e]) @ d[3][e].t()))[None])
    want = torch.autograd.grad(out, d, g.double())
    for a, b in zip([y.detach(), *got], [out.detach(), *want]):
        assert (a.double() - b).abs().max() <= 0.05 * b.abs().max()


def test_gradient_against_differences(tg):
    """d<Y, G>/dW along a direction: a step large enough that bf16's rounding
    of the weights is exact (integers), so only Y's own rounding counts."""
    counts = [40, 0, 25]
    X = ints8((65, 32), 1, -2, 3).to(torch.bfloat16)
    W = ints8((3, 32, 24), 2, -2, 3).to(torch.bfloat16).requires_grad_(True)
    G = ints8((65, 24), 3, -2, 3).to(torch.bfloat16)
    D = ints8((3, 32, 24), 4, -1, 2).to(torch.bfloat16)
    o = offsets_of(counts)

    def value(w):
        return (tg.gemm_grouped(X, o, w).double() * G.double()).sum()

    dW, = torch.autograd.grad(tg.expert_matmul(X, W, o), W, G)
    # |Y| <= 32 * 2 * 3 = 192 and |dW| <= 40 * 4 = 160 are integers below 256: exact in bf16
    diff = (value(W.detach() + D) - value(W.detach() - D)) / 2
    assert diff.item() == (dW.double() * D.double()).sum().item()
    _status(tg)


def test_two_graphs_side_by_side(tg):
    """Two captured layers replayed on two streams at once, each with its own
    inputs, against their eager runs."""
    E = 6
    runs = []
    for seed in (0, 50):
        leaves, ids = make_layer(T=400, seed=seed)
        with torch.no_grad():
            args = [t.detach() for t in leaves]
            eager = layer(tg, args[0], args[1], ids, args[2], args[3], E)
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                out = layer(tg, args[0], args[1], ids, args[2], args[3], E)
        runs.append((graph, s, out, eager, args, ids))        # a graph reads its inputs' memory: keep them
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, s, out, eager, *_ in runs:
            with torch.cuda.stream(s):
                graph.replay()
    _status(tg)
    for graph, s, out, eager, *_ in runs:
        assert torch.equal(out, eager)


def test_repeated_calls_give_the_same_bits(tg):
    leaves, ids = make_layer(T=300)
    first = None
    for _ in range(3):
        y = layer(tg, leaves[0], leaves[1], ids, leaves[2], leaves[3], 6)
        got = [y.detach(), *torch.autograd.grad(y, leaves, torch.ones_like(y))]
        if first is None:
            first = got
        assert all(torch.equal(a, b) for a, b in zip(first, got))
    _status(tg)


def test_captured_training_step(tg):
    """Forward and backward in one graph, many enough choices for the sort's two
    launches, replayed on new contents of the same buffers."""
    E = 7
    leaves, ids = make_layer(T=3000, k=3, E=E, seed=5)
    g = normal((3000, 80), torch.bfloat16, 9)

    def step():
        y = layer(tg, leaves[0], leaves[1], ids, leaves[2], leaves[3], E)
        return [y.detach(), *torch.autograd.grad(y, leaves, g)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    with torch.no_grad():
        ids.copy_(make_ids(3000, 3, E, 77, 0.2))
        leaves[0].copy_(normal((3000, 80), torch.bfloat16, 78))
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    eager = step()
    _status(tg)
    assert all(torch.equal(a, b) for a, b in zip(out, eager))


def test_layer_on_its_own_stream(tg):
    """Every operator on a stream that is not the default one, behind work that
    delays its inputs."""
    leaves, ids = make_layer(T=500)
    want = layer(tg, leaves[0], leaves[1], ids, leaves[2], leaves[3], 6).detach().clone()
    g = torch.ones_like(want)
    want_g = torch.autograd.grad(layer(tg, leaves[0], leaves[1], ids, leaves[2], leaves[3], 6), leaves, g)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        late = torch.full_like(ids, -1)
        late.copy_(ids)
        x = leaves[0].detach().clone().requires_grad_(True)
        y = layer(tg, x, leaves[1], late, leaves[2], leaves[3], 6)
        got_g = torch.autograd.grad(y, [x, *leaves[1:]], g)
    s.synchronize()
    _status(tg)
    assert torch.equal(y.detach(), want) and all(torch.equal(a, b) for a, b in zip(got_g, want_g))


@pytest.mark.parametrize("R,E", [(0, 3), (1, 1), (1, 1024), (5, 1000)])
def test_smallest_and_most_groups(tg, R, E):
    counts = [0] * E
    for i in range(R):
        counts[(i * 313) % E] += 1
    X = normal((R, 24), torch.bfloat16, 1).requires_grad_(True)
    W = normal((E, 24, 16), torch.bfloat16, 2).requires_grad_(True)
    Y = tg.expert_matmul(X, W, offsets_of(counts))
    dX, dW = torch.autograd.grad(Y, (X, W), normal((R, 16), torch.bfloat16, 3))
    _status(tg)
    assert tuple(Y.shape) == (R, 16) and tuple(dX.shape) == (R, 24)
    row = 0
    for e, n in enumerate(counts):
        if n:
            ref, bound = product16(X.detach()[row:row + n], W.detach()[e], torch.bfloat16)
            close(Y.detach()[row:row + n], ref, bound)
        else:
            assert not dW[e].any()
        row += n


def test_shared_gradient_of_expanded_weights(tg):
    """One matrix for all experts, expanded: its gradient adds all groups'."""
    counts = [20, 0, 33]
    X = ints8((53, 32), 1, -2, 3).to(torch.bfloat16)
    W1 = ints8((32, 24), 2, -1, 2).to(torch.bfloat16).requires_grad_(True)
    G = ints8((53, 24), 3, -1, 2).to(torch.bfloat16)
    Y = tg.expert_matmul(X, W1[None].expand(3, 32, 24), offsets_of(counts))
    dW, = torch.autograd.grad(Y, W1, G)
    _status(tg)
    # integers: |Y| <= 32 * 2, the groups' gradients at most 66, their sum at most 106: all exact
    assert torch.equal(Y.detach().double(), X.double() @ W1.detach().double())
    assert torch.equal(dW.double(), X.double().t() @ G.double())


def test_gather_the_same_token_to_one_expert_twice(tg):
    ids = torch.tensor([[1, 1], [0, 1]], device="cuda")
    plan = tg.expert_sort(ids, 2)
    assert plan.offsets.tolist() == [0, 1, 4] and plan.src.tolist() == [2, 0, 1, 3]
    X = normal((2, 24), torch.float16, 1).requires_grad_(True)
    Xs = tg.expert_gather(X, plan)
    assert torch.equal(Xs.detach(), X.detach()[[1, 0, 0, 1]])
    dX, = torch.autograd.grad(Xs, X, torch.ones(4, 24, dtype=torch.float16, device="cuda"))
    assert bool((dX == 2).all())
    _status(tg)


@pytest.mark.parametrize("pos", [[[7, 100]], [[-1, -2147483648]], [[2147483647, 1]]])
def test_positions_outside_the_rows_are_skipped(tg, pos):
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    for offsets in ([0, 2], [0, -7], [0, 2147483647]):
        plan = tg.ExpertPlan(torch.tensor(offsets, dtype=torch.int32, device="cuda"), p)
        X = normal((1, 40), torch.bfloat16, 1).requires_grad_(True)
        Y = normal((2, 40), torch.bfloat16, 2).requires_grad_(True)
        w = torch.ones((1, 2), device="cuda").requires_grad_(True)
        tg.expert_gather(X, plan).sum().backward()
        tg.expert_combine(Y, plan, w).sum().backward()
    _status(tg)


def test_rows_past_32_bit_offsets(tg):
    """More than 2^31 elements: the last rows are where they belong."""
    T, k, H = 300_001, 2, 4096                            # 2.46e9 sorted values
    ids = (torch.arange(T * k, device="cuda") % 3).view(T, k)
    plan = tg.expert_sort(ids, 3)
    X = torch.arange(T, device="cuda", dtype=torch.float32)[:, None].remainder(251).to(torch.bfloat16).expand(T, H)
    X = X.contiguous()
    Xs = tg.expert_gather(X, plan)
    tail = plan.src[-5:].long() // k
    assert torch.equal(Xs[-5:], X[tail])
    Y = tg.expert_combine(Xs, plan)
    assert torch.equal(Y[-5:], X[-5:] * 2)                # small integers: exact
    W = torch.zeros(3, 4096, 16, dtype=torch.bfloat16, device="cuda")
    W[:, 7, :] = 1
    P = tg.gemm_grouped(Xs, plan, W)
    assert torch.equal(P[-5:], X[tail][:, :16])
    del Y, P
    q, s = tg.quant_i8(Xs)
    _status(tg)
    top = Xs[-5:, :1].float().abs()
    assert torch.equal(q[-5:, :1].float() * s[-5:, None], torch.where(top > 0, 127 * (top / 127), 0))


def test_activations_kept_on_the_host(tg):
    """torch.autograd.graph.save_on_cpu gives back contiguous copies of the
    strided operands."""
    E, counts = 3, [20, 0, 33]
    o = offsets_of(counts)
    X = normal((53, 20), torch.bfloat16, 1, extra=1).requires_grad_(True)
    S = normal((E, 20, 13), torch.bfloat16, 2).requires_grad_(True)
    g = normal((53, 13), torch.bfloat16, 3)
    want = torch.autograd.grad(tg.expert_matmul(X, S, o), (X, S), g)
    with torch.autograd.graph.save_on_cpu():
        Y = tg.expert_matmul(X, S, o)
    got = torch.autograd.grad(Y, (X, S), g)
    _status(tg)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_moves_against_differences(tg):
    """Gather and combine are linear in each argument: central differences of
    <output, G> along a direction equal <gradient, direction> exactly on small
    integers (every sum below 256, exact in bf16)."""
    ids = make_ids(30, 4, 5, 3, 0.2)
    plan = tg.expert_sort(ids, 5)
    X, D = (ints8((30, 40), i, -3, 4).to(torch.bfloat16) for i in (1, 2))
    Y, F = (ints8((120, 40), i, -3, 4).to(torch.bfloat16) for i in (3, 4))
    w, v = (ints8((30, 4), i, -2, 3).float().contiguous() for i in (5, 6))
    Gx, Gy = ints8((120, 40), 7, -3, 4).to(torch.bfloat16), ints8((30, 40), 8, -3, 4).to(torch.bfloat16)

    def check(f, at, along, grad):
        diff = (f(at + along).double() - f(at - along).double()) / 2
        assert diff.item() == (grad.double() * along.double()).sum().item()

    x = X.clone().requires_grad_(True)
    dX, = torch.autograd.grad(tg.expert_gather(x, plan), x, Gx)
    check(lambda t: (tg.expert_gather(t, plan).double() * Gx.double()).sum(), X, D, dX)
    y, u = Y.clone().requires_grad_(True), w.clone().requires_grad_(True)
    dY, dw = torch.autograd.grad(tg.expert_combine(y, plan, u), (y, u), Gy)
    check(lambda t: (tg.expert_combine(t, plan, w).double() * Gy.double()).sum(), Y, F, dY)
    check(lambda t: (tg.expert_combine(Y, plan, t).double() * Gy.double()).sum(), w, v, dw)
    _status(tg)


def test_empty_products(tg):
    """No columns, no k: what is left of the outputs is zero."""
    o = offsets_of([3, 0, 2])
    for K, N in ((0, 16), (16, 0), (0, 0)):
        X = pitched((5, K), torch.bfloat16).requires_grad_(True)
        W = pitched((3, K, N), torch.bfloat16).requires_grad_(True)
        Y = tg.expert_matmul(X, W, o)
        dX, dW = torch.autograd.grad(Y, (X, W), torch.ones(5, N, dtype=torch.bfloat16, device="cuda"))
        assert tuple(Y.shape) == (5, N) and not Y.any()
        assert tuple(dX.shape) == (5, K) and tuple(dW.shape) == (3, K, N) and not dX.any() and not dW.any()
    A, B = ints8((5, 0), 1), ints8((0, 24), 2)
    C = tg.gemm_w8a8(A, positive((5,), 1), B, positive((24,), 2))
    assert tuple(C.shape) == (5, 24) and not C.any()
    q, s = tg.quant_i8(pitched((4, 0), torch.float16))
    assert tuple(q.shape) == (4, 0) and not s.any()
    for M in (0, 3):
        C = tg.gemm_w8a8(ints8((M, 16), 1), positive((M,), 1), ints8((16, 0 if M else 8), 2), positive((0 if M else 8,), 2))
        assert tuple(C.shape) == (M, 0 if M else 8)
    _status(tg)


@pytest.mark.parametrize("handle", [False, True])
def test_outputs_for_another_stream_use_its_memory(tg, handle):
    """A call on another stream does not write into memory that the current
    stream has freed but is still to use."""
    s = torch.cuda.Stream()
    A, B, o = normal((256, 64), torch.bfloat16, 1), normal((1, 64, 512), torch.bfloat16, 2), offsets_of([256])
    q, w = ints8((256, 64), 3), ints8((64, 512), 4)
    rs, cs = positive((256,), 5), positive((512,), 6)
    calls = [lambda st: tg.gemm_grouped(A, o, B, stream=st), lambda st: tg.gemm_w8a8(q, rs, w, cs, stream=st),
             lambda st: tg.gemm_grouped_w8a8(q, rs, o, w[None], cs[None], stream=st),
             lambda st: tg.gemm_grouped_wgrad(A, A, o, stream=st), lambda st: tg.quant_i8(A, stream=st)[0]]
    for call in calls:
        want = call(None).clone()
        torch.cuda.synchronize()
        late = torch.empty_like(want)
        torch.cuda._sleep(20_000_000)
        late.fill_(7)                                     # pending on the current stream
        del late                                          # its block is free for the current stream
        got = call(s.cuda_stream if handle else s)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        del got, want
    _status(tg)
