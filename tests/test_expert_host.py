"""Host checks of the 8-bit and experts' operators (no GPU): the entry points'
refusals, which come before any CUDA call, and the binding's marshalling,
checked with a fake library that reads its operands through the pointers,
pitches and planes it is given and computes in float64."""
import ctypes

import numpy as np
import pytest
import torch

from tiled_dense_gemm_tma_b200 import binding, build as tg_build

OK, INVALID, ALIGN, UNSUP = 0, 1, 2, 3
P = 0x10000          # a fake, 16-byte aligned "device" address (never dereferenced)
BIG = 1 << 31


@pytest.fixture(scope="module")
def lib():
    tg_build.build()
    return binding.load_library()


def call(fn, names, defaults, **kw):
    a = dict(defaults, **kw)
    assert set(kw) <= set(names)
    return fn(*[a[n] for n in names])


QUANT = "M K X ldx type Q ldq scales stream".split()
QUANT_OK = dict(M=4, K=16, X=P, ldx=16, type=1, Q=P, ldq=16, scales=P, stream=None)
W8 = "M N K A lda rs B ldb trans cs C ldc type epi stream".split()
W8_OK = dict(M=4, N=16, K=32, A=P, lda=32, rs=P, B=P, ldb=16, trans=0, cs=P, C=P, ldc=16, type=0, epi=0, stream=None)
GRP = "M N K E A lda off B ldb plane trans C ldc epi stream".split()
GRP_OK = dict(M=4, N=16, K=32, E=3, A=P, lda=32, off=P, B=P, ldb=16, plane=512, trans=0, C=P, ldc=16, epi=0, stream=None)
WG = "M N K E A lda G ldg off C ldc plane stream".split()
WG_OK = dict(M=4, N=16, K=32, E=3, A=P, lda=32, G=P, ldg=16, off=P, C=P, ldc=16, plane=512, stream=None)
G8 = "M N K E A lda rs off B ldb plane trans cs planes C ldc type epi stream".split()
G8_OK = dict(M=4, N=16, K=32, E=3, A=P, lda=32, rs=P, off=P, B=P, ldb=16, plane=512, trans=0, cs=P, planes=16, C=P,
             ldc=16, type=1, epi=0, stream=None)
SORT = "T k E ids idb off pos src scratch stream".split()
SORT_OK = dict(T=4, k=2, E=3, ids=P, idb=8, off=P, pos=P, src=P, scratch=None, stream=None)
GATHER = "T k H eb X ldx sc pos kept out ldo osc stream".split()
GATHER_OK = dict(T=4, k=2, H=16, eb=2, X=P, ldx=16, sc=None, pos=P, kept=P, out=P, ldo=16, osc=None, stream=None)
COMB = "T k H type Y ldy pos kept w out ldo stream".split()
COMB_OK = dict(T=4, k=2, H=16, type=1, Y=P, ldy=16, pos=P, kept=P, w=P, out=P, ldo=16, stream=None)
CGRAD = "T k H type Y ldy d ldd pos kept w dY lddy dw stream".split()
CGRAD_OK = dict(T=4, k=2, H=16, type=1, Y=P, ldy=16, d=P, ldd=16, pos=P, kept=P, w=P, dY=P, lddy=16, dw=P, stream=None)

REFUSED = [
    # name, argument list, good values, {changes: status}
    ("tg_quant_i8", QUANT, QUANT_OK, [
        (dict(M=-1), INVALID), (dict(K=-1), INVALID), (dict(type=2), INVALID), (dict(X=None), INVALID),
        (dict(Q=None), INVALID), (dict(scales=None), INVALID), (dict(ldx=8), INVALID), (dict(ldq=8), INVALID),
        (dict(X=P + 2), ALIGN), (dict(Q=P + 4), ALIGN), (dict(ldx=20), ALIGN), (dict(ldq=24), ALIGN),
        (dict(scales=P + 2), ALIGN), (dict(M=BIG), UNSUP), (dict(ldx=1 << 40), UNSUP), (dict(M=0, X=None), OK)]),
    ("tg_gemm_w8a8", W8, W8_OK, [
        (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=-1), INVALID), (dict(type=-1), INVALID),
        (dict(epi=2), INVALID), (dict(trans=2), INVALID), (dict(A=None), INVALID), (dict(B=None), INVALID),
        (dict(C=None), INVALID), (dict(rs=None), INVALID), (dict(cs=None), INVALID), (dict(lda=16), INVALID),
        (dict(ldb=0), INVALID), (dict(trans=1, ldb=16), INVALID), (dict(ldc=8), INVALID), (dict(A=P + 8), ALIGN),
        (dict(lda=40), ALIGN), (dict(ldc=20), ALIGN), (dict(rs=P + 1), ALIGN), (dict(K=131072, lda=131072), UNSUP),
        (dict(M=BIG), UNSUP), (dict(M=BIG - 1024), UNSUP), (dict(ldb=1 << 40), UNSUP), (dict(M=0), OK),
        (dict(N=0), OK)]),
    ("tg_gemm_grouped_bf16", GRP, GRP_OK, [
        (dict(M=-1), INVALID), (dict(E=0), INVALID), (dict(E=1025), UNSUP), (dict(off=None), INVALID),
        (dict(off=P + 2), ALIGN), (dict(plane=0), INVALID), (dict(plane=-8), INVALID), (dict(plane=516), ALIGN),
        (dict(plane=1 << 39), UNSUP), (dict(B=P + 2), ALIGN), (dict(ldb=20), ALIGN), (dict(trans=-1), INVALID),
        (dict(epi=7), INVALID), (dict(C=None), INVALID), (dict(M=0, off=None), OK), (dict(N=0), OK)]),
    ("tg_gemm_grouped_wgrad_f16", WG, WG_OK, [
        (dict(K=-1), INVALID), (dict(E=0), INVALID), (dict(E=2000), UNSUP), (dict(G=None), INVALID),
        (dict(A=None), INVALID), (dict(off=None), INVALID), (dict(C=None), INVALID), (dict(plane=504), INVALID),
        (dict(plane=516), ALIGN), (dict(ldg=8), INVALID), (dict(ldg=20), ALIGN), (dict(C=P + 8), ALIGN),
        (dict(K=BIG - 1, lda=BIG, ldc=1 << 38, plane=1 << 38), INVALID), (dict(K=0), OK), (dict(N=0), OK)]),
    ("tg_gemm_grouped_w8a8", G8, G8_OK, [
        (dict(E=0), INVALID), (dict(rs=None), INVALID), (dict(cs=None), INVALID), (dict(planes=-1), INVALID),
        (dict(type=5), INVALID), (dict(plane=520), ALIGN), (dict(plane=0), INVALID), (dict(lda=40), ALIGN),
        (dict(K=131072, lda=131072), UNSUP), (dict(off=None), INVALID), (dict(M=0), OK)]),
    ("tg_expert_sort", SORT, SORT_OK, [
        (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(E=0), INVALID), (dict(E=1025), UNSUP),
        (dict(idb=2), INVALID), (dict(ids=None), INVALID), (dict(ids=P + 4), ALIGN), (dict(off=None), INVALID),
        (dict(pos=P + 1), ALIGN), (dict(src=None), INVALID), (dict(T=BIG), UNSUP), (dict(T=1 << 30, k=2), UNSUP),
        (dict(T=10000), INVALID)]),                       # a size that needs scratch
    ("tg_expert_gather", GATHER, GATHER_OK, [
        (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(H=-1), INVALID), (dict(eb=4), INVALID),
        (dict(sc=P), INVALID), (dict(osc=P), INVALID), (dict(X=None), INVALID), (dict(ldx=8), INVALID),
        (dict(ldx=20), ALIGN), (dict(eb=1, ldx=24), ALIGN), (dict(pos=None), INVALID), (dict(kept=None), INVALID),
        (dict(out=P + 2), ALIGN), (dict(T=1 << 30, k=2), UNSUP), (dict(T=0), OK), (dict(H=0), OK)]),
    ("tg_expert_combine", COMB, COMB_OK, [
        (dict(type=3), INVALID), (dict(Y=None), INVALID), (dict(w=P + 2), ALIGN), (dict(ldo=8), INVALID),
        (dict(out=P + 8), ALIGN), (dict(kept=P + 2), ALIGN), (dict(T=0), OK), (dict(H=0), OK)]),
    ("tg_expert_combine_grad", CGRAD, CGRAD_OK, [
        (dict(w=None), INVALID), (dict(dw=None), INVALID), (dict(dY=None), INVALID), (dict(ldd=8), INVALID),
        (dict(d=P + 2), ALIGN), (dict(H=-1), INVALID), (dict(k=-1), INVALID), (dict(T=0), OK)]),
]


@pytest.mark.parametrize("name,names,good,cases", REFUSED, ids=[r[0] for r in REFUSED])
def test_refusals(lib, name, names, good, cases):
    for change, want in cases:
        assert call(getattr(lib, name), names, good, **change) == want, change


def test_scratch_sizes(lib):
    assert lib.tg_expert_sort_scratch(100, 8) == 0
    assert lib.tg_expert_sort_scratch(100000, 8) % (9 * 4) == 0 and lib.tg_expert_sort_scratch(100000, 8) > 0
    for n, e in ((-1, 8), (BIG, 8), (10, 0), (10, 1025)):
        assert lib.tg_expert_sort_scratch(n, e) == -1


# -------------------------------------------------------------- marshalling

def mat(p, rows, cols, ld, dtype):
    """rows x cols numpy view of host memory at p with row pitch ld."""
    if rows == 0 or cols == 0:
        return np.zeros((rows, cols), dtype)
    ct = {np.int8: ctypes.c_int8, np.uint16: ctypes.c_uint16, np.int32: ctypes.c_int32,
          np.float32: ctypes.c_float}[dtype]
    n = (rows - 1) * ld + cols
    flat = np.ctypeslib.as_array((ct * n).from_address(p))
    return np.lib.stride_tricks.as_strided(flat, (rows, cols), (ld * flat.itemsize, flat.itemsize))


def value(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def bits(v):
    return torch.from_numpy(np.ascontiguousarray(v, np.float32)).bfloat16().view(torch.int16).numpy().view(np.uint16)


class Fake:
    """bfloat16 stand-ins of the entry points, on host memory."""

    def tg_gemm_grouped_bf16(self, M, N, K, E, A, lda, off, B, ldb, plane, trans, C, ldc, epi, stream):
        o = mat(off, 1, E + 1, E + 1, np.int32)[0]
        a, c = value(mat(A, M, K, lda, np.uint16)), mat(C, M, N, ldc, np.uint16)
        c[:] = 0
        for e in range(E):
            w = value(mat(B + 2 * e * plane, *((N, K) if trans else (K, N)), ldb, np.uint16))
            y = a[o[e]:o[e + 1]] @ (w.T if trans else w)
            c[o[e]:o[e + 1]] = bits(np.maximum(y, 0) if epi else y)
        return 0

    def tg_gemm_grouped_wgrad_bf16(self, M, N, K, E, A, lda, G, ldg, off, C, ldc, plane, stream):
        o = mat(off, 1, E + 1, E + 1, np.int32)[0]
        a, g = value(mat(A, M, K, lda, np.uint16)), value(mat(G, M, N, ldg, np.uint16))
        for e in range(E):
            mat(C + 2 * e * plane, K, N, ldc, np.uint16)[:] = bits(a[o[e]:o[e + 1]].T @ g[o[e]:o[e + 1]])
        return 0

    def tg_gemm_w8a8(self, M, N, K, A, lda, rs, B, ldb, trans, cs, C, ldc, type, epi, stream):
        w = mat(B, *((N, K) if trans else (K, N)), ldb, np.int8).astype(np.float64)
        y = mat(A, M, K, lda, np.int8).astype(np.float64) @ (w.T if trans else w)
        y = y * mat(rs, 1, M, M, np.float32).T * mat(cs, 1, N, N, np.float32)
        assert type == 1
        mat(C, M, N, ldc, np.uint16)[:] = bits(np.maximum(y, 0) if epi else y)
        return 0

    def tg_expert_gather(self, T, k, H, eb, X, ldx, sc, pos, kept, out, ldo, osc, stream):
        dt = np.int8 if eb == 1 else np.uint16
        p, n = mat(pos, T, k, k, np.int32), mat(kept, 1, 1, 1, np.int32)[0, 0]
        x, o = mat(X, T, H, ldx, dt), mat(out, T * k, H, ldo, dt)
        for t in range(T):
            for j in range(k):
                o[p[t, j]] = x[t] if p[t, j] < n else 0
                if sc:
                    mat(osc, 1, T * k, T * k, np.float32)[0, p[t, j]] = \
                        mat(sc, 1, T, T, np.float32)[0, t] if p[t, j] < n else 0
        return 0

    def tg_expert_combine(self, T, k, H, type, Y, ldy, pos, kept, w, out, ldo, stream):
        p, n = mat(pos, T, k, k, np.int32), mat(kept, 1, 1, 1, np.int32)[0, 0]
        y, o = value(mat(Y, T * k, H, ldy, np.uint16)), mat(out, T, H, ldo, np.uint16)
        wt = mat(w, T, k, k, np.float32) if w else np.ones((T, k))
        for t in range(T):
            o[t] = bits(sum((wt[t, j] * y[p[t, j]] for j in range(k) if p[t, j] < n), np.zeros(H)))
        return 0

    def tg_expert_combine_grad(self, T, k, H, type, Y, ldy, d, ldd, pos, kept, w, dY, lddy, dw, stream):
        p, n = mat(pos, T, k, k, np.int32), mat(kept, 1, 1, 1, np.int32)[0, 0]
        y, g = value(mat(Y, T * k, H, ldy, np.uint16)), value(mat(d, T, H, ldd, np.uint16))
        wt, o, od = mat(w, T, k, k, np.float32), mat(dY, T * k, H, lddy, np.uint16), mat(dw, T, k, k, np.float32)
        for t in range(T):
            for j in range(k):
                r, on = p[t, j], p[t, j] < n
                o[r] = bits(wt[t, j] * g[t]) if on else 0
                od[t, j] = y[r] @ g[t] if on else 0
        return 0


@pytest.fixture
def fake(monkeypatch):
    lib = Fake()
    monkeypatch.setattr(binding, "_launch",
                        lambda name, device, stream, *args: getattr(lib, name)(*args, stream))
    monkeypatch.setattr(binding, "_require_cuda", lambda device, *named: None)
    return lib


def bf(shape, seed, pitch=None):
    g = torch.Generator().manual_seed(seed)
    out = torch.zeros(*shape[:-1], pitch or shape[-1], dtype=torch.bfloat16)[..., :shape[-1]]
    out.copy_(torch.randn(shape, generator=g))
    return out


def plan_of(ids, E):
    flat = torch.where((ids >= 0) & (ids < E), ids, E).reshape(-1)
    src = torch.argsort(flat, stable=True)
    pos = torch.empty_like(src)
    pos[src] = torch.arange(len(src))
    offsets = torch.zeros(E + 1, dtype=torch.int32)
    offsets[1:] = torch.bincount(flat, minlength=E + 1)[:E].cumsum(0)
    return binding.ExpertPlan(offsets, pos.to(torch.int32).view(ids.shape), src.to(torch.int32))


IDS = torch.tensor([[0, 2], [1, -1], [2, 0], [7, 2], [0, 1]])


def near(a, b, steps=4):
    """Within `steps` bf16 roundings of the largest value."""
    assert a.shape == b.shape
    assert (a.double() - b.double()).abs().max() <= steps * 2.0 ** -8 * b.abs().max() + 1e-30


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("odd", [False, True])
def test_product_and_its_gradients(fake, trans, odd):
    K, N, E = (13, 11, 3) if odd else (16, 24, 3)
    pk, pn = -(-K // 8) * 8 + 8, -(-N // 8) * 8 + 8
    X = bf((10, K), 1, pk).requires_grad_(True)
    S = (bf((E, N, K), 2, pk) if trans else bf((E, K, N), 2, pn)).requires_grad_(True)
    W = S.transpose(1, 2) if trans else S
    plan = plan_of(IDS, E)
    Y = binding.expert_matmul(X, W, plan)
    g = bf((10, N), 3)                                # odd N: a pitch the kernels do not take
    dX, dS = torch.autograd.grad(Y, (X, S), g)
    o = plan.offsets.tolist()
    x, w = X.detach().double().requires_grad_(True), S.detach().double().requires_grad_(True)
    rows = [x[o[e]:o[e + 1]] @ (w[e].t() if trans else w[e]) for e in range(E)]
    ref = torch.cat(rows + [torch.zeros(10 - o[E], N, dtype=torch.float64)])
    rX, rS = torch.autograd.grad(ref, (x, w), g.double())
    near(Y.detach(), ref.detach(), 1)
    near(dX, rX, 1)
    near(dS, rS, 1)
    assert torch.equal(binding.expert_matmul(X.detach(), W.detach(), plan.offsets), Y.detach())


def test_gather_and_combine(fake):
    plan = plan_of(IDS, 3)
    n = int(plan.offsets[-1])
    X = bf((5, 9), 1, 16).requires_grad_(True)
    Xs = binding.expert_gather(X, plan)
    tok = (plan.src // 2).long()
    assert torch.equal(Xs.detach()[:n], X.detach()[tok[:n]]) and not Xs.detach()[n:].any()
    dX, = torch.autograd.grad(Xs.sum(), X)            # an expanded gradient
    near(dX, ((IDS >= 0) & (IDS < 3)).sum(1, keepdim=True).expand(5, 9).double(), 1)
    Y = bf((10, 9), 2, 16).requires_grad_(True)
    w = torch.rand(5, 2, generator=torch.Generator().manual_seed(3)).requires_grad_(True)
    g = bf((5, 9), 4)
    for weights in (w, None):
        out = binding.expert_combine(Y, plan, weights)
        leaves = (Y, w) if weights is not None else (Y,)
        got = torch.autograd.grad(out, leaves, g)
        y, ww = Y.detach().double().requires_grad_(True), w.detach().double().requires_grad_(True)
        kept = ((IDS >= 0) & (IDS < 3)).double()
        ref = ((kept * (ww if weights is not None else 1))[:, :, None] * y[plan.pos.long()]).sum(1)
        want = torch.autograd.grad(ref, (y, ww) if weights is not None else (y,), g.double())
        near(out.detach(), ref.detach(), 1)
        for a, b in zip(got, want):
            near(a, b, 1)


def test_only_the_gradients_asked_for(fake):
    plan = plan_of(IDS, 3)
    X, W = bf((10, 16), 1), bf((3, 16, 8), 2)
    for gx, gw in ((True, False), (False, True)):
        x, w = X.clone().requires_grad_(gx), W.clone().requires_grad_(gw)
        binding.expert_matmul(x, w, plan).sum().backward()
        assert (x.grad is not None) == gx and (w.grad is not None) == gw
    Y, wt = bf((10, 8), 3), torch.rand(5, 2)
    y = Y.clone().requires_grad_(True)
    binding.expert_combine(y, plan, wt).sum().backward()
    assert y.grad is not None


def test_differentiable_once(fake):
    plan = plan_of(IDS, 3)
    X = bf((5, 8), 1).requires_grad_(True)
    Xs = binding.expert_gather(X, plan)
    with pytest.raises(RuntimeError, match="once"):
        torch.autograd.grad(Xs.sum(), X, create_graph=True)


def test_changed_plans_and_weights_are_noticed(fake):
    plan = plan_of(IDS, 3)
    X, W = bf((10, 16), 1).requires_grad_(True), bf((3, 16, 8), 2)
    offsets = plan.offsets.clone()
    Y = binding.expert_matmul(X, W, offsets)
    offsets.add_(0)
    with pytest.raises(RuntimeError, match="in-?place"):
        Y.sum().backward()
    Z = binding.expert_gather(bf((5, 8), 1).requires_grad_(True), plan)
    plan.pos.add_(0)
    with pytest.raises(RuntimeError, match="in-?place"):
        Z.sum().backward()


def test_dense_product8(fake):
    g = torch.Generator().manual_seed(1)
    A = torch.randint(-128, 128, (3, 20), generator=g, dtype=torch.int8)
    W = torch.randint(-128, 128, (20, 7), generator=g, dtype=torch.int8)
    rs, cs = torch.rand(3, generator=g), torch.rand(7, generator=g)
    ref = (A.double() @ W.double()) * rs.double()[:, None] * cs.double()
    Ap = torch.zeros(3, 32, dtype=torch.int8)[:, :20]
    Ap.copy_(A)
    for trans in (False, True):
        src = W.t() if trans else W
        Wp = torch.zeros(src.shape[0], 32, dtype=torch.int8)[:, :src.shape[1]]
        Wp.copy_(src)
        near(binding.gemm_w8a8(Ap, rs, Wp, cs, trans_b=trans), ref, 1)
        near(binding.gemm_w8a8(Ap, rs, Wp, cs, trans_b=trans, relu=True), ref.clamp(min=0), 1)


def test_how_weights_reach_the_kernels():
    S = torch.empty(4, 24, 40, dtype=torch.bfloat16)
    st, tr = binding._stored3(S)
    assert not tr and st is S
    st, tr = binding._stored3(S.transpose(1, 2))
    assert tr and st.data_ptr() == S.data_ptr() and tuple(st.shape) == (4, 24, 40)
    st, tr = binding._stored3(S[:, :, 8:24])              # a column slice keeps its pitch
    assert not tr and st.stride(1) == 40
    x = bf((4, 24, 40), 1)[:, ::2, ::2]
    st, tr = binding._stored3(x)
    assert not tr and torch.equal(st, x) and st.stride() == (12 * 24, 24, 1)      # 20 columns, 16-byte pitch
    one = torch.empty(1, 24, 40, dtype=torch.bfloat16).expand(4, 24, 40)
    st, tr = binding._stored3(one)                        # shared weights are copied
    assert not tr and st.stride(0) == 24 * 40


def test_python_refusals(fake):
    plan = plan_of(IDS, 3)
    X, W = bf((10, 16), 1), bf((3, 16, 8), 2)
    q, s = torch.zeros(4, 16, dtype=torch.int8), torch.ones(4)
    bad = [
        (ValueError, lambda: binding.gemm_grouped(X, plan, W[:2])),
        (ValueError, lambda: binding.gemm_grouped(X[:, :8], plan, W)),
        (TypeError, lambda: binding.gemm_grouped(X, plan, W.half())),
        (TypeError, lambda: binding.gemm_grouped(X.float(), plan, W.float())),
        (TypeError, lambda: binding.gemm_grouped(X, plan.offsets.long(), W)),
        (ValueError, lambda: binding.gemm_grouped(X, plan.offsets[:1], W)),
        (ValueError, lambda: binding.gemm_grouped(X, plan, W, C=bf((10, 9), 1))),
        (ValueError, lambda: binding.gemm_grouped(X.t().contiguous().t(), plan, W)),
        (ValueError, lambda: binding.gemm_grouped_wgrad(X, X[:5], plan)),
        (ValueError, lambda: binding.expert_gather(X, plan)),
        (TypeError, lambda: binding.expert_gather(X[:5].float(), plan)),
        (TypeError, lambda: binding.expert_gather(X[:5], plan, scales=torch.ones(5))),
        (ValueError, lambda: binding.expert_combine(X[:5], plan)),
        (TypeError, lambda: binding.expert_combine(X, plan, torch.ones(5, 2, dtype=torch.bfloat16))),
        (ValueError, lambda: binding.expert_combine(X, plan, torch.ones(2, 5))),
        (ValueError, lambda: binding.expert_matmul(X, W[0], plan)),
        (ValueError, lambda: binding.expert_sort(torch.zeros(4, dtype=torch.int64), 3)),
        (TypeError, lambda: binding.expert_sort(torch.zeros(4, 2), 3)),
        (ValueError, lambda: binding.expert_sort(torch.zeros(4, 2, dtype=torch.int64), 1025)),
        (TypeError, lambda: binding.ExpertPlan(plan.offsets.long(), plan.pos)),
        (ValueError, lambda: binding.ExpertPlan(plan.offsets, plan.pos.t())),
        (TypeError, lambda: binding.quant_i8(X.float())),
        (ValueError, lambda: binding.quant_i8(X[0])),
        (TypeError, lambda: binding.gemm_w8a8(X, s, q.t(), s)),
        (ValueError, lambda: binding.gemm_w8a8(q, s[:3], torch.zeros(16, 16, dtype=torch.int8), torch.ones(16))),
        (TypeError, lambda: binding.gemm_w8a8(q, s, torch.zeros(16, 16, dtype=torch.int8), torch.ones(16),
                                              out_dtype=torch.float32)),
        (ValueError, lambda: binding.gemm_w8a8(q, s, torch.zeros(8, 16, dtype=torch.int8), torch.ones(16))),
    ]
    for i, (kind, f) in enumerate(bad):
        with pytest.raises(kind):
            f()
            pytest.fail(f"case {i} was not refused")


def test_cpu_tensors_are_refused():
    """There is no fallback: tensors must be on a GPU."""
    for f in (lambda: binding.quant_i8(bf((4, 16), 1)),
              lambda: binding.expert_sort(torch.zeros(4, 2, dtype=torch.int64), 3),
              lambda: binding.gemm_grouped(bf((4, 16), 1), torch.tensor([0, 4], dtype=torch.int32), bf((1, 16, 8), 2))):
        with pytest.raises(ValueError, match="CUDA"):
            f()


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("N", [8, 11])
def test_saved_tensors_in_another_layout(fake, trans, N):
    """A saved-tensor hook (offloading) may give back contiguous copies of what
    were strided views; shared weights were copied in forward."""
    K, E = 13, 3
    plan = plan_of(IDS, E)
    X = bf((10, K), 1, 24).requires_grad_(True)
    S = (bf((E, N, K), 2, 24) if trans else bf((E, K, N), 2, 24)).requires_grad_(True)
    g = bf((10, N), 3, 16)

    def grads(x, s):
        y = binding.expert_matmul(x, s.transpose(1, 2) if trans else s, plan)
        return torch.autograd.grad(y, (X, S), g)

    want = grads(X, S)
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t.clone(memory_format=torch.contiguous_format), lambda t: t):
        got = grads(X, S)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    one = bf((K, N), 4, 24).requires_grad_(True)
    y = binding.expert_matmul(X.detach(), one.expand(E, K, N), plan)
    d, = torch.autograd.grad(y, one, g)
    n = int(plan.offsets[-1])
    # the groups' gradients are rounded before autograd adds them, in bfloat16
    near(d, X.detach().double()[:n].t() @ g.double()[:n], 2 * E)
    Y = bf((10, N), 5, 16).requires_grad_(True)
    w = torch.rand(5, 2).requires_grad_(True)
    want = torch.autograd.grad(binding.expert_combine(Y, plan, w), (Y, w), bf((5, N), 6, 16))
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t.clone(memory_format=torch.contiguous_format), lambda t: t):
        got = torch.autograd.grad(binding.expert_combine(Y, plan, w), (Y, w), bf((5, N), 6, 16))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
