"""Host checks of routing and of the microscaled 4-bit operators (no GPU): the
entry points' refusals, which come before any CUDA call, the binding's own, and
its marshalling, checked with a fake library that reads its operands through the
pointers, pitches and planes it is given and computes in float64."""
import ctypes
import math

import numpy as np
import pytest
import torch

from mxfp4_util import quantised, values
from route_util import choose, weights_of
from tiled_dense_gemm_tma_b200 import binding, build as tg_build

OK, INVALID, ALIGN, UNSUP = 0, 1, 2, 3
P = 0x10000          # a fake, 16-byte aligned "device" address (never dereferenced)
BIG = 1 << 31


@pytest.fixture(scope="module")
def lib():
    tg_build.build()
    return binding.load_library()


QUANT = "M K X ldx type Q ldq S lds stream".split()
QUANT_OK = dict(M=4, K=64, X=P, ldx=64, type=1, Q=P, ldq=32, S=P, lds=16, stream=None)
BACK = "M K Q ldq S lds Y ldy type stream".split()
BACK_OK = dict(M=4, K=64, Q=P, ldq=32, S=P, lds=16, Y=P, ldy=64, type=0, stream=None)
PLACE = "T k K X ldx type pos kept Q ldq S lds stream".split()
PLACE_OK = dict(T=4, k=2, K=64, X=P, ldx=64, type=1, pos=P, kept=P, Q=P, ldq=32, S=P, lds=16, stream=None)
MUL = "M N K A lda SA ldsa B ldb SB ldsb C ldc type epi stream".split()
MUL_OK = dict(M=4, N=24, K=64, A=P, lda=32, SA=P, ldsa=16, B=P, ldb=32, SB=P, ldsb=16, C=P, ldc=24, type=1, epi=0,
              stream=None)
GRP = "M N K E A lda SA ldsa off B ldb pb SB ldsb ps C ldc type epi stream".split()
GRP_OK = dict(M=4, N=24, K=64, E=3, A=P, lda=32, SA=P, ldsa=16, off=P, B=P, ldb=32, pb=768, SB=P, ldsb=16, ps=384, C=P,
              ldc=24, type=0, epi=1, stream=None)
ROUTE = "T E X ldl type bias score groups keep k renorm scale ids w stream".split()
ROUTE_OK = dict(T=4, E=8, X=P, ldl=8, type=2, bias=None, score=0, groups=1, keep=1, k=2, renorm=1, scale=1.0, ids=P,
                w=P, stream=None)
RGRAD = "T E X ldl type score k renorm scale ids dw d ldd stream".split()
RGRAD_OK = dict(T=4, E=8, X=P, ldl=8, type=2, score=0, k=2, renorm=1, scale=1.0, ids=P, dw=P, d=P, ldd=8, stream=None)

REFUSED = [
    ("tg_quant_mxfp4", QUANT, QUANT_OK, [
        (dict(M=-1), INVALID), (dict(K=-1), INVALID), (dict(type=2), INVALID), (dict(X=None), INVALID),
        (dict(Q=None), INVALID), (dict(S=None), INVALID), (dict(ldx=56), INVALID), (dict(ldq=16), INVALID),
        (dict(lds=1), INVALID), (dict(X=P + 2), ALIGN), (dict(Q=P + 8), ALIGN), (dict(S=P + 1), ALIGN),
        (dict(ldx=68), ALIGN), (dict(ldq=40), ALIGN), (dict(lds=4), ALIGN), (dict(M=BIG), UNSUP),
        (dict(ldx=1 << 40), UNSUP), (dict(K=65), INVALID), (dict(M=0, X=None), OK), (dict(K=0, Q=None), OK)]),
    ("tg_dequant_mxfp4", BACK, BACK_OK, [
        (dict(M=-1), INVALID), (dict(K=-1), INVALID), (dict(type=7), INVALID), (dict(Y=None), INVALID),
        (dict(Q=None), INVALID), (dict(S=None), INVALID), (dict(ldy=56), INVALID), (dict(ldy=68), ALIGN),
        (dict(Y=P + 8), ALIGN), (dict(ldq=24), INVALID), (dict(M=BIG), UNSUP), (dict(M=0), OK), (dict(K=0), OK)]),
    ("tg_expert_quant_mxfp4", PLACE, PLACE_OK, [
        (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(K=-1), INVALID), (dict(type=2), INVALID),
        (dict(pos=None), INVALID), (dict(kept=None), INVALID), (dict(pos=P + 2), ALIGN), (dict(kept=P + 1), ALIGN),
        (dict(X=None), INVALID), (dict(Q=P + 4), ALIGN), (dict(lds=8), ALIGN), (dict(T=1 << 30, k=2), UNSUP),
        (dict(T=0), OK), (dict(K=0), OK)]),
    ("tg_gemm_mxfp4", MUL, MUL_OK, [
        (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=-1), INVALID), (dict(type=2), INVALID),
        (dict(epi=2), INVALID), (dict(A=None), INVALID), (dict(SA=None), INVALID), (dict(B=None), INVALID),
        (dict(SB=None), INVALID), (dict(C=None), INVALID), (dict(lda=16), INVALID), (dict(ldb=16), INVALID),
        (dict(ldsa=1), INVALID), (dict(ldsb=0), INVALID), (dict(ldc=16), INVALID), (dict(lda=40), ALIGN),
        (dict(ldsb=24), ALIGN), (dict(ldc=28), ALIGN), (dict(A=P + 8), ALIGN), (dict(SB=P + 4), ALIGN),
        (dict(C=P + 2), ALIGN), (dict(M=BIG - 1024), UNSUP), (dict(N=BIG, ldc=BIG), UNSUP),
        (dict(ldb=1 << 40), UNSUP), (dict(M=0, A=None), OK), (dict(N=0), OK)]),
    ("tg_gemm_grouped_mxfp4", GRP, GRP_OK, [
        (dict(M=-1), INVALID), (dict(E=0), INVALID), (dict(E=1025), UNSUP), (dict(off=None), INVALID),
        (dict(off=P + 2), ALIGN), (dict(pb=0), INVALID), (dict(ps=-16), INVALID), (dict(pb=776), ALIGN),
        (dict(ps=392), ALIGN), (dict(pb=1 << 40), UNSUP), (dict(SA=None), INVALID), (dict(epi=3), INVALID),
        (dict(type=2), INVALID), (dict(M=0, off=None), OK), (dict(N=0), OK)]),
    ("tg_expert_route", ROUTE, ROUTE_OK, [
        (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(k=9), INVALID), (dict(type=3), INVALID),
        (dict(score=2), INVALID), (dict(renorm=2), INVALID), (dict(groups=0), INVALID), (dict(groups=3), INVALID),
        (dict(groups=16), INVALID), (dict(groups=4, keep=5), INVALID), (dict(keep=0), INVALID),
        (dict(groups=4, keep=1, k=3), INVALID), (dict(X=None), INVALID), (dict(ids=None), INVALID),
        (dict(w=None), INVALID), (dict(ldl=7), INVALID), (dict(X=P + 2), ALIGN), (dict(type=1, X=P + 1), ALIGN),
        (dict(bias=P + 2), ALIGN), (dict(ids=P + 2), ALIGN), (dict(E=1025, ldl=1025), UNSUP),
        (dict(E=64, ldl=64, k=33), UNSUP), (dict(E=66, ldl=66, groups=33, keep=33), UNSUP), (dict(T=BIG), UNSUP),
        (dict(ldl=1 << 40), UNSUP), (dict(T=0, X=None, ids=None, w=None), OK), (dict(T=0, k=0), INVALID)]),
    ("tg_expert_route_grad", RGRAD, RGRAD_OK, [
        (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(k=9), INVALID), (dict(type=-1), INVALID),
        (dict(score=-1), INVALID), (dict(dw=None), INVALID), (dict(d=None), INVALID), (dict(ldd=7), INVALID),
        (dict(d=P + 2), ALIGN), (dict(dw=P + 2), ALIGN), (dict(E=2000, ldl=2000, ldd=2000), UNSUP),
        (dict(E=64, ldl=64, ldd=64, k=40), UNSUP), (dict(T=0, X=None, ids=None, dw=None, d=None), OK)]),
]


@pytest.mark.parametrize("name,names,good,cases", REFUSED, ids=[r[0] for r in REFUSED])
def test_refusals(lib, name, names, good, cases):
    for change, want in cases:
        a = dict(good, **change)
        assert set(change) <= set(names)
        assert getattr(lib, name)(*[a[n] for n in names]) == want, change


# -------------------------------------------------------------- marshalling

def mat(p, rows, cols, ld, dtype):
    """rows x cols numpy view of host memory at p with row pitch ld."""
    if rows == 0 or cols == 0:
        return np.zeros((rows, cols), dtype)
    ct = {np.uint8: ctypes.c_uint8, np.uint16: ctypes.c_uint16, np.int32: ctypes.c_int32,
          np.float32: ctypes.c_float}[dtype]
    n = (rows - 1) * ld + cols
    flat = np.ctypeslib.as_array((ct * n).from_address(p))
    return np.lib.stride_tricks.as_strided(flat, (rows, cols), (ld * flat.itemsize, flat.itemsize))


def value(bits):
    return torch.from_numpy((bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64))


def bits(v):
    return v.float().bfloat16().view(torch.int16).numpy().view(np.uint16)


def held(q, ldq, s, lds, rows, K):
    return values(torch.from_numpy(mat(q, rows, -(-K // 2), ldq, np.uint8).copy()),
                  torch.from_numpy(mat(s, rows, -(-K // 32), lds, np.uint8).copy()), K)


class Fake:
    """bfloat16 (logits: float32) stand-ins of the entry points, on host memory."""

    def tg_quant_mxfp4(self, M, K, X, ldx, type, Q, ldq, S, lds, stream):
        assert type == 1
        q, s = quantised(value(mat(X, M, K, ldx, np.uint16)))
        mat(Q, M, -(-K // 2), ldq, np.uint8)[:] = q.numpy()
        mat(S, M, -(-K // 32), lds, np.uint8)[:] = s.numpy()
        return 0

    def tg_expert_quant_mxfp4(self, T, k, K, X, ldx, type, pos, kept, Q, ldq, S, lds, stream):
        q, s = quantised(value(mat(X, T, K, ldx, np.uint16)))
        p, n = mat(pos, T, k, k, np.int32), mat(kept, 1, 1, 1, np.int32)[0, 0]
        oq, os = mat(Q, T * k, -(-K // 2), ldq, np.uint8), mat(S, T * k, -(-K // 32), lds, np.uint8)
        for t in range(T):
            for j in range(k):
                oq[p[t, j]] = q[t] if p[t, j] < n else 0
                os[p[t, j]] = s[t] if p[t, j] < n else 0
        return 0

    def tg_dequant_mxfp4(self, M, K, Q, ldq, S, lds, Y, ldy, type, stream):
        mat(Y, M, K, ldy, np.uint16)[:] = bits(held(Q, ldq, S, lds, M, K))
        return 0

    def tg_gemm_mxfp4(self, M, N, K, A, lda, SA, ldsa, B, ldb, SB, ldsb, C, ldc, type, epi, stream):
        y = held(A, lda, SA, ldsa, M, K) @ held(B, ldb, SB, ldsb, N, K).t()
        mat(C, M, N, ldc, np.uint16)[:] = bits(y.clamp(min=0) if epi else y)
        return 0

    def tg_gemm_grouped_mxfp4(self, M, N, K, E, A, lda, SA, ldsa, off, B, ldb, pb, SB, ldsb, ps, C, ldc, type, epi, stream):
        o, c = mat(off, 1, E + 1, E + 1, np.int32)[0], mat(C, M, N, ldc, np.uint16)
        a = held(A, lda, SA, ldsa, M, K)
        c[:] = 0
        for e in range(E):
            y = a[o[e]:o[e + 1]] @ held(B + e * pb, ldb, SB + e * ps, ldsb, N, K).t()
            c[o[e]:o[e + 1]] = bits(y.clamp(min=0) if epi else y)
        return 0

    def tg_expert_route(self, T, E, X, ldl, type, bias, score, groups, keep, k, renorm, scale, ids, w, stream):
        assert type == 2
        x = torch.from_numpy(mat(X, T, E, ldl, np.float32).astype(np.float64))
        b = mat(bias, 1, E, E, np.float32)[0].tolist() if bias else None
        kind = ("softmax", "sigmoid")[score]
        i = torch.tensor([choose(r, k, kind, b, groups, keep) for r in x.tolist()]).view(T, k)
        mat(ids, T, k, k, np.int32)[:] = i.numpy()
        mat(w, T, k, k, np.float32)[:] = weights_of(x, i, kind, renorm, scale).numpy()
        return 0

    def tg_expert_route_grad(self, T, E, X, ldl, type, score, k, renorm, scale, ids, dw, d, ldd, stream):
        x = torch.from_numpy(mat(X, T, E, ldl, np.float32).astype(np.float64)).requires_grad_(True)
        i = torch.from_numpy(mat(ids, T, k, k, np.int32).copy())
        with torch.enable_grad():
            w = weights_of(x, i, ("softmax", "sigmoid")[score], renorm, scale)
            g, = torch.autograd.grad(w, x, torch.from_numpy(mat(dw, T, k, k, np.float32).astype(np.float64)))
        mat(d, T, E, ldd, np.float32)[:] = g.numpy()
        return 0


@pytest.fixture
def fake(monkeypatch):
    lib = Fake()
    monkeypatch.setattr(binding, "_launch",
                        lambda name, device, stream, *args: getattr(lib, name)(*args, stream))
    monkeypatch.setattr(binding, "_require_cuda", lambda device, *named: None)
    return lib


def rows(M, K, seed, pitch=None):
    out = torch.zeros(M, pitch or K, dtype=torch.bfloat16)[:, :K]
    out.copy_(torch.randn((M, K), generator=torch.Generator().manual_seed(seed)))
    return out


def close(got, ref):
    """One bfloat16 rounding of the 64-bit result."""
    assert torch.equal(got, ref.float().bfloat16())


@pytest.mark.parametrize("K,pitch", [(64, 64), (70, 80), (33, 40), (7, 7), (2000, 2000), (1, 8)])
def test_quant_and_back(fake, K, pitch):
    X = rows(5, K, K, pitch)
    q, s = binding.quant_mxfp4(X)
    wq, ws = quantised(X)
    assert torch.equal(q, wq) and torch.equal(s, ws)
    assert q.stride(0) % 16 == 0 and s.stride(0) % 16 == 0 and q.stride(0) >= q.shape[1]
    close(binding.dequant_mxfp4(q, s, K), values(wq, ws, K))
    given = torch.zeros(5, 2048, dtype=torch.uint8)[:, :q.shape[1]], torch.zeros(5, 64, dtype=torch.uint8)[:, :s.shape[1]]
    got = binding.quant_mxfp4(X, Q=given[0], scales=given[1])
    assert got[0] is given[0] and got[1] is given[1] and torch.equal(got[0], wq) and torch.equal(got[1], ws)


def test_quant_sorted(fake):
    pos = torch.tensor([[0, 3], [4, 1], [2, 5]], dtype=torch.int32)
    plan = binding.ExpertPlan(torch.tensor([0, 2, 4], dtype=torch.int32), pos)
    X = rows(3, 40, 1)
    q, s = binding.quant_mxfp4(X, plan)
    wq, ws = quantised(X)
    for t in range(3):
        for j in range(2):
            r = int(pos[t, j])
            assert torch.equal(q[r], wq[t] if r < 4 else torch.zeros_like(wq[t]))
            assert torch.equal(s[r], ws[t] if r < 4 else torch.zeros_like(ws[t]))


@pytest.mark.parametrize("relu", [False, True])
def test_products(fake, relu):
    (a, sa), (w, sw) = binding.quant_mxfp4(rows(6, 96, 1)), binding.quant_mxfp4(rows(10, 96, 2))
    ref = values(a, sa) @ values(w, sw).t()
    close(binding.gemm_mxfp4(a, sa, w, sw, relu=relu), ref.clamp(min=0) if relu else ref)
    C = torch.zeros(6, 24, dtype=torch.bfloat16)[:, :10]
    assert binding.gemm_mxfp4(a, sa, w, sw, C=C, relu=relu) is C
    close(C, ref.clamp(min=0) if relu else ref)
    W = torch.zeros(3, 10, 64, dtype=torch.uint8)[..., :48]
    S = torch.full((3, 12, 16), 127, dtype=torch.uint8)[:, :10, :3]
    for e in range(3):
        W[e], S[e] = binding.quant_mxfp4(rows(10, 96, e + 5))
    o = torch.tensor([0, 2, 2, 5], dtype=torch.int32)
    C = binding.gemm_grouped_mxfp4(a, sa, o, W, S, relu=relu)
    for e in range(3):
        ref = values(a, sa)[o[e]:o[e + 1]] @ values(W[e], S[e]).t()
        close(C[o[e]:o[e + 1]], ref.clamp(min=0) if relu else ref)
    assert not C[5:].any()


def test_binding_refusals(fake):
    X = rows(4, 64, 1)
    q, s = binding.quant_mxfp4(X)
    W, S = q[None].repeat(2, 1, 1), s[None].repeat(2, 1, 1)
    o = torch.tensor([0, 1, 4], dtype=torch.int32)
    u8 = torch.uint8
    for error, call in [
            (ValueError, lambda: binding.quant_mxfp4(X[0])), (TypeError, lambda: binding.quant_mxfp4(X.float())),
            (ValueError, lambda: binding.quant_mxfp4(X, Q=q[:3])), (ValueError, lambda: binding.quant_mxfp4(X, scales=s.int())),
            (ValueError, lambda: binding.quant_mxfp4(X, binding.ExpertPlan(o, torch.zeros(3, 2, dtype=torch.int32)))),
            (TypeError, lambda: binding.dequant_mxfp4(q.int(), s)), (ValueError, lambda: binding.dequant_mxfp4(q, s[:, :1])),
            (ValueError, lambda: binding.dequant_mxfp4(q, s, 62)), (TypeError, lambda: binding.dequant_mxfp4(q, s, out_dtype=torch.float32)),
            (ValueError, lambda: binding.dequant_mxfp4(q, s, C=torch.zeros(4, 60, dtype=torch.bfloat16))),
            (TypeError, lambda: binding.gemm_mxfp4(q.view(torch.int8), s, q, s)), (TypeError, lambda: binding.gemm_mxfp4(q, s, q, s.int())),
            (ValueError, lambda: binding.gemm_mxfp4(q, s[:3], q, s)), (ValueError, lambda: binding.gemm_mxfp4(q, s, q[:, :16], s[:, :1])),
            (ValueError, lambda: binding.gemm_mxfp4(q[0], s[0], q, s)), (TypeError, lambda: binding.gemm_mxfp4(q, s, q, s, out_dtype=u8)),
            (ValueError, lambda: binding.gemm_mxfp4(q, s, q, s, C=torch.zeros(4, 5, dtype=torch.bfloat16))),
            (ValueError, lambda: binding.gemm_mxfp4(q.t().contiguous().t(), s, q, s)),
            (ValueError, lambda: binding.gemm_grouped_mxfp4(q, s, o, W[:1], S[:1])), (ValueError, lambda: binding.gemm_grouped_mxfp4(q, s, o, W, S[:, :2])),
            (TypeError, lambda: binding.gemm_grouped_mxfp4(q, s, o.long(), W, S)), (ValueError, lambda: binding.gemm_grouped_mxfp4(q, s, o, q, s))]:
        with pytest.raises(error):
            call()
    L = torch.zeros(4, 8)
    for error, call in [
            (ValueError, lambda: binding.expert_route(L[0], 2)), (ValueError, lambda: binding.expert_route(L, 0)),
            (ValueError, lambda: binding.expert_route(L, 2, score="tanh")), (TypeError, lambda: binding.expert_route(L.double(), 2)),
            (TypeError, lambda: binding.expert_route(L, 2, bias=torch.zeros(8).double())),
            (ValueError, lambda: binding.expert_route(L, 2, bias=torch.zeros(7)))]:
        with pytest.raises(error):
            call()


def test_tensors_off_the_gpu_are_refused():
    """No CPU path: the checks that tests replace are there."""
    X = rows(4, 64, 1)
    q, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    for call in (lambda: binding.quant_mxfp4(X), lambda: binding.dequant_mxfp4(q, s), lambda: binding.gemm_mxfp4(q, s, q, s),
                 lambda: binding.gemm_grouped_mxfp4(q, s, torch.tensor([0, 4], dtype=torch.int32), q[None], s[None]),
                 lambda: binding.expert_route(torch.zeros(4, 8), 2)):
        with pytest.raises((ValueError, RuntimeError, AssertionError)):
            call()


@pytest.mark.parametrize("kw", [dict(), dict(renorm=False, scale=2.0), dict(score="sigmoid", groups=4, topk_groups=2),
                                dict(score="sigmoid", groups=2, renorm=False)])
@pytest.mark.parametrize("layout", ["dense", "pitched", "transposed"])
def test_route_and_its_gradient(fake, kw, layout):
    g = torch.Generator().manual_seed(3)
    base = torch.randn((6, 8), generator=g)
    x = {"dense": lambda: base.clone(), "pitched": lambda: torch.cat((base, torch.full((6, 3), 9.0)), 1)[:, :8],
         "transposed": lambda: base.t().contiguous().t()}[layout]().requires_grad_(True)
    bias = torch.randn(8, generator=g) * 0.1
    ids, w = binding.expert_route(x, 3, bias=bias, **kw)
    args = dict(score="softmax", groups=1, topk_groups=kw.get("groups", 1), renorm=True, scale=1.0)
    args.update(kw)
    want = torch.tensor([choose(r, 3, args["score"], bias.tolist(), args["groups"], args["topk_groups"])
                         for r in x.detach().double().tolist()])
    assert torch.equal(ids.long(), want) and not ids.requires_grad
    x64 = base.double().requires_grad_(True)
    ref = weights_of(x64, want, args["score"], args["renorm"], args["scale"])
    assert torch.equal(w.detach(), ref.detach().float())
    gw = torch.randn((6, 3), generator=g)
    dx, = torch.autograd.grad(w, x, gw)
    want_dx, = torch.autograd.grad(ref, x64, gw.double())
    assert torch.allclose(dx.double(), want_dx, rtol=1e-6, atol=1e-12)
    plain = binding.expert_route(x.detach(), 3, bias=bias, **kw)
    assert torch.equal(plain[0], ids) and torch.equal(plain[1], w.detach())


def test_route_gradient_forms(fake):
    """Expanded and missing gradients; differentiable once; changes are noticed."""
    x = torch.randn((5, 8), generator=torch.Generator().manual_seed(1)).requires_grad_(True)
    ids, w = binding.expert_route(x, 2, renorm=False)
    dx, = torch.autograd.grad(w.sum(), x, retain_graph=True)
    want, = torch.autograd.grad(w, x, torch.ones(5, 2), retain_graph=True)
    assert torch.equal(dx, want)
    with pytest.raises(RuntimeError, match="once"):
        torch.autograd.grad(w.sum(), x, create_graph=True, retain_graph=True)
    ids.add_(0)
    with pytest.raises(RuntimeError, match="in-?place"):
        w.sum().backward()


# ------------------------------------------------- arithmetic of the kernels

@pytest.fixture(scope="module")
def chk(tmp_path_factory):
    import os
    import shutil
    import subprocess
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    here = os.path.dirname(os.path.abspath(__file__))
    out = str(tmp_path_factory.mktemp("mx") / "libmx_check.so")
    subprocess.run([gxx, "-O2", "-std=c++17", "-shared", "-fPIC", "-I",
                    os.path.join(os.path.dirname(here), "tiled_dense_gemm_tma_b200", "csrc"),
                    os.path.join(here, "mx_check.cpp"), "-o", out], check=True)
    return ctypes.CDLL(out)


@pytest.mark.parametrize("name", ["check_even_tiles", "check_route_lanes", "check_scale_places"])
def test_kernel_arithmetic(chk, name):
    fn = getattr(chk, name)
    fn.restype = ctypes.c_longlong
    n = ctypes.c_longlong(0)
    assert fn(ctypes.byref(n)) == 0 and n.value > 0


def test_slack_covers_the_errors(chk):
    """What two keys may differ by covers the errors of 32-bit scores and sums and
    the bits that number a lane's experts."""
    f = chk.slack
    f.restype = ctypes.c_float
    for sigmoid, highest in ((1, 1.0), (0, 1.0), (0, 0.01)):
        for size in (0.0, 0.5, 1.0, 100.0):
            for v in (1, 8, 64):
                got = f(sigmoid, ctypes.c_float(highest), ctypes.c_float(size), v)
                score = 2.0 ** -22 if sigmoid else 2.0 ** -18 * highest
                assert got >= 2 * score + 2 * 2.0 ** -24 * size + (v - 1) * 2.0 ** -23 * size
                assert got <= 1e-3 * (highest + size)


def test_sigmoid_bound_by_arithmetic():
    """s (1 - s) (2 + 1.5 |x|) 2^-23 and a reciprocal of one unit stay below 2^-22."""
    for i in range(-3000, 3001):
        x = i / 100
        s = 1 / (1 + math.exp(-x))
        assert s * (1 - s) * (2 + 1.5 * abs(x)) * 2.0 ** -23 + s * 2.0 ** -23 < 2.0 ** -22
