"""8-bit linear layers on a B200: the row quantiser and the 8-bit product
against their definitions in 64 bits."""
import numpy as np
import pytest
import torch

from expert_util import DTYPES, H, close, ints8, normal, pitched, positive, product8
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


def quant_ref(X):
    """q and scale from the formula in 64 bits: x * 127 and the quotient's
    exact halves are exact there."""
    x = X.double()
    top = x.abs().amax(1, keepdim=True) if x.shape[1] else torch.zeros(x.shape[0], 1, dtype=torch.float64, device=X.device)
    q = torch.where(top > 0, torch.round(x * 127 / torch.where(top > 0, top, 1)), 0)
    return q, (top / 127)[:, 0]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,K", [(1, 1), (3, 7), (5, 8), (2, 9), (7, 1000), (130, 1024), (4, 1030), (3, 4096), (2, 4104),
                                 (3, 8191), (1, 16384), (2, 16391), (2, 40000), (1000, 136)])
def test_quant_rows(tg, M, K, dtype):
    X = normal((M, K), DTYPES[dtype], M * 31 + K, extra=1)
    Q = pitched((M, K), torch.int8, extra=1)
    Q._base.fill_(99)
    q, s = tg.quant_i8(X, Q=Q)
    _status(tg)
    rq, rs = quant_ref(X)
    assert torch.equal(q.double(), rq)
    close(s, rs, rs * 2.0 ** -24 * 1.01, "scale")
    assert bool((Q._base[:, K:] == 99).all()), "write past the row"


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_quant_halves_go_to_even(tg, dtype):
    """Rows whose quotients are exact halves, just above and just below: every
    value of the type up to the largest one of the row."""
    dt = DTYPES[dtype]
    tops = [254.0, 127.0, 2.0 ** -10 * 254, 2.0 ** -14 * 127, 1.984375, 381.0]
    bits = torch.arange(0, 0x7c00 if dtype == "f16" else 0x7f80, dtype=torch.int32).to(torch.int16).view(dt)
    for top in tops:
        row = bits[bits.double() <= torch.tensor(top, dtype=dt).double()]
        K = row.numel()
        X = pitched((2, K), dt)
        X[0] = row.cuda()
        X[1] = -row.cuda()
        assert X.double().abs().max() == torch.tensor(top, dtype=dt).double()
        q, s = tg.quant_i8(X)
        rq, rs = quant_ref(X)
        assert torch.equal(q.double(), rq), top
    _status(tg)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_quant_special_rows(tg, dtype):
    dt = DTYPES[dtype]
    X = normal((8, 300), dt, 3)
    X[0] = 0
    X[1, 299] = float("inf")
    X[2, 0] = float("nan")
    X[3, 17] = -float("inf")
    X[4] = 0
    X[4, 5] = torch.finfo(dt).tiny * torch.finfo(dt).eps           # the smallest subnormal
    X[4, 6] = -X[4, 5]
    X[5] = torch.finfo(dt).max
    X[6] = -torch.finfo(dt).max
    q, s = tg.quant_i8(X)
    _status(tg)
    assert s[0].item() == 0 and not q[0].any()
    for r in (1, 2, 3):
        assert torch.isnan(s[r]) and not q[r].any()
    assert q[4, 5].item() == 127 and q[4, 6].item() == -127 and int(q[4].abs().sum()) == 254
    assert bool((q[5] == 127).all()) and bool((q[6] == -127).all())
    rq, rs = quant_ref(X)
    assert torch.equal(q[4:].double(), rq[4:])
    # the scale of a subnormal row is itself subnormal in fp32: off by half of 2^-149
    close(s[4:], rs[4:], rs[4:] * 2.0 ** -24 * 1.01 + 2.0 ** -150, "scale")


SHAPES = [(1, 1, 1), (1, 8, 16), (2, 33, 40), (5, 130, 127), (16, 256, 128), (17, 255, 129), (31, 640, 1000),
          (64, 100, 384), (127, 257, 500), (128, 512, 2048), (129, 520, 300), (255, 70, 129), (256, 256, 256),
          (300, 257, 1111), (513, 1000, 4096), (1025, 264, 100), (2, 4096, 8200), (3000, 72, 64)]


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(tg, M, N, K, trans):
    dtype = "bf16" if (M + N) % 2 else "f16"
    dt = DTYPES[dtype]
    relu = (M + K) % 3 == 0
    A = ints8((M, K), 1, extra=1)
    W = ints8((N, K) if trans else (K, N), 2)
    rs, cs = positive((M,), 3, 1e-3, 2e-3), positive((N,), 4, 1e-3, 2e-3)
    big, C, pad = guarded_out(M, N, dtype)
    tg.gemm_w8a8(A, rs, W, cs, C=C, relu=relu, trans_b=trans)
    _status(tg)
    ref, bound = product8(A, rs, W.t() if trans else W, cs, dt)
    if relu:
        ref = ref.clamp(min=0)
    close(C, ref, bound, f"{M} {N} {K}")
    check_guard(big, dtype, M, N, pad)


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("M", [3, 200])
def test_largest_sums_are_exact(tg, M, trans):
    """All operands at -128: the sum K * 2^14 grows to the edge of 32 bits."""
    K, N = 131071, 40
    A = pitched((M, K), torch.int8)
    A.fill_(-128)
    W = pitched((N, K) if trans else (K, N), torch.int8)
    W.fill_(-128)
    one = torch.ones(M, device="cuda")
    C = tg.gemm_w8a8(A, one, W, torch.full((N,), 2.0 ** -16, device="cuda"), trans_b=trans)
    _status(tg)
    # 131071 * 2^14 * 2^-16 = 32767.75, to bf16: 32768
    assert bool((C == 32768).all())


def test_scales_keep_their_order(tg):
    """Scales whose product would leave fp32's range, though the result does not."""
    A, W = ints8((4, 64), 1), ints8((64, 8), 2)
    rs = torch.full((4,), 1e-30, device="cuda")
    cs = torch.full((8,), 1e28, device="cuda")
    C = tg.gemm_w8a8(A, rs, W, cs)
    ref, bound = product8(A, rs, W, cs, torch.bfloat16)
    close(C, ref, bound)
    rs = torch.full((4,), float("nan"), device="cuda")
    rs[1:] = 1.0
    C = tg.gemm_w8a8(A, rs, W, torch.ones(8, device="cuda"))
    assert bool(torch.isnan(C[0]).all()) and not bool(torch.isnan(C[1:]).any())
    _status(tg)


def test_linear_layer_end_to_end(tg):
    """Quantiser and product together, as a layer uses them, on their own
    stream and replayed from a graph."""
    X = normal((300, 520), torch.bfloat16, 1)
    W = ints8((264, 520), 2, -127)
    ws = positive((264,), 3)
    q, s = tg.quant_i8(X)
    eager = tg.gemm_w8a8(q, s, W, ws, trans_b=True)
    rq, rs = quant_ref(X)
    ref = (rq @ W.double().t()) * rs[:, None] * ws.double()
    close(eager, ref, ref.abs() * (H[torch.bfloat16] * 1.01 + 5 * 2.0 ** -24) + 1e-30)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        q2, s2 = tg.quant_i8(X)
        out = tg.gemm_w8a8(q2, s2, W, ws, trans_b=True)
    out.zero_()
    for _ in range(3):
        g.replay()
    _status(tg)
    assert torch.equal(out, eager)
    X.copy_(normal((300, 520), torch.bfloat16, 9))                # new contents, same buffers
    g.replay()
    q, s = tg.quant_i8(X)
    assert torch.equal(out, tg.gemm_w8a8(q, s, W, ws, trans_b=True))
    _status(tg)
