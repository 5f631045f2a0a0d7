"""Edges of the 8-bit linear layers on a B200: rows of very large values, rows
that hold a NaN or an infinity under ReLU."""
import pytest
import torch

from expert_util import DTYPES, close, ints8, normal, offsets_of, pitched, positive, product8

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


# ---------------------------------------------------------------- quantiser

TOPS = [2.0 ** 127, 2.0 ** 125, 254 * 2.0 ** 119, 254 * 2.0 ** 120, 255 * 2.0 ** 120, 127 * 2.0 ** 114, 2.0 ** 8, 1.0,
        255 / 256, 2.0 ** -99, 2.0 ** -100, 129 * 2.0 ** -108, 254 * 2.0 ** -133]


def quant_ref(X):
    """In 64 bits x * 127 and exact halves of the quotient are exact."""
    x = X.double()
    top = x.abs().amax(1, keepdim=True)
    return torch.round(x * 127 / top), (top / 127)[:, 0]


@pytest.mark.parametrize("top", TOPS)
def test_quant_of_every_value_up_to_any_maximum(tg, top):
    """Every bfloat16 value up to a row's maximum, from the largest maxima there
    are to subnormal ones: one long row, and rows of eight values that put the
    maximum beside each value (the two are rounded together)."""
    bits = torch.arange(0, 0x7f80, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    row = bits[bits.double() <= top]
    assert row.double().max() == top
    X = pitched((2, row.numel()), torch.bfloat16)
    X[0], X[1] = row.cuda(), -row.cuda()
    near = row[row.double() >= top * 2.0 ** -9].cuda()        # |q| of 1/4 and more
    pairs = pitched((near.numel(), 8), torch.bfloat16)
    pairs[:, 0::2], pairs[:, 1::2] = near[:, None], torch.tensor(-top, dtype=torch.bfloat16)
    for x in (X, pairs):
        q, s = tg.quant_i8(x)
        _status(tg)
        rq, rs = quant_ref(x)
        assert torch.equal(q.double(), rq)
        close(s, rs, rs * 2.0 ** -24 * 1.01 + 2.0 ** -150, "scale")


def test_quant_of_the_largest_halves(tg):
    """A maximum of 2^127 beside its half: 63.5 goes to 64, the maximum to 127."""
    X = pitched((1, 8), torch.bfloat16)
    X[0] = torch.tensor([2.0 ** 127, 2.0 ** 126, -2.0 ** 126, -2.0 ** 127, 0.0, 2.0 ** 125, 1.0, 2.0 ** -133])
    q, s = tg.quant_i8(X)
    _status(tg)
    assert q[0].tolist() == [127, 64, -64, -127, 0, 32, 0, 0]     # 31.75 -> 32


# ------------------------------------------------------------ NaN under ReLU

@pytest.mark.parametrize("relu", [False, True])
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("M,N", [(3, 40), (16, 9000), (100, 264), (200, 264), (100, 20000)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_rows_with_a_nan_stay_nan(tg, M, N, trans, relu, dtype):
    """A row that holds an infinity or a NaN makes its products NaN, also under
    ReLU, on both kernels; its neighbours are as without it."""
    dt = DTYPES[dtype]
    K = 96
    X = normal((M, K), dt, 1)
    X[1, 5], X[M - 1, 95] = float("inf"), float("nan")
    W = ints8((N, K) if trans else (K, N), 2)
    ws = positive((N,), 3, 1e-3, 2e-3)
    q, s = tg.quant_i8(X)
    C = tg.gemm_w8a8(q, s, W, ws, out_dtype=dt, relu=relu, trans_b=trans)
    _status(tg)
    bad = torch.zeros(M, dtype=torch.bool, device="cuda")
    bad[1] = bad[M - 1] = True
    assert bool(torch.isnan(C[bad]).all())
    ref, bound = product8(q[~bad], s[~bad], W.t() if trans else W, ws, dt)
    close(C[~bad], ref.clamp(min=0) if relu else ref, bound)


@pytest.mark.parametrize("trans", [False, True])
def test_rows_with_a_nan_stay_nan_in_groups(tg, trans):
    counts, K, N = [40, 0, 300, 7], 80, 136
    R = sum(counts) + 5
    A, B = ints8((R, K), 1), ints8((4, N, K) if trans else (4, K, N), 2)
    rs, cs = positive((R,), 3, 1e-3, 2e-3), positive((4, N), 4, 1e-3, 2e-3)
    rs[[0, 39, 41, 346, 350]] = float("nan")                  # row 350 lies behind the last group
    C = tg.gemm_grouped_w8a8(A, rs, offsets_of(counts), B, cs, relu=True, trans_b=trans)
    _status(tg)
    nan = torch.isnan(C)
    assert bool(nan[[0, 39, 41, 346]].all()) and int(nan.any(1).sum()) == 4
    assert not C[347:].any()
    at = 0
    for e, n in enumerate(counts):
        part = torch.arange(at, at + n, device="cuda")
        part = part[~torch.isnan(rs[part])]
        ref, bound = product8(A[part], rs[part], B[e].t() if trans else B[e], cs[e], torch.bfloat16)
        close(C[part], ref.clamp(min=0), bound)
        at += n
