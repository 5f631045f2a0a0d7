"""Microscaled 4-bit floating point: quantisation, back, and the products,
against their definitions in 64 bits."""
import pytest
import torch

import tiled_dense_gemm_tma_b200 as tg
from expert_util import DTYPES, close, normal, offsets_of, pitched
from mxfp4_util import bytes_like, product, quantised, random_blocks, values

pytestmark = pytest.mark.gpu


def guarded(M, N):
    """A uint8 M x N view with rows and columns of 0xa5 around it."""
    ld = -(-N // 16) * 16 + 16
    big = torch.full((M + 2, ld), 0xa5, dtype=torch.uint8, device="cuda")
    return big, big[1:M + 1, :N]


def untouched(big, view):
    mask = torch.ones_like(big, dtype=torch.bool)
    mask[1:1 + view.shape[0], :view.shape[1]] = False
    assert bool((big[mask] == 0xa5).all())


# ---------------------------------------------------------------- quantiser

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 2), (3, 7), (2, 31), (5, 33), (7, 64), (2, 255), (300, 257), (33, 1000),
                                 (17, 2040), (9, 8192), (2500, 1032), (1, 100003)])
def test_quant_rows(M, K, dtype):
    X = normal((M, K), DTYPES[dtype], seed=M + K, extra=1)
    bq, Q = guarded(M, (K + 1) // 2)
    bs, S = guarded(M, -(-K // 32))
    out = tg.quant_mxfp4(X, Q=Q, scales=S)
    assert out[0] is Q and out[1] is S
    q, s = quantised(X)
    assert torch.equal(S.cpu(), s)
    assert torch.equal(Q.cpu(), q)
    untouched(bq, Q)
    untouched(bs, S)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_quant_borders(dtype):
    """Every multiple of 1/16 below 8 at every power of two: halves between
    codes, what saturates, subnormals and the largest values."""
    dt = DTYPES[dtype]
    steps = torch.arange(-127, 128, dtype=torch.float64) / 16
    rows = []
    for e in range(-130, 126, 3) if dtype == "bf16" else range(-24, 13):
        x = (steps * 2.0 ** e).to(dt)
        x = torch.where(torch.isfinite(x.double()), x, torch.zeros_like(x))
        # each block holds the largest one, so that the scale is 2^e
        parts = [torch.cat((x[-1:], x[i:i + 31])) for i in range(0, 255, 31)]
        rows.append(torch.cat([torch.nn.functional.pad(p, (0, 32 - len(p))) for p in parts]))
    X = torch.stack(rows).cuda()
    Q, S = tg.quant_mxfp4(X)
    q, s = quantised(X)
    assert torch.equal(S.cpu(), s)
    assert torch.equal(Q.cpu(), q)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_quant_special_blocks(dtype):
    dt = DTYPES[dtype]
    X = normal((8, 96), dt, seed=3)
    X[0, 32:64] = 0
    X[1, :] = -0.0
    X[2, 40] = float("inf")
    X[3, 95] = float("nan")
    X[4, 0] = -float("inf")
    X[5, 64:] = torch.finfo(dt).max
    X[6, :32] = torch.finfo(dt).smallest_normal
    X[7, 32:64] = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps     # the smallest subnormal
    Q, S = tg.quant_mxfp4(X)
    q, s = quantised(X)
    assert torch.equal(S.cpu(), s) and torch.equal(Q.cpu(), q)
    Y = tg.dequant_mxfp4(Q, S, out_dtype=dt)
    assert bool(Y[2, 32:64].isnan().all()) and bool(Y[3, 64:].isnan().all()) and bool(Y[4, :32].isnan().all())
    assert bool((Y[0, 32:64] == 0).all()) and int(Y.isnan().sum()) == 96


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,k,H,E", [(1, 1, 32, 4), (5, 2, 40, 3), (130, 6, 2040, 64), (64, 8, 33, 8), (300, 4, 1024, 16)])
def test_quant_sorted(T, k, H, E, dtype):
    """Rows sorted on the way are the quantised rows gathered."""
    g = torch.Generator().manual_seed(T)
    ids = torch.randint(-1, E + 1, (T, k), generator=g).int().cuda()        # repeated experts, dropped choices
    plan = tg.expert_sort(ids, E)
    X = normal((T, H), DTYPES[dtype], seed=H)
    bq, Q = guarded(T * k, (H + 1) // 2)
    bs, S = guarded(T * k, -(-H // 32))
    tg.quant_mxfp4(X, plan, Q=Q, scales=S)
    q, s = quantised(X)
    token = plan.src.long().cpu() // k
    kept = int(plan.offsets[-1])
    q, s = q[token], s[token]
    q[kept:] = 0
    s[kept:] = 0
    assert torch.equal(Q.cpu(), q) and torch.equal(S.cpu(), s)
    untouched(bq, Q)
    untouched(bs, S)


def test_quant_sorted_skips_positions_outside():
    T, k, H = 3, 2, 64
    pos = torch.tensor([[0, -1], [7, 2], [1, 5]], dtype=torch.int32, device="cuda")
    plan = tg.ExpertPlan(torch.tensor([0, 3], dtype=torch.int32, device="cuda"), pos)
    X = normal((T, H), torch.bfloat16, seed=1)
    bq, Q = guarded(T * k, H // 2)
    bs, S = guarded(T * k, H // 32)
    tg.quant_mxfp4(X, plan, Q=Q, scales=S)
    q, s = quantised(X)
    for row, token in ((0, 0), (2, 1), (1, 2)):
        assert torch.equal(Q[row].cpu(), q[token]) and torch.equal(S[row].cpu(), s[token])
    assert bool((Q[5] == 0).all()) and bool((S[5] == 0).all())
    assert bool((Q[3:5] == 0xa5).all())
    untouched(bq, Q)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_dequant_every_code_and_scale(dtype):
    """All 256 scales times all 16 codes, rounded once to the type."""
    q = torch.zeros(256, 16, dtype=torch.uint8)
    q[:, :8] = torch.arange(8) * 34 + 16                                    # 0|1, 2|3, ... 14|15
    s = torch.arange(256, dtype=torch.uint8)[:, None].contiguous()
    Y = tg.dequant_mxfp4(bytes_like(q.cuda()), bytes_like(s.cuda()), 32, out_dtype=DTYPES[dtype])
    # two significant bits: exact in float32 but for what that cannot hold at all
    want = values(q, s).float().to(DTYPES[dtype])
    same = (Y.cpu() == want) | (Y.cpu().isnan() & want.isnan())
    assert bool(same.all())


@pytest.mark.parametrize("K", [1, 6, 8, 31, 33, 2040])
def test_dequant_widths(K):
    q, s = random_blocks((5, K), seed=K)
    big = torch.full((7, K + 16 + (-K) % 8), 7.0, dtype=torch.float16, device="cuda")
    C = big[1:6, :K]
    tg.dequant_mxfp4(q, s, K, C=C)
    assert torch.equal(C.double(), values(q, s, K))
    big[1:6, :K] = 7.0
    assert bool((big == 7.0).all())


# ------------------------------------------------------------------ products

def check_dense(M, N, K, dtype, relu=False, seed=0, lo=120, hi=130):
    a, sa = random_blocks((M, K), seed, lo, hi)
    w, sw = random_blocks((N, K), seed + 1, lo, hi, extra=1)
    out = pitched((M + 2, N), DTYPES[dtype], extra=1)
    big = out.new_full((M + 2, out.stride(0)), 7.0)
    C = big[1:M + 1, :N]
    tg.gemm_mxfp4(a, sa, w, sw, C=C, relu=relu)
    ref, bound = product(values(a, sa), values(w, sw), DTYPES[dtype])
    close(C, ref.clamp(min=0) if relu else ref, bound, f"{M}x{N}x{K}")
    C.fill_(7.0)
    assert bool((big == 7.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 2), (1, 8, 32), (1, 128, 64), (3, 100, 30), (16, 129, 512), (16, 1000, 544), (1, 8192, 2048),
    (17, 300, 1056), (33, 8, 4096), (64, 256, 100), (100, 513, 2000), (128, 8192, 1024), (128, 24, 514)])
def test_product_few_rows(M, N, K, dtype):
    check_dense(M, N, K, dtype, relu=M % 2 == 0, seed=M)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [
    (129, 8, 2), (129, 128, 32), (200, 256, 256), (224, 260, 512), (225, 256, 770), (256, 24, 1024), (300, 1000, 500),
    (449, 512, 1280), (1000, 777, 2016), (40, 10000, 96), (700, 5000, 800), (2000, 2048, 256)])
def test_product_many_rows(M, N, K, dtype):
    check_dense(M, N, K, dtype, relu=M % 2 == 0, seed=M)


@pytest.mark.parametrize("M", [5, 128, 700])
def test_product_scale_of_each_block(M):
    """One block of each row of A and W is not zero: a scale taken from
    another row, block or byte shows as a power of two."""
    N, K = 300, 1312
    g = torch.Generator().manual_seed(M)
    nb = K // 32
    q = torch.zeros(M, nb, 16, dtype=torch.uint8)
    at = torch.randint(0, nb, (M,), generator=g)
    q[torch.arange(M), at] = 0x22                                           # ones
    s = torch.randint(60, 70, (M, nb), generator=g, dtype=torch.uint8)
    a, sa = bytes_like(q.view(M, -1).cuda()), bytes_like(s.cuda())
    w = bytes_like(torch.full((N, K // 2), 0x22, dtype=torch.uint8).cuda())
    t = torch.randint(180, 190, (N, nb), generator=g, dtype=torch.uint8)
    C = tg.gemm_mxfp4(a, sa, w, bytes_like(t.cuda()), out_dtype=torch.bfloat16)
    e = s.long()[torch.arange(M), at][:, None] + t.long()[:, at].t() - 254
    assert torch.equal(C.cpu().double(), 32.0 * torch.exp2(e.double()))


@pytest.mark.parametrize("M,N,K", [(1, 256, 512), (16, 200, 4096), (100, 300, 1024), (300, 400, 2048), (1000, 512, 512)])
def test_product_exact_sums(M, N, K):
    """Sums that fp32 holds exactly come out as the one rounding of them."""
    g = torch.Generator().manual_seed(K)
    codes = torch.tensor([0, 1, 2, 4, 9, 10, 12], dtype=torch.uint8)        # 0, .5, 1, 2 and negatives
    def make(rows):
        c = codes[torch.randint(0, 7, (rows, K // 2, 2), generator=g)]
        return bytes_like((c[..., 0] | c[..., 1] << 4).cuda())
    a, w = make(M), make(N)
    sa = bytes_like(torch.full((M, K // 32), 127, dtype=torch.uint8).cuda())
    sw = bytes_like(torch.randint(126, 129, (N, K // 32), generator=g, dtype=torch.uint8).cuda())
    C = tg.gemm_mxfp4(a, sa, w, sw, out_dtype=torch.float16)
    ref = values(a, sa) @ values(w, sw).t()
    assert torch.equal(C, ref.to(torch.float16))


@pytest.mark.parametrize("M", [3, 40, 300])
def test_product_odd_width(M):
    """Rows of odd length end in a zero half byte."""
    X, W = normal((M, 77), torch.bfloat16, 1), normal((50, 77), torch.bfloat16, 2)
    (a, sa), (w, sw) = tg.quant_mxfp4(X), tg.quant_mxfp4(W)
    C = tg.gemm_mxfp4(a, sa, w, sw)
    ref, bound = product(values(a, sa, 77), values(w, sw, 77), torch.bfloat16)
    close(C, ref, bound)


@pytest.mark.parametrize("relu", [False, True])
@pytest.mark.parametrize("M", [2, 100, 400])
def test_product_nan_scale(M, relu):
    """A NaN block makes its own row (or column) NaN and nothing else."""
    a, sa = random_blocks((M, 640), 1)
    w, sw = random_blocks((200, 640), 2)
    sa[1, 3] = 255
    sw[7, 19] = 255
    C = tg.gemm_mxfp4(a, sa, w, sw, relu=relu)
    assert bool(C[1].isnan().all()) and bool(C[:, 7].isnan().all())
    assert int(C.isnan().sum()) == 200 + M - 1


@pytest.mark.parametrize("M", [4, 300])
def test_product_empty(M):
    a, s = torch.zeros(M, 0, dtype=torch.uint8, device="cuda"), torch.zeros(M, 0, dtype=torch.uint8, device="cuda")
    w, t = torch.zeros(9, 0, dtype=torch.uint8, device="cuda"), torch.zeros(9, 0, dtype=torch.uint8, device="cuda")
    assert torch.equal(tg.gemm_mxfp4(a, s, w, t), torch.zeros(M, 9, dtype=torch.bfloat16, device="cuda"))
    assert tg.gemm_mxfp4(a[:0], s[:0], w, t).shape == (0, 9)
    assert tg.gemm_mxfp4(a, s, w[:0], t[:0]).shape == (M, 0)


def check_grouped(counts, tail, N, K, dtype, relu=False, seed=0):
    R, E = sum(counts) + tail, len(counts)
    a, sa = random_blocks((R, K), seed)
    w, sw = random_blocks((E, N, K), seed + 1)
    if tail:
        sa[R - tail:] = 255                                                 # rows behind the last group are not read
    C = tg.gemm_grouped_mxfp4(a, sa, offsets_of(counts), w, sw, out_dtype=DTYPES[dtype], relu=relu)
    at = 0
    for e, n in enumerate(counts):
        part = slice(at, at + n)
        ref, bound = product(values(a[part], sa[part]), values(w[e], sw[e]), DTYPES[dtype])
        close(C[part], ref.clamp(min=0) if relu else ref, bound, f"group {e}")
        at += n
    assert bool((C[at:] == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("counts,tail,N,K", [
    ([1], 0, 8, 32), ([3, 0, 5], 2, 100, 64), ([0, 0, 1, 0], 0, 256, 512), ([32, 33, 31, 0, 1], 7, 300, 1056),
    ([224, 225, 448, 449, 1], 3, 264, 800), ([1000, 24], 0, 520, 2016), ([0, 0], 5, 64, 64), ([1] * 70, 0, 1000, 160),
    ([700], 100, 257, 96)])
def test_grouped(counts, tail, N, K, dtype):
    check_grouped(counts, tail, N, K, dtype, relu=tail % 2 == 1, seed=N)


def test_grouped_nan_stays_in_its_group():
    """A NaN in the scales of one group's rows or weights reaches no other's,
    although tiles read past a group's end."""
    counts = [5, 40, 3]
    a, sa = random_blocks((48, 256), 1)
    w, sw = random_blocks((3, 128, 256), 2)
    sa[5] = 255
    sw[2] = 255
    C = tg.gemm_grouped_mxfp4(a, sa, offsets_of(counts), w, sw)
    nan = C.isnan().any(1).cpu()
    assert nan.nonzero().flatten().tolist() == [5, 45, 46, 47]


def test_grouped_equals_dense_rows():
    """One group of all rows is the dense product, bit for bit."""
    a, sa = random_blocks((300, 1024), 5)
    w, sw = random_blocks((1, 512, 1024), 6)
    C = tg.gemm_grouped_mxfp4(a, sa, offsets_of([300]), w, sw)
    assert torch.equal(C, tg.gemm_mxfp4(a, sa, w[0], sw[0]))
    assert torch.equal(C, tg.gemm_grouped_mxfp4(a, sa, offsets_of([300]), w, sw))


@pytest.mark.parametrize("M", [3, 200])
def test_scales_at_the_ends_of_their_range(M):
    """Scales of 2^-127 to 2^127 whose product is moderate are exact together."""
    N, K = 140, 64
    a = bytes_like(torch.full((M, K // 2), 0x22, dtype=torch.uint8).cuda())             # ones
    w = bytes_like(torch.full((N, K // 2), 0x22, dtype=torch.uint8).cuda())
    for ea, ew in ((0, 254), (254, 0), (1, 250), (3, 240), (127, 127), (0, 200), (200, 0), (64, 190)):
        sa = bytes_like(torch.full((M, 2), ea, dtype=torch.uint8).cuda())
        sw = bytes_like(torch.full((N, 2), ew, dtype=torch.uint8).cuda())
        C = tg.gemm_mxfp4(a, sa, w, sw)
        assert bool((C.double() == 64.0 * 2.0 ** (ea + ew - 254)).all()), (ea, ew, C[0, 0].item())
