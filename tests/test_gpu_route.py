"""Routing to experts against its definition in 64 bits: choices, weights and
the gradient of the logits."""
import math

import pytest
import torch

import tiled_dense_gemm_tma_b200 as tg
from expert_util import close
from route_util import choose, relative, weights_of

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
SMALL = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -24}


def check(x, topk, bias=None, score="softmax", groups=1, keep=1, renorm=True, scale=1.0, grad=True, seed=0):
    """x: logits on the device, without NaN and plus infinity."""
    T, E = x.shape
    leaf = x.detach().requires_grad_(grad)
    ids, w = tg.expert_route(leaf, topk, bias=bias, score=score, groups=groups, topk_groups=keep, renorm=renorm,
                             scale=scale)
    assert ids.dtype == torch.int32 and w.dtype == torch.float32 and ids.shape == w.shape == (T, topk)
    rows = x.double().tolist()
    b = None if bias is None else bias.double().tolist()
    want = torch.tensor([choose(r, topk, score, b, groups, keep) for r in rows], dtype=torch.int32).view(T, topk)
    assert torch.equal(ids.cpu(), want)
    x64 = x.detach().cpu().double().requires_grad_(True)
    ref = weights_of(x64, want, score, renorm, scale)
    rel = relative(x).cpu()
    close(w.detach().cpu(), ref.detach(), ref.detach() * rel + scale * 2.0 ** -126, "weights")
    if not grad:
        return ids, w
    g = torch.randn((T, topk), generator=torch.Generator().manual_seed(seed))
    dx, = torch.autograd.grad(w, leaf, g.cuda())
    want_dx, = torch.autograd.grad(ref, x64, g.double())
    # each entry is a weight (or the whole row's softmax) times a difference of g and
    # a mean of g, each a product and a sum of topk terms
    p = torch.softmax(torch.where(torch.isneginf(x64), -1e300, x64), 1).detach() if score == "softmax" and not renorm else 0
    size = torch.zeros(T, E, dtype=torch.float64) + p * scale
    size.scatter_add_(1, want.clamp(min=0).long(), ref.detach().abs())
    most = g.abs().double().amax(1, keepdim=True)
    bound = size * most * 2 * (2 * rel + (topk + 8) * 2.0 ** -24)
    # the reference's own rounding: terms of at most scale * most that cancel (with renorm
    # those of the row's other logits to 0), summed over the row in 64 bits
    bound = bound + (topk + E) * scale * most * 2.0 ** -52
    close(dx.cpu(), want_dx, bound + HALF[dx.dtype] * want_dx.abs() + SMALL[dx.dtype], "gradient")
    return ids, w


def logits(T, E, dtype, seed, scale=1.5, pitch=None):
    x = torch.randn((T, E), generator=torch.Generator().manual_seed(seed)) * scale
    if pitch is None:
        return x.to(DT[dtype]).cuda()
    big = torch.full((T, pitch), math.nan, dtype=DT[dtype], device="cuda")
    big[:, :E] = x
    return big[:, :E]


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,dtype", [
    (1, 1, 1, "f32"), (1, 2, 2, "bf16"), (7, 3, 1, "f16"), (8, 8, 2, "bf16"), (9, 31, 4, "f32"), (100, 33, 5, "f32"),
    (65, 60, 6, "bf16"), (1000, 128, 8, "f32"), (33, 256, 8, "f16"), (20, 500, 32, "f32"), (17, 1000, 1, "bf16"),
    (5, 1024, 32, "f32"), (12, 32, 32, "f32")])
def test_route(T, E, k, dtype, score, renorm):
    check(logits(T, E, dtype, T + E), k, score=score, renorm=renorm, scale=1.0 if E % 2 else 2.5)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,dtype", [(9, 8, 2, "bf16"), (50, 60, 6, "f32"), (300, 256, 8, "f32"), (10, 1024, 31, "f32"),
                                         (6, 64, 32, "f16"), (40, 7, 7, "f32")])
def test_route_bias(T, E, k, dtype, score, renorm):
    bias = torch.randn(E, generator=torch.Generator().manual_seed(E)).cuda() * (0.05 if score == "sigmoid" else 0.01)
    check(logits(T, E, dtype, T), k, bias=bias, score=score, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("with_bias", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,groups,keep,k,dtype", [
    (30, 256, 8, 4, 8, "f32"), (9, 8, 2, 1, 2, "bf16"), (20, 15, 5, 2, 6, "f32"), (11, 6, 6, 3, 3, "f16"),
    (13, 96, 3, 2, 9, "f32"), (25, 160, 32, 5, 4, "f32"), (8, 1024, 16, 3, 32, "f32"), (7, 640, 20, 20, 8, "f32"),
    (5, 32, 32, 1, 1, "f32"), (6, 999, 27, 2, 20, "bf16")])
def test_route_groups(T, E, groups, keep, k, dtype, score, with_bias):
    bias = torch.randn(E, generator=torch.Generator().manual_seed(E)).cuda() * 0.03 if with_bias else None
    check(logits(T, E, dtype, T + 1), k, bias=bias, score=score, groups=groups, keep=keep, renorm=with_bias)


@pytest.mark.parametrize("groups,keep", [(1, 1), (4, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [True, False])
def test_route_ties_go_to_the_lowest(with_bias, score, groups, keep):
    """Few distinct logits and biases: most comparisons are ties."""
    g = torch.Generator().manual_seed(5)
    x = torch.randint(-1, 2, (200, 64), generator=g).float().cuda() + 0.0
    x[:20] = 0
    x[20:30] = -0.0
    x[30:40, ::2] = -0.0
    x[30:40, 1::2] = 0.0
    bias = (torch.randint(0, 2, (64,), generator=g).float() * 0.25).cuda() if with_bias else None
    check(x, 6, bias=bias, score=score, groups=groups, keep=keep)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_order_below_32_bits(score):
    """Keys that differ by less than 32 bits show, either way round."""
    g = torch.Generator().manual_seed(9)
    wrong = 0
    for flip in (1, -1):
        x = torch.randn(16, generator=g) * 0.1
        row = x.double().tolist()
        if score == "softmax":
            top = max(row)
            e = [math.exp(v - top) for v in row]
            p = [v / math.fsum(e) for v in e]
        else:
            p = [1 / (1 + math.exp(-v)) for v in row]
        # expert j's key equals expert 0's but for 2^-20 of the distance of their scores
        bias = torch.tensor([(p[0] - q) * (1 + flip * 2.0 ** -20) for q in p])
        keys = [a + b for a, b in zip(p, bias.double().tolist())]
        assert len(set(keys)) == 16
        narrow = [torch.tensor(a).float().item() + b for a, b in zip(p, bias.tolist())]
        wrong += sorted(range(16), key=lambda e: -keys[e]) != sorted(range(16), key=lambda e: -torch.tensor(narrow[e]).float().item())
        check(x[None].repeat(3, 1).cuda(), 7, bias=bias.cuda(), score=score)
    assert wrong                                       # 32 bits alone would not do


def test_route_groups_below_32_bits():
    """Groups whose sums differ by less than 32 bits."""
    for flip in (1, -1):
        x = torch.tensor([0.3, 0.1, 0.2, -0.1, 0.4, 0.15, 0.25, 0.05])
        p = [1 / (1 + math.exp(-v)) for v in x.double().tolist()]
        first = p[0] + p[1]
        bias = torch.zeros(8)
        for gr in range(1, 4):
            gap = first - p[2 * gr] - p[2 * gr + 1]
            bias[2 * gr] = gap * (1 + flip * gr * 2.0 ** -21)
        check(x[None].cuda(), 4, bias=bias.cuda(), score="sigmoid", groups=4, keep=2)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,keep,with_bias", [(1, 1, False), (1, 1, True), (4, 2, False), (4, 2, True)])
def test_route_masked(groups, keep, with_bias, score, renorm):
    """Rows with no expert, fewer than topk, and whole groups gone."""
    x = logits(12, 32, "f32", 4)
    x[0] = -math.inf
    x[1, 1:] = -math.inf
    x[2, :31] = -math.inf
    x[3, 3:30] = -math.inf
    x[4, 8:] = -math.inf
    x[5, :24] = -math.inf
    x[6, ::2] = -math.inf
    x[7] = torch.finfo(torch.float32).min               # the lowest value masks no expert
    x[8, 5:] = torch.finfo(torch.float32).min
    x[9, :] = -math.inf
    x[9, [0, 8, 16, 24]] = torch.tensor([0.1, 0.5, 0.2, 0.3], device="cuda")     # one expert to a group
    bias = torch.randn(32, generator=torch.Generator().manual_seed(1)).cuda() * 0.02 if with_bias else None
    ids, w = tg.expert_route(x, 6, bias=bias, score=score, groups=groups, topk_groups=keep, renorm=renorm)
    rows = x.double().tolist()
    b = None if bias is None else bias.double().tolist()
    want = torch.tensor([choose(r, 6, score, b, groups, keep) for r in rows], dtype=torch.int32)
    assert torch.equal(ids.cpu(), want)
    assert bool((w[ids < 0] == 0).all()) and bool((ids[0] == -1).all())
    assert bool(torch.isfinite(w).all())
    if renorm:
        total = w.double().sum(1).cpu()
        some = (want >= 0).any(1)
        assert bool(((total - 1).abs() <= 16 * 2.0 ** -24)[some].all())
    leaf = x.requires_grad_(True)
    ids2, w2 = tg.expert_route(leaf, 6, bias=bias, score=score, groups=groups, topk_groups=keep, renorm=renorm)
    g = torch.randn((12, 6), generator=torch.Generator().manual_seed(2)).cuda()
    g[want.cuda() < 0] = math.nan                        # what a dropped choice is told matters to nothing
    dx, = torch.autograd.grad(w2, leaf, g)
    assert bool(torch.isfinite(dx).all())
    assert bool((dx[x.detach() == -math.inf] == 0).all())
    keep_rows = [1, 2, 3, 4, 5, 6, 9, 10, 11]
    x64 = x.detach().cpu().double().requires_grad_(True)
    ref = weights_of(x64, want, score, renorm, 1.0)
    # minus infinity in a softmax has gradient 0 by the formula, NaN by its chain rule
    gd = torch.where(want < 0, 0.0, g.cpu().double())
    if score == "sigmoid" or not renorm:
        live = ~torch.isneginf(x64.detach())
        p = torch.softmax(x64.detach(), 1) if score == "softmax" else torch.sigmoid(x64.detach())
    want_dx = torch.zeros(12, 32, dtype=torch.float64)
    wr = ref.detach()
    for t in keep_rows:
        for j in range(6):
            e = int(want[t, j])
            if e < 0:
                continue
            mean = float((gd[t] * wr[t]).sum())
            if renorm:
                want_dx[t, e] += wr[t, j] * (gd[t, j] - mean) * (1 if score == "softmax" else 1 - p[t, e])
            elif score == "sigmoid":
                want_dx[t, e] += gd[t, j] * p[t, e] * (1 - p[t, e])
            else:
                want_dx[t] -= gd[t, j] * p[t, e] * p[t]
                want_dx[t, e] += gd[t, j] * p[t, e]
    bound = 2.0 ** -24 * 400 * gd.abs().amax(1, keepdim=True).expand(-1, 32)
    close(dx.cpu()[keep_rows], want_dx[keep_rows], bound[keep_rows], "gradient")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,with_bias,renorm", [(1, False, True), (1, True, True), (4, True, True), (4, False, False),
                                                     (1, False, False)])
def test_route_nan_and_infinity_show(groups, with_bias, renorm, score):
    x = logits(6, 16, "f32", 8)
    x[1, 5] = math.nan
    x[2, 9] = math.inf
    x[3, 0] = math.nan
    x[3, 15] = math.inf
    x[4] = math.nan
    clean = x[[0, 5]].clone()
    bias = torch.zeros(16, device="cuda") if with_bias else None
    args = dict(bias=bias, score=score, groups=groups, topk_groups=min(2, groups), renorm=renorm)
    ids, w = tg.expert_route(x, 3, **args)
    assert bool(w[1:5].isnan().all()) and not bool(w[[0, 5]].isnan().any())
    assert bool(((ids >= 0) & (ids < 16)).all())
    assert all(len(set(r)) == 3 for r in ids.tolist())
    assert ids[1, 0] == 5 and ids[2, 0] == 9 and {0, 15} <= set(ids[3].tolist())
    ids2, w2 = tg.expert_route(clean, 3, **args)
    assert torch.equal(ids[[0, 5]], ids2) and torch.equal(w[[0, 5]], w2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype,scale", [("f32", 200.0), ("bf16", 3000.0), ("f16", 10000.0)])
def test_route_large_logits(dtype, scale, score):
    """Scores that vanish or saturate in 32 bits keep their order and their
    shares."""
    x = logits(40, 64, dtype, 2, scale=scale).clamp(-60000, 60000)
    rows = x.double().tolist()
    ids, w = tg.expert_route(x, 4, score=score)
    want = torch.tensor([choose(r, 4, score) for r in rows], dtype=torch.int32)
    assert torch.equal(ids.cpu(), want)
    ref = weights_of(x.cpu().double(), want, score, True, 1.0)
    close(w.cpu(), ref, ref * relative(x).cpu() + 2.0 ** -126)
    low = -x.abs() - 300
    ids, w = tg.expert_route(low, 4, score=score)
    want = torch.tensor([choose(r, 4, score) for r in low.double().tolist()], dtype=torch.int32)
    assert torch.equal(ids.cpu(), want)
    ref = weights_of(low.cpu().double(), want, score, True, 1.0)
    close(w.cpu(), ref, ref * relative(low).cpu() + 2.0 ** -126)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_route_layouts(dtype):
    """Any row pitch and element-aligned base; other layouts are copied."""
    x = logits(21, 40, dtype, 3)
    want = tg.expert_route(x, 4)
    for pitch in (41, 43, 48):
        y = logits(21, 40, dtype, 3, pitch=pitch)
        got = tg.expert_route(y, 4)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    flat = torch.zeros(21 * 40 + 1, dtype=DT[dtype], device="cuda")
    flat[1:] = x.flatten()
    z = flat[1:].view(21, 40)
    for y in (z, x.t().contiguous().t(), x[:, :].flip(0).flip(0), x.repeat_interleave(2, 1)[:, ::2]):
        got = tg.expert_route(y.detach().requires_grad_(True), 4)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        leaf = y.detach().requires_grad_(True)
        dx, = torch.autograd.grad(tg.expert_route(leaf, 4, renorm=False)[1].sum(), leaf)
        leaf2 = x.detach().requires_grad_(True)
        dx2, = torch.autograd.grad(tg.expert_route(leaf2, 4, renorm=False)[1].sum(), leaf2)
        assert torch.equal(dx, dx2)
    one = x[3:4].expand(5, 40)
    got = tg.expert_route(one, 4)
    assert torch.equal(got[0], want[0][3:4].expand(5, 4))


def test_route_empty():
    ids, w = tg.expert_route(torch.zeros(0, 8, device="cuda", requires_grad=True), 2)
    assert ids.shape == w.shape == (0, 2)
    w.sum().backward()


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_route_gradient_against_differences(score, renorm):
    """The gradient predicts how the weights of the same choices change."""
    x = logits(10, 24, "f32", 11)
    leaf = x.detach().requires_grad_(True)
    ids, w = tg.expert_route(leaf, 5, score=score, renorm=renorm, scale=1.5)
    g = torch.randn((10, 5), generator=torch.Generator().manual_seed(3)).cuda()
    dx, = torch.autograd.grad(w, leaf, g)
    step = torch.randn((10, 24), generator=torch.Generator().manual_seed(4)).double()
    h = 1e-4
    x64 = x.cpu().double()
    up = weights_of(x64 + h * step, ids.cpu(), score, renorm, 1.5)
    down = weights_of(x64 - h * step, ids.cpu(), score, renorm, 1.5)
    change = ((up - down) * g.cpu().double()).sum(1) / (2 * h)
    told = (dx.cpu().double() * step).sum(1)
    # the central difference is off by h^2 times a third derivative of the order of |step|^3 |g|
    assert bool(((change - told).abs() <= 1e-5 * (1 + change.abs())).all())


def test_route_feeds_sort_and_combine():
    """Logits' gradient through a whole mixture-of-experts layer, against the
    same layer in 64 bits with the choices that were made."""
    T, E, k, D, F = 96, 8, 2, 64, 48
    g = torch.Generator().manual_seed(7)
    x = (torch.randn((T, D), generator=g) / 2).bfloat16().cuda()
    wr = (torch.randn((D, E), generator=g) / 4).cuda().requires_grad_(True)
    w1 = (torch.randn((E, D, F), generator=g) / 8).bfloat16().cuda().requires_grad_(True)
    lg = x.float() @ wr
    lg.retain_grad()
    ids, w = tg.expert_route(lg, k)
    plan = tg.expert_sort(ids, E)
    y = tg.expert_combine(tg.expert_matmul(tg.expert_gather(x, plan), w1, plan), plan, w)
    dy = torch.randn((T, F), generator=g).bfloat16().cuda()
    y.backward(dy)
    lg64 = lg.detach().double().requires_grad_(True)
    w64 = weights_of(lg64.cpu(), ids.cpu(), "softmax", True, 1.0).cuda()
    rows = torch.einsum("td,tkdf->tkf", x.double(), w1.detach().double()[ids.long()])
    ref = (w64[..., None] * rows).sum(1)
    want, = torch.autograd.grad(ref, lg64, dy.double())
    # the products are rounded to bf16 (half a step, 2^-8) before the sum over F; the rest is 32 bits
    size = (rows.abs() * dy.double().abs()[:, None]).sum(2).amax(1, keepdim=True)
    close(lg.grad, want, size * 2 * 2.0 ** -8 * 1.01 + 1e-6)
    assert wr.grad is not None and w1.grad is not None


def test_layer_in_4_bits():
    """Routing, sort, quantisation into sorted rows, product, quantisation,
    product, combine: each step against its definition on the step's own inputs."""
    from mxfp4_util import product, quantised, random_blocks, values
    T, E, k, D, F = 150, 16, 4, 256, 544
    g = torch.Generator().manual_seed(1)
    x = torch.randn((T, D), generator=g).bfloat16().cuda()
    lg = torch.randn((T, E), generator=g).cuda()
    lg[::7] = -math.inf                                 # padding tokens
    (w1, s1), (w2, s2) = random_blocks((E, F, D), 2, 120, 124), random_blocks((E, D, F), 3, 120, 124)
    bias = torch.randn(E, generator=g).cuda() * 0.1
    ids, wt = tg.expert_route(lg, k, bias=bias, score="sigmoid", groups=4, topk_groups=2, scale=2.5)
    plan = tg.expert_sort(ids, E)
    q, s = tg.quant_mxfp4(x, plan)
    h = tg.gemm_grouped_mxfp4(q, s, plan, w1, s1, relu=True)
    q2, t2 = tg.quant_mxfp4(h)
    y = tg.gemm_grouped_mxfp4(q2, t2, plan, w2, s2)
    out = tg.expert_combine(y, plan, wt)
    src, cut = plan.src.long(), plan.offsets.tolist()
    qx, sx = quantised(x)
    token = (src // k).cpu()[:cut[-1]]
    assert torch.equal(q[:cut[-1]].cpu(), qx[token]) and torch.equal(s[:cut[-1]].cpu(), sx[token])
    qh, sh = quantised(h)
    assert torch.equal(q2.cpu(), qh) and torch.equal(t2.cpu(), sh)
    for e in range(E):
        part = slice(cut[e], cut[e + 1])
        for got, a, b, w, sw, relu in ((h, q, s, w1, s1, True), (y, q2, t2, w2, s2, False)):
            ref, bound = product(values(a[part], b[part]), values(w[e], sw[e]), torch.bfloat16)
            close(got[part], ref.clamp(min=0) if relu else ref, bound)
    want = torch.zeros(T, D, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)
    for j in range(k):
        live = (ids[:, j] >= 0)[:, None]
        rows = torch.where(live, y.double()[plan.pos[:, j].long()] * wt[:, j, None].double(), 0.0)
        want += rows
        size += rows.abs()
    close(out, want, want.abs() * 2.0 ** -8 * 1.01 + size * k * 2.0 ** -23 + 2.0 ** -134)
    assert bool((out[::7] == 0).all())
