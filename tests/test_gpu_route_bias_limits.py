"""The router's bias at its limits: minus infinity switches an expert off, the
lowest finite value puts it last."""
import math

import pytest
import torch

import tiled_dense_gemm_tma_b200 as tg
from expert_util import close
from route_util import choose, relative, scores, weights_of

pytestmark = pytest.mark.gpu

LOWEST = torch.finfo(torch.float32).min


def definition(x, topk, score, bias, groups, keep):
    """choose, with experts of a bias of minus infinity as good as masked for the
    choice (their scores are still part of a softmax)."""
    p = scores(x, score)
    E, per = len(x), len(x) // groups
    key = [a + b for a, b in zip(p, bias)]
    live = [v > -math.inf and b > -math.inf for v, b in zip(x, bias)]
    if groups > 1:
        rank = []
        for g in range(groups):
            best = sorted((key[e] for e in range(g * per, g * per + per) if live[e]), reverse=True)[:2]
            rank.append((-sum(best) if best else math.inf, g))
        kept = {g for _, g in sorted(rank)[:keep]}
        live = [v and e // per in kept for e, v in enumerate(live)]
    order = sorted((e for e in range(E) if live[e]), key=lambda e: (-key[e], e))[:topk]
    return order + [-1] * (topk - len(order))


def run(x, topk, bias, score, groups, keep, renorm):
    leaf = x.cuda().requires_grad_(True)
    ids, w = tg.expert_route(leaf, topk, bias=bias.cuda(), score=score, groups=groups, topk_groups=keep, renorm=renorm)
    b = bias.double().tolist()
    want = torch.tensor([definition(r, topk, score, b, groups, keep) for r in x.double().tolist()], dtype=torch.int32)
    assert torch.equal(ids.cpu(), want)
    ref = weights_of(x.double(), want, score, renorm, 1.0)
    close(w.detach().cpu(), ref, ref * relative(x) + 2.0 ** -126, "weights")
    assert bool((w[ids < 0] == 0).all())
    dx, = torch.autograd.grad(w.sum(), leaf)
    assert bool(torch.isfinite(dx).all())
    return want


def logits(T, E, dtype, seed):
    return (torch.randn((T, E), generator=torch.Generator().manual_seed(seed)) * 1.5).to(dtype)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,groups,keep,topk", [(8, 1, 1, 4), (64, 1, 1, 6), (60, 4, 2, 8), (256, 8, 4, 8), (1024, 2, 1, 5),
                                                (32, 32, 6, 6), (999, 27, 5, 12)])
def test_minus_infinity_switches_off(E, groups, keep, topk, dtype, score, renorm):
    g = torch.Generator().manual_seed(E)
    x = logits(20, E, dtype, E)
    some = torch.randn(E, generator=g) * 0.02
    off = torch.rand(E, generator=g) < 0.5
    per = E // groups
    few = torch.ones(E, dtype=torch.bool)               # all off but two, of which one is masked in some rows
    few[[1, E - 1]] = False
    x[::3, 1] = -math.inf
    whole = torch.arange(E) // per % 2 == 0             # every other group (or expert) off
    if groups == 1:
        whole = torch.arange(E) % 2 == 0
    for gone in (off, few, whole, torch.ones(E, dtype=torch.bool)):
        run(x, topk, torch.where(gone, -math.inf, some), score, groups, keep, renorm)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_minus_infinity_among_near_ties(score):
    """Rows that are decided in 64 bits."""
    x = torch.zeros(4, 64)
    x[1] = 20.0
    x[2, ::2] = 2.0 ** -24
    x[3, ::3] = 20.0
    x[3, 1::3] = 20.125
    bias = torch.zeros(64)
    bias[::4] = -math.inf
    for groups, keep in ((1, 1), (8, 3)):
        run(x, 6, bias, score, groups, keep, True)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_a_bad_logit_and_a_bias_of_minus_infinity(score):
    x = logits(3, 16, torch.float32, 1)
    x[0, 3] = math.nan
    x[1, 3] = math.inf
    bias = torch.zeros(16)
    bias[[3, 4, 5]] = -math.inf
    for groups, keep in ((1, 1), (4, 2)):
        ids, w = tg.expert_route(x.cuda(), 4, bias=bias.cuda(), score=score, groups=groups, topk_groups=keep)
        assert bool(w[:2].isnan().all()) and not bool(w[2].isnan().any())
        assert not ((ids >= 3) & (ids <= 5)).any() and bool((ids < 16).all())


@pytest.mark.parametrize("low", [LOWEST, LOWEST / 2, -1e30])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,keep,topk", [(16, 1, 1, 8), (16, 4, 3, 10), (64, 8, 4, 20), (256, 8, 8, 32), (32, 32, 9, 9)])
def test_the_lowest_value_comes_last(E, groups, keep, topk, score, low):
    """A finite bias excludes nobody: its experts, and groups that hold no others,
    are there when the rest is used up."""
    x = logits(12, E, torch.float32, E)
    x[3, E // 2:] = -math.inf
    per = E // groups
    bias = torch.zeros(E)
    bias[torch.arange(E) // per != groups // 2] = low
    if groups == 1:
        bias[4:] = low
    want = run(x, topk, bias, score, groups, keep, True)
    assert choose(x[0].double().tolist(), topk, score, bias.double().tolist(), groups, keep) == want[0].tolist()
