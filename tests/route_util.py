"""Routing in 64 bits, one row at a time, and the bounds of the 32-bit weights
and gradients."""
import math

import torch

H32 = 2.0 ** -24


def scores(x, score):
    """Scores of a row of 64-bit logits without NaN or plus infinity; 0 for
    minus infinity."""
    if score == "sigmoid":
        return [1 / (1 + math.exp(-v)) if v > -700 else 0.0 for v in x]
    top = max(x)
    if top == -math.inf:
        return [0.0] * len(x)
    e = [math.exp(v - top) for v in x]
    total = math.fsum(e)
    return [v / total for v in e]


def choose(x, topk, score, bias=None, groups=1, keep=1):
    """The choices of a row (Python floats), -1 where none is left."""
    E, per = len(x), len(x) // groups
    p = scores(x, score)
    key = list(x) if bias is None else [a + b for a, b in zip(p, bias)]
    biased = p if bias is None else key
    live = [v > -math.inf for v in x]
    if groups > 1:
        rank = []
        for g in range(groups):
            best = sorted((biased[e] for e in range(g * per, g * per + per) if live[e]), reverse=True)[:2]
            rank.append((-sum(best) if best else math.inf, g))
        kept = {g for _, g in sorted(rank)[:keep]}
        live = [v and e // per in kept for e, v in enumerate(live)]
    order = sorted((e for e in range(E) if live[e]), key=lambda e: (-key[e], e))[:topk]
    return order + [-1] * (topk - len(order))


def weights_of(logits, ids, score, renorm, scale):
    """Weights of given choices, differentiable, in 64 bits."""
    gone = ids < 0
    dead = torch.isneginf(logits).all(1, keepdim=True)
    safe = torch.where(dead, torch.zeros_like(logits), logits)
    if score == "softmax":
        logp = torch.log_softmax(safe, 1)
    else:
        logp = torch.nn.functional.logsigmoid(safe)
    l = logp.gather(1, ids.clamp(min=0).long()).masked_fill(gone, -math.inf)
    if renorm:
        none = gone.all(1, keepdim=True)
        w = torch.softmax(torch.where(none, torch.zeros_like(l), l), 1)
        w = torch.where(gone, torch.zeros_like(w), w)
    else:
        w = torch.where(gone, torch.zeros_like(l), torch.exp(l))
    return w * scale


def relative(logits):
    """Relative error that a weight of each row may have.  A difference of
    logits (or a logarithm of a sigmoid) is off by 2^-24 of the largest
    magnitude that entered it, twice in a quotient; the exponential by 2 units in
    the last place, 4 * 2^-24; a sum of E terms in 32 lanes by (E / 32 + 5) *
    2^-24; logarithm, quotient and products by 2 * 2^-24 each."""
    x = logits.double()
    x = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    spread = x.abs().amax(1, keepdim=True)
    return H32 * (8 * spread + 40 + logits.shape[1] / 32)
