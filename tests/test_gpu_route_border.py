"""Choices of the router where exact ties and near ties meet: at the border
between the last choice and the first expert left out.  Every row against the definition in 64 bits."""
import pytest
import torch

import tiled_dense_gemm_tma_b200 as tg
from route_util import choose

pytestmark = pytest.mark.gpu


def same(x, topk, bias=None, score="softmax", groups=1, keep=1):
    """The kernel's choices for x (on the host) are the definition's."""
    b = None if bias is None else bias.double().tolist()
    want = torch.tensor([choose(r, topk, score, b, groups, keep) for r in x.double().tolist()], dtype=torch.int32)
    ids, _ = tg.expert_route(x.cuda(), topk, bias=None if bias is None else bias.cuda(), score=score, groups=groups,
                             topk_groups=keep)
    wrong = (ids.cpu() != want).any(1).nonzero().flatten().tolist()
    assert not wrong, [(t, ids[t].tolist(), want[t].tolist()) for t in wrong[:3]]
    return want


def row(E, rest, **at):
    x = torch.full((1, E), rest)
    for e, v in at.items():
        x[0, int(e[1:])] = v
    return x


def test_a_tie_at_the_border_hides_nothing():
    u = 2.0 ** -23
    assert same(row(64, -1.0, e0=1.0, e2=1.0, e4=1.0 + u), 1).item() == 4
    assert same(row(128, -5.0, e0=1.0, e4=1.0, e8=1.0 + u), 1).item() == 8
    v = 0.5
    x = row(256, -1.0, e100=2.0, e0=v, e8=v, e16=v + 5 * 2.0 ** -24)
    assert same(x, 2).tolist() == [[100, 16]]
    # the same expert further down in the tied one's own lane, and in the last lane
    assert same(row(256, -1.0, e8=v, e9=v, e10=v + 2 * 2.0 ** -24), 1).item() == 10
    assert same(row(256, -1.0, e8=v, e16=v, e255=v + 2 * 2.0 ** -24), 1).item() == 255
    # with a bias: saturated sigmoids of 16-bit logits
    zero = torch.zeros(64)
    assert same(row(64, -1.0, e0=20.0, e4=20.0, e8=20.125).bfloat16(), 1, bias=zero, score="sigmoid").item() == 8
    assert same(row(32, -1.0, e0=20.0, e4=20.0, e8=20.125).bfloat16(), 1, bias=zero[:32], score="sigmoid").item() == 8


@pytest.mark.parametrize("c", [0.5, 1.0, -3.0, 1000.0])
@pytest.mark.parametrize("E", [64, 100, 128, 256, 512, 1024])
def test_ties_among_neighbours(E, c):
    """Runs of logits that are equal or differ by fewer units than a lane numbers
    experts, across the border and behind it, in one lane and in several."""
    V = -(-E // 32)
    V = 1 << (V - 1).bit_length()
    g = torch.Generator().manual_seed(E)
    T = 160
    x = torch.randn((T, E), generator=g) * 0.3 + c - 3
    unit = torch.nextafter(torch.tensor(c), torch.tensor(2000.0)) - c
    for t in range(T):
        n = 3 + t % 9
        where = torch.randperm(E, generator=g)[:n] if t % 2 else (t * 7) % (E - n) + torch.randperm(n, generator=g)
        step = torch.randint(0, V, (n,), generator=g) * (torch.rand(n, generator=g) < 0.5)
        x[t, where] = c + step * unit
        if t % 3 == 0:
            x[t, (where[0] + E // 2) % E] = c + 1
    for topk in (1, 2, 4):
        same(x, topk)


@pytest.mark.parametrize("dtype,score,lo,step", [("f32", "sigmoid", 12.0, 0.5), ("bf16", "sigmoid", 16.0, 0.125),
                                                 ("f16", "sigmoid", 9.0, 2.0 ** -7), ("f32", "softmax", -12.0, 0.25),
                                                 ("bf16", "softmax", -12.0, 0.0625), ("f32", "sigmoid", -16.0, 0.5)])
@pytest.mark.parametrize("E,groups,keep", [(24, 1, 1), (64, 1, 1), (256, 1, 1), (1024, 1, 1), (256, 8, 3), (1020, 17, 4)])
def test_ties_among_neighbours_with_a_bias(E, groups, keep, dtype, score, lo, step):
    """Scores that differ by less than the keys hold, under biases that are equal,
    or equal in steps: saturated sigmoids, and scores that are small beside what
    they are added to."""
    g = torch.Generator().manual_seed(E + groups)
    T = 60
    x = lo + step * torch.randint(0, 3, (T, E), generator=g)
    x = torch.where(torch.rand((T, E), generator=g) < 0.8, lo - 4.0 - torch.rand((T, E), generator=g), x)
    if score == "softmax":
        x[:, -1] = 0.0
    x = x.to({"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dtype])
    for bias in (torch.zeros(E), torch.full((E,), 7.0), (torch.arange(E) % 5 > 3).float() * 0.25):
        for topk in (1, 3):
            same(x, topk, bias=bias, score=score, groups=groups, keep=keep)
