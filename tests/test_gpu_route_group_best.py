"""A group's two best logits where a lane holds several that are nearly equal:
large ones, whose last bits weigh much in a score.  Choices against the definition
in 64 bits."""
import pytest
import torch

import tiled_dense_gemm_tma_b200 as tg
from route_util import choose

pytestmark = pytest.mark.gpu


def same(x, topk, groups, keep, score="softmax"):
    want = torch.tensor([choose(r, topk, score, None, groups, keep) for r in x.double().tolist()], dtype=torch.int32)
    ids, _ = tg.expert_route(x.cuda(), topk, score=score, groups=groups, topk_groups=keep)
    wrong = (ids.cpu() != want).any(1).nonzero().flatten().tolist()
    assert not wrong, [(t, ids[t].tolist(), want[t].tolist()) for t in wrong[:3]]
    return want


def test_the_best_two_of_three_neighbours():
    u = 2.0 ** -14                                     # of numbers from 512 to 1024
    x = torch.zeros(1, 128)
    x[0, [0, 1, 2]] = torch.tensor([1000.0, 1000.0, 1000.0 + 3 * u])
    x[0, [64, 68]] = torch.tensor([1000.0 + 4 * u, 1000.0 - 3 * u])
    # group 0 holds 3 units more than twice 1000, group 1 one
    assert same(x, 1, 2, 1).item() == 2


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("c", [1.0, 100.0, 1000.0, -5.0, -1000.0])
@pytest.mark.parametrize("E,groups", [(128, 2), (256, 8), (512, 16), (1024, 2), (1020, 17), (96, 3)])
def test_neighbours_in_every_group(E, groups, c, score):
    """Three or more logits a few units apart in one lane of each group; the other
    logits are far below."""
    per = E // groups
    lanes = 32
    while lanes * groups > 32:
        lanes //= 2
    V = 1 << (-(-per // lanes) - 1).bit_length()
    g = torch.Generator().manual_seed(E + groups)
    unit = torch.nextafter(torch.tensor(c), torch.tensor(2000.0)) - c
    T = 100
    x = torch.full((T, E), c - 30.0)
    for t in range(T):
        for gr in range(groups):
            lane = int(torch.randint(0, -(-per // V), (1,), generator=g))
            live = min(V, per - lane * V)
            n = min(live, 3 + t % 3)
            where = gr * per + lane * V + torch.randperm(live, generator=g)[:n]
            x[t, where] = c + unit * torch.randint(0, V, (n,), generator=g)
    if score == "sigmoid":                              # and among groups of one logit less
        x[T // 2:] = x[T // 2:].clamp(max=c + unit)
    for keep in {1, max(1, groups // 2)}:
        same(x, 2, groups, keep, score)
