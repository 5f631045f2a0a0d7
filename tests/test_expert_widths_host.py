"""The differentiable experts' operators on operands whose rows do not start on
16-byte boundaries, through the binding with stand-ins of the entry points that
refuse what the library refuses."""
import pytest
import torch

from test_expert_host import IDS, Fake, bf, near, plan_of
from tiled_dense_gemm_tma_b200 import binding


class Strict(Fake):
    """The stand-ins behind the library's checks of pointers, pitches and planes."""
    ROWS = {"tg_gemm_grouped_bf16": ((4, 5, 2), (7, 8, 2), (11, 12, 2)), "tg_expert_gather": ((4, 5, 0), (9, 10, 0)),
            "tg_gemm_grouped_wgrad_bf16": ((4, 5, 2), (6, 7, 2), (9, 10, 2)),
            "tg_expert_combine": ((4, 5, 2), (9, 10, 2)), "tg_expert_combine_grad": ((4, 5, 2), (6, 7, 2), (11, 12, 2))}
    PLANES = {"tg_gemm_grouped_bf16": (3, 9), "tg_gemm_grouped_wgrad_bf16": (3, 11)}

    def launch(self, name, device, stream, *args):
        for p, ld, eb in self.ROWS[name]:
            eb = eb or args[3]                            # gather: bytes of an element
            assert args[p] % 16 == 0 and args[ld] * eb % 16 == 0, (name, args)
        if name in self.PLANES:
            e, at = self.PLANES[name]
            assert args[e] == 1 or (args[at] > 0 and args[at] % 8 == 0), (name, args)
        return getattr(self, name)(*args, stream)


@pytest.fixture
def strict(monkeypatch):
    monkeypatch.setattr(binding, "_launch", Strict().launch)
    monkeypatch.setattr(binding, "_require_cuda", lambda device, *named: None)


def off(t):
    """The same values, rows one element past a boundary and oddly pitched."""
    shape = t.shape[:-1] + (t.shape[-1] + 1,)
    out = torch.zeros(shape, dtype=t.dtype)[..., 1:]
    return out.copy_(t)


MAKE = {"dense": lambda t: t.detach().contiguous(), "off": off,
        "columns": lambda t: t.detach().transpose(-1, -2).contiguous().transpose(-1, -2)}


@pytest.mark.parametrize("rows", MAKE)
@pytest.mark.parametrize("weights", MAKE)
@pytest.mark.parametrize("K,N", [(11, 13), (16, 11), (1, 8), (13, 1), (8, 16)])
def test_product(strict, rows, weights, K, N):
    plan = plan_of(IDS, 3)
    X = MAKE[rows](bf((10, K), 1)).requires_grad_(True)
    W = MAKE[weights](bf((3, K, N), 2)).requires_grad_(True)
    g = MAKE[rows](bf((10, N), 3))
    Y = binding.expert_matmul(X, W, plan)
    got = torch.autograd.grad(Y, (X, W), g)
    o = plan.offsets.tolist()
    x, w = X.detach().double().requires_grad_(True), W.detach().double().requires_grad_(True)
    parts = [x[o[e]:o[e + 1]] @ w[e] for e in range(3)]
    ref = torch.cat(parts + [torch.zeros(10 - o[3], N, dtype=torch.float64)])
    want = torch.autograd.grad(ref, (x, w), g.double())
    for a, b in zip((Y.detach(), *got), (ref.detach(), *want)):
        near(a, b, 1)


@pytest.mark.parametrize("rows", MAKE)
@pytest.mark.parametrize("H", [1, 9, 16])
def test_moves(strict, rows, H):
    plan = plan_of(IDS, 3)
    make = MAKE[rows]
    pitched, Yp = bf((5, H), 1, 24), bf((10, H), 2, 24)
    X, Y = make(pitched).requires_grad_(True), make(Yp).requires_grad_(True)
    w = torch.rand(5, 2, generator=torch.Generator().manual_seed(3)).requires_grad_(True)
    Xs, out = binding.expert_gather(X, plan), binding.expert_combine(Y, plan, w)
    assert torch.equal(Xs.detach(), binding.expert_gather(pitched, plan))
    assert torch.equal(out.detach(), binding.expert_combine(Yp, plan, w.detach()))
    dX, = torch.autograd.grad(Xs, X, make(bf((10, H), 4)))
    dY, dw = torch.autograd.grad(out, (Y, w), make(bf((5, H), 5)))
    p, q = pitched.detach().requires_grad_(True), Yp.detach().requires_grad_(True)
    rX, = torch.autograd.grad(binding.expert_gather(p, plan), p, bf((10, H), 4, 24))
    rY, rw = torch.autograd.grad(binding.expert_combine(q, plan, w), (q, w), bf((5, H), 5, 24))
    assert torch.equal(dX, rX) and torch.equal(dY, rY) and torch.equal(dw, rw)
    q8 = torch.randint(-128, 128, (5, H), dtype=torch.int8)
    s = torch.rand(5)
    a = binding.expert_gather(make(q8), plan, scales=s)
    n = int(plan.offsets[-1])
    assert torch.equal(a[0][:n], q8[(plan.src[:n] // 2).long()]) and torch.equal(a[1][:n], s[(plan.src[:n] // 2).long()])


def test_aligned_operands_are_not_copied(strict, monkeypatch):
    """Rows on 16-byte boundaries reach the kernels where they are."""
    def refuse(*a):
        raise AssertionError("copied")
    monkeypatch.setattr(binding, "_pitched_copy3", refuse)
    X, W = bf((10, 13), 1, 16), bf((3, 13, 11), 2, 16)
    assert binding._aligned_rows(X) is X and binding._aligned3(W) is W
    plan = plan_of(IDS, 3)
    binding.expert_matmul(X, W, plan)
    binding.expert_matmul(X, bf((3, 11, 13), 3, 16).transpose(1, 2), plan)
