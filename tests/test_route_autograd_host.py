"""expert_route in autograd's other ways, on the host: forward mode is refused, as by
the other experts' operators."""
import pytest
import torch
import torch.autograd.forward_ad as fw

from test_mxfp4_host import fake  # noqa: F401  (a library on host memory)
from tiled_dense_gemm_tma_b200 import binding


def test_forward_mode_is_refused(fake):
    x = torch.randn((5, 8), generator=torch.Generator().manual_seed(1))
    plain = binding.expert_route(x, 2)
    with fw.dual_level():
        dual = fw.make_dual(x, torch.ones_like(x))
        with pytest.raises((RuntimeError, NotImplementedError), match="jvp"):
            binding.expert_route(dual, 2)
        with torch.no_grad(), pytest.raises((RuntimeError, NotImplementedError), match="jvp"):
            binding.expert_route(dual, 2)
        ids, w = binding.expert_route(x, 2)             # no tangent: nothing is lost
        assert torch.equal(ids, plain[0]) and torch.equal(w, plain[1])
    ids, w = binding.expert_route(x, 2)
    assert torch.equal(ids, plain[0]) and not w.requires_grad


def test_forward_mode_of_a_function_is_refused(fake):
    x = torch.randn((5, 8), generator=torch.Generator().manual_seed(1))
    with pytest.raises((RuntimeError, NotImplementedError)):
        torch.func.jvp(lambda v: binding.expert_route(v, 2)[1], (x,), (torch.ones_like(x),))


@pytest.mark.parametrize("renorm", [True, False])
def test_saved_tensors_in_another_layout(fake, renorm):
    """What a saved-tensor hook gives back is read in the layout that it has."""
    def column_major(t):
        return t.t().contiguous().t()

    def wide(t):
        big = torch.full((t.shape[0], t.shape[1] + 3), -7, dtype=t.dtype)
        big[:, :t.shape[1]] = t
        return big[:, :t.shape[1]]

    base = torch.randn((6, 8), generator=torch.Generator().manual_seed(2))
    g = torch.randn((6, 3), generator=torch.Generator().manual_seed(3))
    leaf = base.clone().requires_grad_(True)
    want, = torch.autograd.grad(binding.expert_route(leaf, 3, renorm=renorm)[1], leaf, g)
    for other in (column_major, wide):
        leaf = base.clone().requires_grad_(True)
        with torch.autograd.graph.saved_tensors_hooks(lambda t: t.detach().clone(), other):
            w = binding.expert_route(leaf, 3, renorm=renorm)[1]
        dx, = torch.autograd.grad(w, leaf, g)
        assert torch.equal(dx, want), other.__name__
