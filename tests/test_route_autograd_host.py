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
