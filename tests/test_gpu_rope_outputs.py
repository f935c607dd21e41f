"""Rotary positions into fresh outputs: what autograd and other streams see of them."""
import numpy as np
import pytest

from gpu_helpers import dev, torch_mod

pytestmark = pytest.mark.gpu


def test_fresh_outputs_are_not_on_the_inputs_graph():
    """The call is not recorded: outputs of inputs that need a gradient need none, instead of passing theirs through."""
    torch = torch_mod()
    import spectral_transform_coding_b200 as st
    r = st.Rope()
    pos = torch.arange(6, dtype=torch.int32, device=dev()) * 5
    q, k = (torch.randn((6, h, 64), device=dev(), requires_grad=True) for h in (4, 2))
    want = r.apply(pos, q.detach(), k.detach())
    for x, y, z in zip((q, k), r.apply(pos, q, k), want):
        assert not y.requires_grad and y.grad_fn is None
        assert torch.equal(y, z)
