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


@pytest.mark.parametrize("n_k", [0, 2])
def test_rows_left_out_are_copied_in_the_stream_of_the_call(n_k):
    """Inputs that an earlier kernel of the call's stream has yet to write."""
    torch = torch_mod()
    import spectral_transform_coding_b200 as st
    r = st.Rope()
    data = torch.randn((40, 3, 64), device=dev())
    x, k = torch.zeros_like(data), torch.zeros_like(data[:, :2]) if n_k else None
    pos = torch.arange(40, dtype=torch.int32, device=dev())
    pos[::3] = -1
    want, want_k = r.apply(pos, data, data[:, :2].contiguous() if n_k else None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # about 10 ms
        x.copy_(data)
        if n_k:
            k.copy_(data[:, :2])
    got, got_k = r.apply(pos, x, k, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    if n_k:
        assert torch.equal(got_k, want_k)
