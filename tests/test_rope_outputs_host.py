"""What autograd knows of the rotary call's outputs, as far as it needs no GPU."""
import pytest

torch = pytest.importorskip("torch")


class _Current:
    side = None


def _pair(x, out):
    from spectral_transform_coding_b200.serve import _pair
    return _pair("q", x, out, x.shape[0], x.shape[2], x, _Current())[2]


def test_a_fresh_output_is_a_copy_off_the_graph():
    x = torch.randn((3, 2, 8), requires_grad=True)
    y = _pair(x, None)
    assert not y.requires_grad and y.grad_fn is None and y.data_ptr() != x.data_ptr()
    assert torch.equal(y, x)
    wide = torch.randn((3, 4, 8)).requires_grad_()[:, :2]
    y = _pair(wide, None)
    assert not y.requires_grad and y.is_contiguous() and torch.equal(y, wide)


def test_outputs_that_need_a_gradient_are_refused_while_gradients_are_recorded():
    leaf = torch.randn((3, 2, 8), requires_grad=True)
    inner = leaf * 2
    for x, out in ((leaf, leaf), (inner, inner), (leaf.detach(), inner)):
        with pytest.raises(ValueError):
            _pair(x, out)
        with torch.no_grad():
            assert _pair(x, out) is out


def test_a_written_output_invalidates_what_a_graph_saved_of_it():
    w = torch.ones(8, requires_grad=True)
    x = torch.randn((3, 2, 8))
    loss = (x * w).sum()  # (its backward pass needs x)
    assert _pair(x, x) is x
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_inference_tensors_are_taken():
    with torch.inference_mode():
        x = torch.randn((3, 2, 8))
    assert _pair(x, x) is x
