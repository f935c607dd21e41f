"""One workspace for steps of different batch sizes: the largest batch's, zeroed once."""
import numpy as np
import pytest

from gpu_helpers import dev, torch_mod
from test_gpu_shared_prefix import _codec, _filled, _queries

pytestmark = pytest.mark.gpu

ORDERS = [(64, 3, 64), (1, 40, 2, 40, 64, 5, 1), (17, 16, 17)]


def _steps(s, batches):
    """Cache, prefix and queries of each batch."""
    out = {}
    for b in set(batches):
        cache, _, prefix, _ = _filled(s, 3, [(29 * i) % 90 for i in range(b)], seed=b)
        out[b] = (cache, prefix, _queries(s, b, b)[0])
    return out


@pytest.mark.parametrize("batches", ORDERS)
@pytest.mark.parametrize("name", ["toy", "llama4x"])
def test_shared_decode(name, batches):
    torch = torch_mod()
    s = _codec(name, 1)
    codec, steps = s["codec"], _steps(s, batches)
    ws = torch.zeros(max(codec.decode_shared_workspace_bytes(b) for b in batches), dtype=torch.uint8, device=dev())
    for b in batches:
        cache, prefix, q = steps[b]
        out = torch.full_like(q, float("nan"))
        codec.decode_attend_shared(cache, q, prefix, out=out, workspace=ws)
        codec.device_status()
        assert torch.equal(out, codec.decode_attend_shared(cache, q, prefix)), b


@pytest.mark.parametrize("batches", ORDERS)
@pytest.mark.parametrize("name", ["toy", "llama4x"])
def test_decode(name, batches):
    torch = torch_mod()
    s = _codec(name, 2)
    codec, steps = s["codec"], _steps(s, batches)
    ws = torch.zeros(max(codec.decode_workspace_bytes(b, steps[b][0].capacity) for b in batches), dtype=torch.uint8,
                     device=dev())
    for b in batches:
        cache, _, q = steps[b]
        q = q.float()
        out = torch.full_like(q, float("nan"))
        codec.decode_attend(cache, q, out=out, workspace=ws)
        codec.device_status()
        assert torch.equal(out, codec.decode_attend(cache, q)), b


def test_a_workspace_for_both_decodes():
    torch = torch_mod()
    s = _codec("llama4x", 3)
    codec, steps = s["codec"], _steps(s, (12, 5))
    ws = torch.zeros(max(max(codec.decode_shared_workspace_bytes(b), codec.decode_workspace_bytes(b, c.capacity))
                         for b, (c, _, _) in steps.items()), dtype=torch.uint8, device=dev())
    for b in (12, 5, 12):
        cache, prefix, q = steps[b]
        for call in (lambda w: codec.decode_attend_shared(cache, q, prefix, workspace=w),  # noqa: B023
                     lambda w: codec.decode_attend(cache, q.float(), workspace=w)):
            got, want = call(ws), call(None)
            codec.device_status()
            assert torch.equal(got, want)


def test_static_scratch():
    import ctypes

    from spectral_transform_coding_b200._lib import lib
    torch = torch_mod()
    s = _codec("llama4x", 4)
    codec, steps = s["codec"], _steps(s, (64, 3))
    lib.spectra_decode_attend_noalloc.argtypes = [ctypes.c_void_p] * 5
    for b in (64, 3, 64, 3):
        cache, _, q = steps[b]
        q = q.float()
        out = torch.full_like(q, float("nan"))
        desc = cache.desc()
        status = lib.spectra_decode_attend_noalloc(codec._h, ctypes.byref(desc), q.data_ptr(), out.data_ptr(),
                                                   torch.cuda.current_stream().cuda_stream)
        if status == 3 and b == 64:
            continue  # (more records than the static area holds)
        assert status == 0
        codec.device_status()
        assert torch.equal(out, codec.decode_attend(cache, q)), b
