"""Every variant of the prefix kernel that the dispatch can pick, at ordinary sizes, by its name in a profile."""
import re

import pytest

import test_gpu_shared_prefix as base
from gpu_helpers import torch_mod

pytestmark = pytest.mark.gpu

SHAPES = {
    **base.SHAPES,
    "g8all8": (256, 8, 2, 64, 64, 8, [[8] * 8, [8] * 8], 64),
    "all8": (256, 8, 2, 128, 128, 16, [[8] * 8, [8] * 8], 64),
    "threewide": (256, 8, 2, 128, 128, 16, [[4, 3, 3, 2, 2, 1, 1, 1], [4, 3, 2, 2, 2, 1, 1, 1]], 64),
}

# shape, batch -> group, rows of a block, warps, CTAs of an SM
CASES = [
    ("llama4x", 2, (16, 16, 16, 2)), ("toy", 3, (8, 16, 16, 2)),
    ("llama4x", 7, (16, 32, 16, 1)), ("llama4x", 8, (16, 32, 16, 1)), ("g8all8", 6, (8, 32, 16, 1)),
    ("qwen8x", 4, (16, 32, 8, 2)), ("toy", 8, (8, 32, 8, 2)),
    ("llama4x", 9, (16, 64, 16, 1)), ("llama4x", 13, (16, 64, 16, 1)), ("llama4x", 16, (16, 64, 16, 1)),
    ("g8all8", 12, (8, 64, 16, 1)),
    ("qwen8x", 9, (16, 64, 8, 2)), ("toy", 16, (8, 64, 8, 2)),
    ("llama4x", 17, (16, 128, 16, 1)), ("llama4x", 40, (16, 128, 16, 1)), ("toy", 33, (8, 128, 16, 1)),
    ("g8wide", 17, (8, 128, 16, 1)),
    # the operands of 128 (or 64) rows would leave less than two tiles of pages
    ("threewide", 33, (16, 64, 16, 1)), ("all8", 9, (16, 32, 16, 1)), ("all8", 33, (16, 32, 16, 1)),
]


@pytest.mark.parametrize("name,batch,variant", CASES)
def test_variant(monkeypatch, name, batch, variant):
    torch = torch_mod()
    monkeypatch.setattr(base, "SHAPES", SHAPES)
    own = [(41 * b + 3) % 100 if b % 5 != 4 else None for b in range(batch)]
    s, cache, table, prefix, lengths, q, out = base._case(name, 5, own, seed=batch, scale=1.0)
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as prof:
        again = s["codec"].decode_attend_shared(cache, q, prefix)
        torch.cuda.synchronize()
    assert torch.equal(again, out)
    seen = [re.search(r"prefix_kernel<(.*?)>", e.name) for e in prof.events()]
    seen = [tuple(int(x) for x in re.findall(r"\d+", re.sub(r"\(int\)", "", m.group(1)))) for m in seen if m]
    assert seen and set(seen) == {variant}


@pytest.mark.parametrize("name,page", [("toy", 0), ("toy", 3), ("toy", 9), ("llama4x", 4)])
def test_bounded_wait_with_128_rows_a_block(monkeypatch, name, page):
    """A page copy that never lands, where the keys are unpacked behind the softmax: the call reports a timeout, and the
    next calls with the same workspace give the exact result."""
    torch = torch_mod()
    import spectral_transform_coding_b200 as st
    s = base._codec(name, 14)
    cache, table, prefix, lengths = base._filled(s, 900, [5] * 33, 14)
    q, _ = base._queries(s, 33, 14)
    codec = s["codec"]
    ws = torch.zeros(codec.decode_shared_workspace_bytes(33), dtype=torch.uint8, device=q.device)
    out = codec.decode_attend_shared(cache, q, prefix, workspace=ws)
    codec.device_status()
    monkeypatch.setenv("SPECTRA_PREFIX_TEST_DROP_PAGE", str(page))
    monkeypatch.setenv("SPECTRA_DECODE_TEST_WAIT_NS", "2000000")
    codec.decode_attend_shared(cache, q, prefix, workspace=ws)
    with pytest.raises(st.SpectraError) as e:
        codec.device_status()
    assert e.value.status == 6
    monkeypatch.delenv("SPECTRA_PREFIX_TEST_DROP_PAGE")
    monkeypatch.delenv("SPECTRA_DECODE_TEST_WAIT_NS")
    for _ in range(2):
        got = codec.decode_attend_shared(cache, q, prefix, workspace=ws)
        codec.device_status()
        assert torch.equal(got, out)
