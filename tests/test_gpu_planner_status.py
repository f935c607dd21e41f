"""The status of one stream while another is busy."""
import pytest

from gpu_helpers import dev, torch_mod

pytestmark = pytest.mark.gpu


def test_the_status_of_a_stream_does_not_wait_for_another():
    """Read and cleared in its own stream: on the default stream the clearing came when that one's work was done, after
    errors of later calls."""
    torch = torch_mod()
    import spectral_transform_coding_b200 as st
    i32 = dict(dtype=torch.int32, device=dev())
    pl = st.PagePlanner(32, dev())
    table, lengths, free = torch.zeros((1, 2), **i32), torch.tensor([-1], **i32), torch.zeros(4, **i32)
    n_free, new, side = torch.tensor([4], **i32), torch.tensor([1], **i32), torch.cuda.Stream()
    plan = st.AppendPlan(4, 1, device=dev())
    pl.plan_append(table, lengths, new, free, n_free, plan=plan, stream=side)  # (everything loaded before the clock runs)
    with pytest.raises(st.SpectraError):
        pl.status(stream=side)
    torch.cuda.synchronize()
    torch.cuda._sleep(1_000_000_000)  # about 500 ms of the default stream
    ended = torch.cuda.Event()
    ended.record()
    pl.plan_append(table, lengths, new, free, n_free, plan=plan, stream=side)
    with pytest.raises(st.SpectraError) as e:
        pl.status(stream=side)
    pl.status(stream=side)  # (cleared)
    assert e.value.status == 1
    assert not ended.query()
    torch.cuda.synchronize()


def test_the_codecs_status_does_not_either():
    torch = torch_mod()
    import spectral_transform_coding_b200 as st
    from test_gpu_shared_prefix import _codec
    codec = _codec("toy")["codec"]
    cache = st.LatentCache(codec, 1, 2, device=dev())
    cache.lengths.fill_(-1)
    q, out, side = torch.zeros((1, 4, 64), device=dev()), torch.zeros((1, 4, 64), device=dev()), torch.cuda.Stream()
    ws = torch.zeros(codec.decode_workspace_bytes(1, cache.capacity), dtype=torch.uint8, device=dev())
    for busy in (False, True):  # (the first call loads the kernel)
        torch.cuda.synchronize()
        if busy:
            torch.cuda._sleep(1_000_000_000)
        ended = torch.cuda.Event()
        ended.record()
        codec.decode_attend(cache, q, out=out, workspace=ws, stream=side)
        with pytest.raises(st.SpectraError) as e:
            codec.device_status(stream=side)
        codec.device_status(stream=side)
        assert e.value.status == 1
        assert not busy or not ended.query()
    torch.cuda.synchronize()
