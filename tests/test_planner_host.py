"""Refusals of the page planner that come before any GPU call."""
import pytest


def test_a_free_stack_of_no_possible_size_is_refused():
    from spectral_transform_coding_b200 import lib
    one = 1 << 20  # (never followed)
    for capacity in (-1, 1 << 31):
        assert lib.spectra_plan_append_ex(one, 1, one, one, None, 0, one, capacity, one, one, one, 1, 1, one, one, one,
                                          one, None) == 1
    assert lib.spectra_plan_append_ex(None, 1, None, None, None, 0, None, 0, None, None, None, 1, 1, None, None, None,
                                      None, None) == 1


@pytest.mark.parametrize("name", ["seq_ids", "positions", "slots", "offsets"])
def test_a_plan_keeps_tensors_of_its_own_size_type_and_device(name):
    torch = pytest.importorskip("torch")
    import spectral_transform_coding_b200 as st
    plan = st.AppendPlan(6, 3, device="cpu")
    old = getattr(plan, name)
    assert old.numel() == (4 if name == "offsets" else 6)
    assert old.dtype == (torch.int64 if name == "slots" else torch.int32)
    setattr(plan, name, torch.zeros(old.numel() + 1, dtype=old.dtype)[1:])
    kept = getattr(plan, name)
    assert kept is not old
    for bad in (old[:-1], torch.zeros(old.numel() + 1, dtype=old.dtype), old.float(),
                torch.zeros(2 * old.numel(), dtype=old.dtype)[::2], old.view(1, -1), old.to("meta")):
        with pytest.raises((TypeError, ValueError)):
            setattr(plan, name, bad)
        assert getattr(plan, name) is kept
    for size in ("max_tokens", "batch"):
        with pytest.raises(AttributeError):
            setattr(plan, size, 100)
