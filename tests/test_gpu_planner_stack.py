"""A count of free pages that the stack's array does not hold: the plan is refused and nothing is written."""
import numpy as np
import pytest

from gpu_helpers import dev, torch_mod

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("count,refused", [(8, False), (9, True), (2 ** 31 - 1, True), (-1, True)])
@pytest.mark.parametrize("new", [[1, 0, 40], [0, 0, 0]])
def test_the_count_is_held_against_the_array(new, count, refused):
    torch = torch_mod()
    import spectral_transform_coding_b200 as st
    i32 = dict(dtype=torch.int32, device=dev())
    P, most = 32, 4
    room = torch.arange(100, 200, **i32)  # (the stack is its first eight entries)
    table, lengths = torch.full((3, most), -5, **i32), torch.tensor([0, 32, 7], **i32)
    n_free = torch.tensor([count], **i32)
    plan = st.AppendPlan(64, 3, device=dev())
    for t in (plan.seq_ids, plan.positions, plan.slots, plan.offsets):
        t.fill_(77)
    pl = st.PagePlanner(P, dev())
    pl.plan_append(table, lengths, torch.tensor(new, **i32), room[:8], n_free, plan=plan)
    if not refused:
        pl.status()
        pages = [p for p in table.flatten().tolist() if p != -5]
        assert pages == ([107, 106] if sum(new) else []) and n_free.item() == 8 - len(pages)
        return
    with pytest.raises(st.SpectraError) as e:
        pl.status()
    assert e.value.status == (3 if count < 0 else 1)
    assert n_free.item() == count and torch.all(table == -5)
    for t in (plan.seq_ids, plan.positions, plan.slots, plan.offsets):
        assert torch.all(t == 77)
