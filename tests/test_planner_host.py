"""Refusals of the page planner that come before any GPU call."""


def test_a_free_stack_of_no_possible_size_is_refused():
    from spectral_transform_coding_b200 import lib
    one = 1 << 20  # (never followed)
    for capacity in (-1, 1 << 31):
        assert lib.spectra_plan_append_ex(one, 1, one, one, None, 0, one, capacity, one, one, one, 1, 1, one, one, one,
                                          one, None) == 1
    assert lib.spectra_plan_append_ex(None, 1, None, None, None, 0, None, 0, None, None, None, 1, 1, None, None, None,
                                      None, None) == 1
