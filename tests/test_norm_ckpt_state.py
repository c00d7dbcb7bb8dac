"""Host-side checks of the norm and checkpoint calls' bookkeeping (CPU)."""

import pytest

import __graft_entry__


@pytest.fixture(scope="module")
def clp():
    __graft_entry__.build()
    import chunked_log_prob_gb300 as m

    return m


def test_lose_copy_refuses_what_is_no_index(clp):
    for bad in (-2, 1 << 30, 1 << 40):
        with pytest.raises(clp.GrpoError) as e:
            clp.grpo_selftest_lose_copy(bad)
        assert e.value.code == -1
    clp.grpo_selftest_lose_copy(5)
    clp.grpo_selftest_lose_copy(-1)  # takes it back
