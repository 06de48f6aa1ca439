"""What the choice of an eviction refuses beside tests/test_slots_refusals.py;
no GPU needed."""
import pytest

from tests.test_slots_refusals import FAKE, built, refused, slots   # noqa: F401 (built: a fixture)


@pytest.mark.parametrize("top", [(1 << 24) + 1, 1 << 30, 2 ** 31 - 1])
def test_more_moves_than_any_list_can_have(top):
    refused("plan_eviction", -1, top=top)
    refused("plan_eviction", -1, top=top, sl=slots(capacity=1 << 24), budget=100)


@pytest.mark.parametrize("where", [0, 4, -4])
@pytest.mark.parametrize("lengths", ["ctx_len", "seq_len"])
def test_lengths_out_over_the_lengths_in(lengths, where):
    """Other lists may not have read theirs yet when one writes."""
    far = {"ctx_len": FAKE + 4096, "seq_len": FAKE + 8192, "ctx_out": FAKE + 12288}
    refused("plan_eviction", -1, **{**far, "ctx_out": far[lengths] + where})
