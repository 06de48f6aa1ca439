"""What the choice of an eviction refuses beside tests/test_slots_refusals.py;
no GPU needed."""
import pytest

from tests.test_slots_refusals import built, refused, slots   # noqa: F401 (built: a fixture)


@pytest.mark.parametrize("top", [(1 << 24) + 1, 1 << 30, 2 ** 31 - 1])
def test_more_moves_than_any_list_can_have(top):
    refused("plan_eviction", -1, top=top)
    refused("plan_eviction", -1, top=top, sl=slots(capacity=1 << 24), budget=100)
