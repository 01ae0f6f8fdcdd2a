"""Groups of no sequences on the CPU: whatever their prefix_lens hold, nothing is flagged and the others are as they are."""
import pytest

from tests.test_paged_groups_host import Call, host  # noqa: F401


@pytest.mark.parametrize("stale", [0, 900, 1 << 30, -7])
def test_prefix_of_a_group_of_none(host, stale):  # noqa: F811
    groups, prefix, lens, cu = [0, 0, 2, 2, 3, 3], [stale, 40, stale, 7, stale], [60, 50, 9], [0, 5, 7, 9]
    call = Call(host, lens, cu, groups, prefix, 4, 16, 8, most=64)
    plain = Call(host, lens, cu, [0, 2, 3], [40, 7], 4, 16, 8, most=64)
    rows = lambda c: sorted((it["s"], it["own"], it["row0"], it["rows"], it["lo"], it["hi"], it["ends"][: it["rows"]])  # noqa: E731
                            for it in map(c.item, range(c.slots)) if it["rows"] > 0)
    assert all(call.item(i)["ok"] for i in range(call.slots))
    assert rows(call) == rows(plain)
