"""A draft that is refused is none (stand-ins for tensors and the library; nothing is launched)."""
import pytest
from test_host_devices import Far
from test_host_tree_streams import cache, i32, launches  # noqa: F401 (a fixture)


def test_a_refused_draft_drops_the_one_before(launches):  # noqa: F811
    """Its nodes may have their cells already: the tree before has none any more."""
    seen, _ = launches
    c = cache()
    c.draft(i32(2), i32(6))
    with pytest.raises(ValueError):
        c.draft(i32(2), i32(6), V=Far(6, 1, 64))            # before anything is launched
    c.commit(i32(6), i32(6))
    c.draft(i32(2), i32(6))
    with pytest.raises(ValueError):
        c.draft(i32(2), i32(5))                             # parents too few: behind the page maps
    assert seen[-1][0] == "sfa_build_page_maps"
    with pytest.raises(ValueError):
        c.commit(i32(6), i32(6))
