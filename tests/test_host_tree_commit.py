"""A draft is committed once, and a draft that is refused is none (stand-ins for tensors and the library;
nothing is launched)."""
import pytest
import torch

from indexer_selected_sparse_block_gb300 import pipeline
from test_host_devices import Far
from test_host_tree_streams import cache, i32, launches  # noqa: F401 (a fixture)


def test_a_draft_is_committed_once(launches):  # noqa: F811
    seen, _ = launches
    c = cache()
    for _ in range(2):
        c.draft(i32(2), i32(6), Far(6, 1, 64))
        with pytest.raises(ValueError):
            c.commit(Far(6, dtype=torch.int64), i32(6))     # refused: nothing was moved
        c.commit(i32(6), i32(6))
        n = len(seen)
        with pytest.raises(ValueError, match="committed"):
            c.commit(i32(6), i32(6))
        assert len(seen) == n


def test_captured_drafts_and_commits(launches, monkeypatch):  # noqa: F811
    """What is recorded does not run; behind a captured draft replays decide, which nobody here sees."""
    capturing = [False]
    monkeypatch.setattr(pipeline, "_capturing", lambda: capturing[0])
    c = cache()
    c.draft(i32(2), i32(6))
    capturing[0] = True
    c.commit(i32(6), i32(6))
    c.commit(i32(6), i32(6))
    capturing[0] = False
    c.commit(i32(6), i32(6))
    with pytest.raises(ValueError):
        c.commit(i32(6), i32(6))
    capturing[0] = True
    c.draft(i32(2), i32(6))
    capturing[0] = False
    for _ in range(3):
        c.commit(i32(6), i32(6))
    c.step(i32(2))
    with pytest.raises(ValueError):
        c.commit(i32(6), i32(6))


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
