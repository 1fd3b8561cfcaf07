"""On which device and stream the drafted-tree calls, the rotation and the cache's methods launch, and where
their workspace comes from (stand-ins for tensors and the library; nothing is launched)."""
import contextlib

import pytest
import torch

from indexer_selected_sparse_block_gb300 import SfaPagedCache
from indexer_selected_sparse_block_gb300 import _binding as B
from test_host_devices import Far, i32


class Rope:
    """What the calls ask of a rope, without the library that makes one."""
    n_rot = 64
    _rope = B._Rope()


@pytest.fixture
def launches(monkeypatch):
    current, seen, taken = [0], [], []

    @contextlib.contextmanager
    def on(dev):
        current.append(dev if isinstance(dev, int) else getattr(dev, "index", dev))
        yield
        current.pop()

    class Lib:
        def __getattr__(self, fn):
            def call(*args):
                seen.append((fn, current[-1], args[-1]))
                return 0
            call.__name__ = fn
            return call

    def empty(n, dtype=None, device=None):
        taken.append(current[-1])
        return Far(n, dtype=torch.uint8)

    monkeypatch.setattr(B, "lib", lambda: Lib())
    monkeypatch.setattr(B, "_tree_workspace", lambda *a: 4096)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "device", on)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 100 + d, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[-1] if isinstance(current[-1], int) else 0,
                        raising=False)
    return seen, taken


def cache():
    c = SfaPagedCache.__new__(SfaPagedCache)
    c.__dict__.update(n_seq=2, n_pages=8, page_size=4, dv=64, K=Far(32, 1, 64), V=None, X=Far(32, 64),
                      page_table=i32(2, 5), cell_of=None, free_pages=i32(8), free_head=i32(1), _head_out=i32(1),
                      length=i32(2), len_total=i32(2), cu_new=i32(3), q_seq=i32(6), q_pos=i32(6), slot=i32(6),
                      status=i32(1), tree_mask=i32(6, 1), cached_pos=i32(6), path=i32(2, 5), n_acc=i32(2),
                      next_token=i32(2), _parent=None)
    return c


@pytest.mark.parametrize("given", [False, True])
def test_a_draft_launches_on_its_own_device(launches, given):
    seen, taken = launches
    stream = type("Stream", (), dict(device_index=1, cuda_stream=77, index=1))() if given else None
    c = cache()
    c.draft(i32(2), i32(6), Far(6, 1, 64), X=Far(6, 64), rope=Rope(), Q=Far(6, 4, 64), stream=stream)
    c.attend_tree(Far(6, 4, 64), 5, 20, 0.1, Far(6, 4, 64, dtype=torch.float32), stream=stream)
    assert c.commit(i32(6), i32(6), stream=stream) is c.next_token
    assert [fn for fn, _, _ in seen] == ["sfa_build_page_maps", "sfa_build_tree_maps", "sfa_rotate_rows",
                                         "sfa_write_cells", "sfa_tree_attend_paged", "sfa_tree_accept",
                                         "sfa_tree_commit"]
    assert all(dev == 1 and st == (77 if given else 101) for _, dev, st in seen), seen
    # the workspace: of the call's stream, not the current one's
    assert taken == [1 if given else 0]
    c.step(i32(2), Far(6, 1, 64), stream=stream)           # drops the tree
    with pytest.raises(ValueError):
        c.commit(i32(6), i32(6))


def test_a_stream_of_another_device_is_refused(launches):
    other = type("Stream", (), dict(device_index=0, cuda_stream=5))()
    for call in (lambda: B.sfa_rotate_rows([(Far(6, 64), Far(6, 64), 0)], i32(6), Rope(), stream=other),
                 lambda: B.sfa_build_tree_maps(i32(6), i32(3), i32(2), i32(6, 1), i32(6), stream=other),
                 lambda: B.sfa_tree_accept(i32(6), i32(6), i32(6), i32(3), i32(2, 4), i32(2), i32(2), stream=other)):
        with pytest.raises(ValueError):
            call()
    assert launches[0] == []


def test_tensors_of_two_devices_are_refused(launches):
    from test_host_scratch import Fake
    near = Fake(6, 64)
    for rows in ([(near, Far(6, 64), 0)], [(Far(6, 64), near, 0)]):
        with pytest.raises(ValueError):
            B.sfa_rotate_rows(rows, i32(6), Rope())
    with pytest.raises(ValueError):
        B.sfa_tree_commit([near], i32(6), i32(3), i32(2, 4), i32(2), i32(2), 4, i32(2, 4), i32(8), i32(1), i32(2), i32(1))
    assert launches[0] == []
