"""On which device and stream a paged cache's step launches when its tensors are not on the current
device (stand-ins for tensors and the library; nothing is launched)."""
import contextlib

import pytest
import torch

from indexer_selected_sparse_block_gb300 import SfaPagedCache
from indexer_selected_sparse_block_gb300 import _binding as B
from test_host_scratch import Fake


class Far(Fake):
    """A contiguous tensor on device 1."""
    device = "cuda:1"

    def get_device(self):
        return 1

    def unsqueeze(self, _):
        return Far(1, *self.shape, dtype=self.dtype)

    def __getitem__(self, _):
        return Far(*self.shape[1:], dtype=self.dtype)


def i32(*s):
    return Far(*s, dtype=torch.int32)


@pytest.mark.parametrize("given", [False, True])
def test_step_launches_on_its_own_device(monkeypatch, given):
    current, launches = [0], []

    @contextlib.contextmanager
    def on(dev):
        current.append(dev if isinstance(dev, int) else dev.index)
        yield
        current.pop()

    class Lib:
        def __getattr__(self, fn):
            def call(*args):
                stream = args[-1]
                launches.append((fn, current[-1], getattr(stream, "value", stream)))
                return 0
            call.__name__ = fn
            return call

    monkeypatch.setattr(B, "lib", lambda: Lib())
    monkeypatch.setattr(torch.cuda, "device", on)
    main = type("Stream", (), dict(device_index=0, cuda_stream=100))()
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: main)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 100 + d, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[-1], raising=False)
    c = SfaPagedCache.__new__(SfaPagedCache)
    c.__dict__.update(n_seq=2, n_pages=8, page_size=4, dv=64, K=Far(32, 1, 64), V=None, X=None,
                      page_table=i32(2, 5), cell_of=None, free_pages=i32(8), free_head=i32(1), _head_out=i32(1),
                      length=i32(2), len_total=i32(2), cu_new=i32(3), q_seq=i32(6), q_pos=i32(6), slot=i32(6),
                      status=i32(1))
    stream = type("Stream", (), dict(device_index=1, cuda_stream=77))() if given else None
    c.step(i32(2), Far(6, 1, 64), stream=stream)
    assert [fn for fn, _, _ in launches] == ["sfa_build_page_maps", "sfa_write_cells", "sfa_copy_cache_rows_multi"]
    assert all(dev == 1 and st == (77 if given else 101) for _, dev, st in launches), launches
