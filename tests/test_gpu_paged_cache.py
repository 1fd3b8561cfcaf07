"""SfaPagedCache beyond one stream's plain steps: streams, refusals, other cache types, and a free
list that runs out."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

sfa = pytest.importorskip("indexer_selected_sparse_block_gb300")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    return torch.device("cuda:0")


def lens(dev, *n):
    return torch.tensor(n, dtype=torch.int32, device=dev)


def test_release_behind_a_step_on_another_stream(dev):
    """A step and a release on a stream that still has other work: the release sees the step's
    lengths and pages."""
    c = sfa.SfaPagedCache(n_seq=2, n_pages=12, page_size=4, max_pages=6, n_tok_cap=20, h_kv=1, dkq=64, dv=64)
    K, new = torch.ones((20, 1, 64), dtype=torch.bfloat16, device=dev), lens(dev, 9, 5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)          # about 10 ms
    c.step(new, K, stream=side)
    c.release(0, stream=side)
    torch.cuda.synchronize()
    assert c.length.tolist() == [0, 5]
    assert c.page_table.tolist() == [[-1] * 6, [3, 4, -1, -1, -1, -1]]
    assert int(c.free_head) == 2
    assert sorted(c.free_pages[2:].tolist()) == sorted(set(range(12)) - {3, 4})
    assert sfa.sfa_read_device_status(c.status) == 0
