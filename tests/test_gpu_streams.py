"""Paged calls on several streams at once, with the workspaces they make for themselves."""
import pytest
import torch

from test_gpu_chunk import DEALT, N128, WIDE, Case

pytestmark = pytest.mark.gpu

sfa = pytest.importorskip("indexer_selected_sparse_block_gb300")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    return torch.device("cuda:0")


def test_own_workspaces_of_overlapping_calls(dev):
    """Calls without a workspace on the current stream and on two others, none of which waits for
    another: each gives what it gives alone."""
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
    runs = []
    for i, (shape, lens) in enumerate(((WIDE, [(4000, 1), (2500, 1)]), (N128, DEALT), (WIDE, [(3500, 2), (37, 1)]))):
        c = Case(dev, lens, 32, shape, seed=i)
        assert c.call() == 0
        n = c.cu[-1]
        need = sfa.sfa_chunk_attend_workspace_bytes(sfa.SFA_BF16, len(lens), n, c.h_q, c.h_kv, c.dkq, c.dv, c.sep,
                                                    max(k for _, k in lens), max(c.total))
        assert need > 0
        runs.append((c, c.Q.to(dev), i32(c.table), i32(c.cu), i32(c.total), torch.empty_like(c.O), torch.empty_like(c.lse)))
    torch.cuda.synchronize()
    streams = [None, torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(30):
        for (c, Q, table, cu, total, O, lse), st in zip(runs, streams):
            sfa.sfa_chunk_attend_paged(Q, c.Kc, c.Vc, table, 32, cu, total, max(k for _, k in c.lens), max(c.total), c.scale,
                                       O, lse=lse, stream=st)
    torch.cuda.synchronize()
    for c, _, _, _, _, O, lse in runs:
        n = c.cu[-1]
        assert torch.equal(O[:n], c.O[:n]) and torch.equal(lse[:n], c.lse[:n])


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_outputs_in_host_memory(dev, out):
    """O and lse in page-locked host memory, of whole and cut lists and of lists whose sums are set
    aside on the way: what the call gives on the device."""
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
    for shape, lens in ((WIDE, [(4000, 1), (70, 9)]), (N128, DEALT), (N128, [(5000, 1)] * 40), (WIDE, [(4000, 2)] * 80)):
        c = Case(dev, lens, 32, shape, out=out, seed=len(lens))
        assert c.call() == 0
        O, lse = torch.full(c.O.shape, 7.0, dtype=c.O.dtype).pin_memory(), torch.full(c.lse.shape, 7.0).pin_memory()
        Q = c.Q.to(dev)
        sfa.sfa_chunk_attend_paged(Q, c.Kc, c.Vc, i32(c.table), 32, i32(c.cu), i32(c.total), max(n for _, n in lens),
                                   max(c.total), c.scale, O, lse=lse)
        torch.cuda.synchronize()
        assert torch.equal(O, c.O.cpu()) and torch.equal(lse, c.lse.cpu())
        with pytest.raises(ValueError):
            sfa.sfa_chunk_attend_paged(Q, c.Kc, c.Vc, i32(c.table), 32, i32(c.cu), i32(c.total), max(n for _, n in lens),
                                       max(c.total), c.scale, torch.empty(O.shape, dtype=O.dtype), lse=lse)


@pytest.mark.parametrize("shape", [WIDE, N128])
def test_a_cache_smaller_than_a_page(dev, shape):
    """No cell of any page: every position is left out, and the call says so."""
    c = Case(dev, [(30, 3)], 64, shape, seed=1)
    c.Kc, c.Vc = c.Kc[:40].contiguous(), None if c.Vc is None else c.Vc[:40].contiguous()
    assert c.call(table=[[0, 1]]) == sfa.SFA_DEV_BAD_CELL
    assert bool((c.O == 0).all()) and bool(torch.isneginf(c.lse).all())
