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
