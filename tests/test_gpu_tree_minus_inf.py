"""A node whose score for a query is minus infinity: its values do not reach that query, finite or not, whichever
kernel the sizes choose; other queries that attend it get what is not finite."""
import math

import pytest
import torch

from paged_util import check_close
from test_gpu_chunk import N64, N64K, N128, N128K, W512, W512K, WIDE
from test_gpu_tree_attend import DRAFTED, Trees

pytestmark = pytest.mark.gpu

sfa = pytest.importorskip("indexer_selected_sparse_block_gb300")

LENS = {"small": [(70, 30), (0, 17), (130, 64)], "large": [(70, 300), (0, 17), (5, 40)]}
DIM = 3                                                 # where the keys are infinite


def check(c, odd):
    """odd: (sequence, node, KV head) with an infinite key.  Queries that it does not reach, because of their mask
    or their sign at DIM, are those of a tree without it."""
    G = c.h_q // c.h_kv
    O, lse = c.O.double().cpu(), c.lse.double().cpu()
    negative = (c.Q[..., DIM] < 0).cpu()                # [n_q][h_q]
    for i in range(c.h_kv):
        heads = slice(i * G, (i + 1) * G)
        # with and without the nodes, by whether a query's sign keeps them out
        without = [[list(v) for v in s] for s in c.seen]
        hit = torch.zeros((c.cu[-1],), dtype=torch.bool)
        for s, x, head in odd:
            if head == i:
                for j, v in enumerate(without[s]):
                    hit[c.cu[s] + j] |= v[x]
                    v[x] = False
        ref, ref_l, tol, tol_l = c.exact(seen=without, twice=True)
        out = hit[:, None] & ~negative[:c.cu[-1], heads]    # a score of plus infinity
        if any(head == i for _, _, head in odd):
            assert bool(hit.any()) and bool(out.any()) and bool((hit[:, None] & ~out).any())
        assert not bool(torch.isfinite(O[:c.cu[-1], heads][out]).any())
        keep = ~out
        for got, r, t, m in ((O, ref, tol, keep[..., None]), (lse, ref_l, tol_l, keep)):
            got, r, t = got[:c.cu[-1], heads], r[:c.cu[-1], heads], t[:c.cu[-1], heads]
            check_close(torch.where(m, got, r), r, t, f"KV head {i}")


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("sizes", sorted(LENS))
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [WIDE, W512, W512K, N128, N128K, N64, N64K])
def test_scores_of_minus_infinity(shape, dtype, sizes, out):
    c = Trees(LENS[sizes], 16, shape, dtype, out, seed=shape[0])
    c.Q[..., DIM] = torch.where(c.Q[..., DIM] < 0, -1.0, 1.0)
    odd = [(0, 4, 0), (0, 20, shape[4] - 1), (1, 1, 0), (2, 0, shape[4] - 1)]
    for s, x, head in odd:
        cell = c.cells[s][LENS[sizes][s][0] + x]
        c.K[cell, head, DIM] = math.inf
        if c.V is not None:
            c.V[cell, head, 5] = math.nan
            c.V[cell, head, 9] = -math.inf
    for part in (DRAFTED, sfa.SFA_PART_ALL):
        assert c.call(part) == 0
        check(c, odd)
