"""attend_tree with as many rows of Q as a step has, and the sparse step of trees behind nothing."""
import random

import pytest
import torch

from paged_util import UBF, check_close
from tree_util import ancestors, random_tree, tree_attend_exact

pytestmark = pytest.mark.gpu

sfa = pytest.importorskip("indexer_selected_sparse_block_gb300")
DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def drafted(old, trees, cap, seed, **kw):
    """A cache with `old` tokens a sequence and the trees behind them."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=g, device=DEV).to(torch.bfloat16)
    c = sfa.SfaPagedCache(n_seq=len(old), n_pages=60, page_size=16, max_pages=16, n_tok_cap=cap, h_kv=1, dkq=576, dv=512,
                          n_draft_max=max(map(len, trees)), **kw)
    X = (lambda: randn(cap, kw["d_idx"])) if "d_idx" in kw else (lambda: None)
    c.step(i32(old), randn(cap, 1, 576), X=X())
    flat = [x for t in trees for x in t]
    c.draft(i32([len(t) for t in trees]), i32(flat + [0] * (cap - len(flat))), randn(cap, 1, 576), X=X())
    return c, randn


@pytest.mark.parametrize("part", [sfa.SFA_PART_ALL, sfa.SFA_PART_DRAFTED])
def test_queries_of_the_nodes_alone(part):
    r, old = random.Random(3), [40, 0, 7]
    trees = [random_tree(n, r) for n in (12, 3, 9)]
    c, randn = drafted(old, trees, 80, 3)
    Q = randn(80, 16, 576)
    full, few = torch.full((80, 16, 512), 7.0, device=DEV), torch.full((24, 16, 512), 7.0, device=DEV)
    lse, few_lse = torch.full((80, 16), 7.0, device=DEV), torch.full((24, 16), 7.0, device=DEV)
    c.attend_tree(Q, 12, 52, 0.04, full, lse=lse, part=part)
    c.attend_tree(Q[:24], 12, 52, 0.04, few, lse=few_lse, part=part)
    torch.cuda.synchronize()
    assert sfa.sfa_read_device_status(c.status) == 0
    assert torch.equal(full[:24], few) and torch.equal(lse[:24], few_lse) and bool((full[24:] == 7.0).all())
    with pytest.raises(ValueError):
        c.attend_tree(randn(81, 16, 576), 12, 52, 0.04, torch.empty((81, 16, 512), device=DEV))


def test_sparse_step_behind_nothing():
    """A tree whose sequence holds nothing yet has cached_pos -1: the sparse calls flag its rows and give 0 and
    minus infinity, and the merge is the drafted part."""
    r, old, cr, top = random.Random(4), [150, 0, 2], 4, 8
    trees = [random_tree(n, r) for n in (5, 7, 3)]
    N = 15
    c, randn = drafted(old, trees, 160, 4, d_idx=64)
    step = sfa.SfaStep(n_seq=3, n_tok_cap=256, n_q=N, h_q=16, h_kv=1, dkq=576, dv=512, h_idx=4, d_idx=64, compress_ratio=cr,
                       indexer_top_k=top, n_blk_max=max(old) // cr, cell_of=c.cell_of)
    Q, q_idx, w = randn(N, 16, 576), randn(N, 4, 64), torch.rand((N, 4), device=DEV)
    q_seq, q_pos, scale = c.q_seq[:N].contiguous(), c.cached_pos[:N].contiguous(), 576 ** -0.5
    assert q_pos.tolist() == [149] * 5 + [-1] * 7 + [1] * 3
    step.pool(c.X, 0, old[0] // cr)
    step.select(q_idx, w, q_seq, q_pos)
    step.O.fill_(7.0)
    step.lse.fill_(7.0)
    step.attend(Q, c.K, None, q_seq, q_pos, scale)
    O, lse = torch.empty((N, 16, 512), device=DEV), torch.empty((N, 16), device=DEV)
    c.attend_tree(Q, 7, 160, scale, O, lse=lse, part=sfa.SFA_PART_DRAFTED)
    part = O[5:12].clone()
    assert not bool(step.O[5:12].any()) and bool((step.lse[5:12] == float("-inf")).all())
    sfa.sfa_combine_attention(step.O, step.lse, O, lse, O, lse)
    torch.cuda.synchronize()
    assert sfa.sfa_read_device_status(step.status) & sfa.SFA_DEV_BAD_QUERY and sfa.sfa_read_device_status(c.status) == 0
    assert torch.equal(O[5:12], part)
    seen = ancestors(trees[1])[0]
    ref, ref_l, tol, tol_l = tree_attend_exact(Q[5:12], c.K, None, [c.cell_of[1].tolist()], [0, 7], [7], [seen], scale, 512,
                                               p_round=UBF ** 2)
    check_close(O[5:12], ref, tol, "O")
    check_close(lse[5:12], ref_l, 2 * tol_l, "lse")
