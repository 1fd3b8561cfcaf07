"""Whole verification steps of drafted trees through SfaPagedCache: page maps, masks, rotated rows into their
cells, attention, the accepted path; against a plain model of the same sequences, over several steps, captured
and replayed; and the sparse step (kept blocks of the cached tokens beside the drafted ones)."""
import math
import random

import pytest
import torch

from paged_util import UBF, check_close
from rotate_util import rotate_reference
from tree_util import accept_reference, ancestors, random_tree, tree_attend_exact

pytestmark = pytest.mark.gpu

sfa = pytest.importorskip("indexer_selected_sparse_block_gb300")
DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Model:
    """What each sequence should hold: its rows K (unrotated, with their positions), V, X."""

    def __init__(self, n_seq):
        self.rows = [[] for _ in range(n_seq)]


def draw_step(r, n_seq, n_max, cap, shape, g, d_idx):
    h_kv, dkq, dv, sep, h_q = shape
    n = [r.choice([0, 1, r.randint(1, n_max)]) for _ in range(n_seq)]
    trees = [random_tree(k, r, chain=0.5) for k in n]
    randn = lambda h, d: torch.randn((cap, h, d), generator=g, device=DEV).to(torch.bfloat16)
    return n, trees, randn(h_kv, dkq), randn(h_kv, dv) if sep else None, randn(1, d_idx)[:, 0], randn(h_q, dkq)


def flat(v, cap):
    x = [e for t in v for e in t]
    return x + [0] * (cap - len(x))


@pytest.mark.parametrize("dkq,dv,h_q,h_kv,sep,rot,pairs", [(576, 512, 16, 1, False, 64, True), (128, 128, 8, 2, True, 128, False),
                                                         (64, 64, 8, 8, True, 32, False)])
@pytest.mark.parametrize("captured", [False, True])
def test_steps(dkq, dv, h_q, h_kv, sep, rot, pairs, captured):
    n_seq, n_max, cap, page, d_idx = 4, 20, 64, 8, 64
    r, g = random.Random(dkq), torch.Generator(device=DEV).manual_seed(dkq)
    c = sfa.SfaPagedCache(n_seq=n_seq, n_pages=70, page_size=page, max_pages=20, n_tok_cap=cap, h_kv=h_kv, dkq=dkq, dv=dv,
                          separate_v=sep, d_idx=d_idx, n_draft_max=n_max)
    rope = sfa.SfaRope(rot, pairs=pairs, factor=4.0, original_len=64, magnitude=1.1)
    scale = dkq ** -0.5
    # prompts by a plain step, turned too
    prompt = [30, 0, 7, 1]
    held = [[] for _ in range(n_seq)]                       # (K, V, X) rows of each position, K turned
    n, _, K, V, X, Q = draw_step(r, n_seq, n_max, cap, (h_kv, dkq, dv, sep, h_q), g, d_idx)
    Q0 = Q.clone()
    c.step(i32(prompt), K, V, X, rope=rope, Q=Q)

    def keep(K, V, X, rows_of, positions):
        """What the rows' cells should hold, and Q's bound: the plain rotation."""
        pos = i32([0 if p < 0 else p for p in positions])
        ref, tol = rotate_reference(K, pos, rope.freqs, rope.magnitude, dkq - rot, pairs, torch.bfloat16)
        return ref, tol

    at = 0
    ref, tol = keep(K, V, X, None, [p for k in prompt for p in range(k)] + [0] * (cap - sum(prompt)))
    for s, k in enumerate(prompt):
        for p in range(k):
            held[s].append((ref[at], tol[at], None if V is None else V[at].clone(), X[at].clone()))
            at += 1
    qref, qtol = rotate_reference(Q0[:at], i32([p for k in prompt for p in range(k)]), rope.freqs, rope.magnitude, dkq - rot,
                                  pairs, torch.bfloat16)
    check_close(Q[:at], qref, qtol, "turned queries")
    assert torch.equal(Q[at:], Q0[at:])

    def check_cache():
        assert c.length.tolist() == [len(h) for h in held]
        for s, h in enumerate(held):
            if not h:
                continue
            t = torch.arange(len(h), device=DEV)
            cells = c.page_table[s].long()[t // page] * page + t % page
            check_close(c.K[cells], torch.stack([x[0] for x in h]), torch.stack([x[1] for x in h]), "K")
            if sep:
                assert torch.equal(c.V[cells], torch.stack([x[2] for x in h]))
            assert torch.equal(c.X[cells], torch.stack([x[3] for x in h]))
            assert torch.equal(c.cell_of[s, :len(h)].long(), cells)
        # no page is lost, or in two places
        used = [e for s, h in enumerate(held) for e in c.page_table[s, :-(-len(h) // page)].tolist()]
        free = c.free_pages[int(c.free_head):].tolist()
        assert sorted(used + free) == list(range(70))

    check_cache()
    new, parent = i32([0] * n_seq), i32([0] * cap)
    token, target, O, lse = i32([0] * cap), i32([0] * cap), torch.empty((cap, h_q, dv), device=DEV), torch.empty((cap, h_q), device=DEV)
    bK, bV, bX, bQ = (None if x is None else torch.empty_like(x) for x in (K, V, X, Q))
    need = sfa.sfa_tree_attend_workspace_bytes(sfa.SFA_BF16, n_seq, cap, h_q, h_kv, dkq, dv, sep, n_max, 160)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)

    def step():
        c.draft(new, parent, bK, bV, bX, rope=rope, Q=bQ)
        c.attend_tree(bQ, n_max, 160, scale, O, lse=lse, workspace=ws)
        c.commit(token, target)

    graph = None
    if captured:
        graph = sfa.SfaStep.graphed(step)                   # its warm-up steps have no node
    for _ in range(5):
        n, trees, K, V, X, Q = draw_step(r, n_seq, n_max, cap, (h_kv, dkq, dv, sep, h_q), g, d_idx)
        tok, tgt = [[r.randrange(2) for _ in t] for t in trees], [[r.randrange(2) for _ in t] for t in trees]
        new.copy_(i32(n))
        for to, v in ((parent, trees), (token, tok), (target, tgt)):
            to.copy_(i32(flat(v, cap)))
        for to, v in ((bK, K), (bV, V), (bX, X), (bQ, Q)):
            if v is not None:
                to.copy_(v)
        old = [len(h) for h in held]
        O.fill_(5.0)
        graph.replay() if captured else step()
        torch.cuda.synchronize()
        assert sfa.sfa_read_device_status(c.status) == 0
        cu, pos, seen = [0], [], []
        for s, t in enumerate(trees):
            cu.append(cu[-1] + len(t))
            v, depth = ancestors(t)
            seen.append(v)
            pos += [old[s] + d for d in depth]
        assert c.q_pos.tolist() == pos + [-1] * (cap - len(pos))
        # the attention, of the queries as they were turned, over the rows as they should have been held
        ref, tol = keep(K, V, X, None, pos + [0] * (cap - len(pos)))
        rows_k = [x[0] for h, t, a in zip(held, trees, cu) for x in h + [(ref[a + j],) for j in range(len(t))]]
        rows_v = None
        if sep:
            rows_v = torch.stack([x[2] for h, t, a in zip(held, trees, cu) for x in h + [(0, 0, V[a + j]) for j in range(len(t))]])
        if rows_k and cu[-1]:
            cells, k = [], 0
            for h, t in zip(held, trees):
                cells.append(list(range(k, k + len(h) + len(t))))
                k += len(h) + len(t)
            # a turned row in its cell is rounded to bf16: half a step of each product, like a product's error
            w, _, bound, _ = tree_attend_exact(bQ[:cu[-1]], torch.stack(rows_k).to(DEV), rows_v, cells, cu,
                                               [a + len(t) for a, t in zip(old, trees)], seen, scale, dv,
                                               product=UBF * 1.01, p_round=UBF ** 2)
            check_close(O[:cu[-1]], w, bound, "O")
        assert bool((O[cu[-1]:] == 5.0).all())
        for s, t in enumerate(trees):
            p, k, nxt = accept_reference(t, tok[s], tgt[s], None, n_max)
            assert c.path[s].tolist() == p + [-1] * (n_max - k) and int(c.n_acc[s]) == k and int(c.next_token[s]) == nxt
            for x in p:
                a = cu[s] + x
                held[s].append((ref[a], tol[a], None if V is None else V[a].clone(), X[a].clone()))
        check_cache()


def test_draft_and_commit_in_graphs_of_their_own():
    """The model's choices are made between them; replayed, they keep what a cache without graphs keeps."""
    kw = dict(n_seq=2, n_pages=20, page_size=4, max_pages=8, n_tok_cap=12, h_kv=1, dkq=64, dv=64, n_draft_max=6)
    a, b = sfa.SfaPagedCache(**kw), sfa.SfaPagedCache(**kw)
    r = random.Random(5)
    new, parent, token, target = i32([0, 0]), i32([0] * 12), i32([0] * 12), i32([0] * 12)
    K = torch.zeros((12, 1, 64), dtype=torch.bfloat16, device=DEV)
    draft = sfa.SfaStep.graphed(lambda: a.draft(new, parent, K))
    commit = sfa.SfaStep.graphed(lambda: a.commit(token, target))
    for _ in range(6):
        n = [r.randint(0, 6), r.randint(0, 6)]
        trees = [random_tree(k, r, chain=0.6) for k in n]
        new.copy_(i32(n))
        parent.copy_(i32(flat(trees, 12)))
        token.copy_(torch.randint(0, 2, (12,), device=DEV))
        target.copy_(torch.randint(0, 2, (12,), device=DEV))
        K.copy_(torch.randn((12, 1, 64), device=DEV))
        draft.replay()
        commit.replay()
        b.draft(new, parent, K)
        b.commit(token, target)
        torch.cuda.synchronize()
        for x, y in ((a.length, b.length), (a.free_head, b.free_head), (a.free_pages, b.free_pages), (a.path, b.path),
                     (a.next_token, b.next_token), (a.K, b.K)):
            assert torch.equal(x, y)
    assert int(a.length.sum()) > 0 and sfa.sfa_read_device_status(a.status) == 0


def test_a_dropped_tree():
    """A draft that is not committed leaves nothing behind: the next step takes its place."""
    kw = dict(n_seq=2, n_pages=12, page_size=4, max_pages=5, n_tok_cap=12, h_kv=1, dkq=64, dv=64, n_draft_max=12)
    c = sfa.SfaPagedCache(**kw)
    K = torch.randn((12, 1, 64), device=DEV).to(torch.bfloat16)
    c.step(i32([5, 3]), K)
    c.draft(i32([6, 6]), i32([-1, 0, 0, 1, 1, 2] * 2), K)
    c.step(i32([1, 1]), K)
    assert c.length.tolist() == [6, 4] and int(c.free_head) == 3
    assert sfa.sfa_read_device_status(c.status) == 0
    with pytest.raises(ValueError):
        c.commit(i32([0] * 12), i32([0] * 12))


def test_sparse_step():
    """The kept blocks and the tail of the cached tokens by the sparse call, the drafted ones by the tree's,
    merged: against the plain attention over both."""
    n_seq, page, cr, top, dkq, dv, h_q, d_idx, h_idx = 3, 16, 4, 8, 576, 512, 16, 64, 4
    r, g = random.Random(7), torch.Generator(device=DEV).manual_seed(7)
    old, n = [150, 203, 61], [12, 1, 9]
    cap = max(sum(old), sum(n))
    c = sfa.SfaPagedCache(n_seq=n_seq, n_pages=60, page_size=page, max_pages=16, n_tok_cap=cap, h_kv=1, dkq=dkq, dv=dv,
                          d_idx=d_idx, n_draft_max=12)
    randn = lambda *s: torch.randn(s, generator=g, device=DEV).to(torch.bfloat16)
    c.step(i32(old), randn(cap, 1, dkq), X=randn(cap, d_idx))
    trees = [random_tree(k, r) for k in n]
    N = sum(n)
    c.draft(i32(n), i32(flat(trees, cap)), randn(cap, 1, dkq), X=randn(cap, d_idx))
    step = sfa.SfaStep(n_seq=n_seq, n_tok_cap=16 * page, n_q=N, h_q=h_q, h_kv=1, dkq=dkq, dv=dv, h_idx=h_idx, d_idx=d_idx,
                       compress_ratio=cr, indexer_top_k=top, n_blk_max=max(old) // cr, cell_of=c.cell_of)
    Q, q_idx, w = randn(N, h_q, dkq), randn(N, h_idx, d_idx), torch.rand((N, h_idx), generator=g, device=DEV)
    q_seq, q_pos, scale = c.q_seq[:N].contiguous(), c.cached_pos[:N].contiguous(), dkq ** -0.5
    # the cached tokens' blocks only: what the nodes' positions complete is not the cache's yet
    step.pool(c.X, 0, min(old) // cr)
    for s in range(n_seq):                                   # the longer sequences' blocks
        step.pool(c.X, 0, old[s] // cr) if old[s] == max(old) else None
    step.select(q_idx, w, q_seq, q_pos)
    step.attend(Q, c.K, None, q_seq, q_pos, scale)
    O, lse = torch.empty((N, h_q, dv), device=DEV), torch.empty((N, h_q), device=DEV)
    sfa.sfa_tree_attend_paged(Q, c.K, None, c.page_table, page, c.cu_new, c.len_total, c.tree_mask[:N].contiguous(), 12,
                              max(old) + 12, scale, O, lse=lse, part=sfa.SFA_PART_DRAFTED)
    sfa.sfa_combine_attention(step.O, step.lse, O, lse, O, lse)
    torch.cuda.synchronize()
    blocks, kept = step.blk_idx.tolist(), step.n_sel.tolist()
    i = 0
    for s in range(n_seq):
        seen, _ = ancestors(trees[s])
        cells = c.cell_of[s].tolist()
        for j in range(n[s]):
            on = [t for b in blocks[i][:kept[i]] for t in range(b * cr, b * cr + cr)] + list(range(old[s] // cr * cr, old[s]))
            assert kept[i] == min(top, old[s] // cr)
            on += [old[s] + x for x in range(n[s]) if seen[j][x]]
            at = [cells[t] for t in on]
            m = len(at)
            ref, ref_l, tol, tol_l = tree_attend_exact(Q[i:i + 1], c.K, None, [at], [0, 1], [m], [[[True]]], scale, dv,
                                                       p_round=UBF ** 2)
            # the sparse call's own bound, 2e-3 of a row's largest value, beside the drafted part's
            check_close(O[i:i + 1], ref, tol + 2e-3 * ref.abs().amax(-1, keepdim=True), f"row {i}")
            # its log-sum-exp: fp32 scores and sums
            check_close(lse[i:i + 1], ref_l, 4 * tol_l + 2.0 ** -14, f"lse {i}")
            i += 1
