"""SfaPagedCache.release while drafted trees wait for their commit, eager and replayed: the other trees are
committed, no page is lost or held twice, and rows are where they belong."""
import random

import pytest
import torch

from tree_util import accept_reference, random_tree

pytestmark = pytest.mark.gpu

sfa = pytest.importorskip("indexer_selected_sparse_block_gb300")
DEV = "cuda"
N_SEQ, N_MAX, CAP, PAGE, PAGES, WIDTH = 4, 9, 36, 4, 60, 14


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Model:
    """The cache beside what it should hold: a number for each row, in every element of the row."""

    def __init__(self, captured):
        self.c = sfa.SfaPagedCache(n_seq=N_SEQ, n_pages=PAGES, page_size=PAGE, max_pages=WIDTH, n_tok_cap=CAP, h_kv=1, dkq=64,
                                   dv=64, dtype=torch.float32, n_draft_max=N_MAX)
        self.held = [[] for _ in range(N_SEQ)]
        self.serial = 0
        self.new, self.parent, self.token, self.target = (i32([0] * k) for k in (N_SEQ, CAP, CAP, CAP))
        self.K = torch.zeros((CAP, 1, 64), device=DEV)
        self.graphs = None
        if captured:
            draft = lambda: self.c.draft(self.new, self.parent, self.K)
            commit = lambda: self.c.commit(self.token, self.target)
            self.graphs = [sfa.SfaStep.graphed(f) for f in (draft, commit)]

    def feed(self, n):
        rows = [[self.serial + sum(n[:s]) + j + 1 for j in range(k)] for s, k in enumerate(n)]
        self.serial += sum(n)
        self.K.fill_(-1)
        flat = [x for v in rows for x in v]
        if flat:
            self.K[:len(flat)] = torch.tensor(flat, dtype=torch.float32, device=DEV)[:, None, None]
        self.new.copy_(i32(n))
        return rows

    def step(self, n):
        rows = self.feed(n)
        self.c.step(self.new, self.K)
        for h, v in zip(self.held, rows):
            h += v

    def verify(self, n, gone, r):
        rows = self.feed(n)
        trees = [random_tree(k, r, chain=0.5) for k in n]
        tok, tgt = ([[r.randrange(2) for _ in t] for t in trees] for _ in range(2))
        for to, v in ((self.parent, trees), (self.token, tok), (self.target, tgt)):
            flat = [x for t in v for x in t]
            to[:len(flat)] = i32(flat)
        self.graphs[0].replay() if self.graphs else self.c.draft(self.new, self.parent, self.K)
        for s in gone:
            self.c.release(s)
            self.held[s] = []
        self.graphs[1].replay() if self.graphs else self.c.commit(self.token, self.target)
        for s, t in enumerate(trees):
            if s not in gone:
                path, k, nxt = accept_reference(t, tok[s], tgt[s], None, N_MAX)
                assert self.c.path[s].tolist() == path + [-1] * (N_MAX - k)
                assert (int(self.c.n_acc[s]), int(self.c.next_token[s])) == (k, nxt)
                self.held[s] += [rows[s][x] for x in path]

    def check(self):
        c = self.c
        torch.cuda.synchronize()
        assert sfa.sfa_read_device_status(c.status) == 0
        assert c.length.tolist() == [len(h) for h in self.held]
        used = []
        for s, h in enumerate(self.held):
            row = c.page_table[s, :-(-len(h) // PAGE)].tolist()
            used += row
            cells = [row[t // PAGE] * PAGE + t % PAGE for t in range(len(h))]
            assert c.K[cells].tolist() == [[[float(x)] * 64] for x in h]
            assert c.cell_of[s, :len(h)].tolist() == cells
        assert sorted(used + c.free_pages[int(c.free_head):].tolist()) == list(range(PAGES))


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("seed", range(4))
def test_release_between_draft_and_commit(seed, captured):
    r, m = random.Random(seed), Model(captured)
    m.step([7, 8, 0, 5])
    m.check()
    for k in range(12):
        n = [r.choice([0, 1, r.randint(1, N_MAX)]) if len(h) < 40 else 0 for h in m.held]
        m.verify(n, r.sample(range(N_SEQ), r.choice([0, 1, 1, 2, 4])), r)
        m.check()
        if k % 4 == 3:                                      # one that is not committed leaves nothing either
            m.feed(n)
            m.parent.fill_(-1)
            m.c.draft(m.new, m.parent, m.K)
            m.c.release(2)
            m.held[2] = []
            m.step([1, 2, 3, 0])
            m.check()


def test_what_is_cancelled_while_its_step_runs():
    """The sequence of two that is cancelled: the other's path stays, and a new prompt takes its place."""
    m, r = Model(False), random.Random(1)
    m.step([7, 8, 0, 0])
    m.verify([3, 2, 0, 0], [1], r)
    m.check()
    m.step([0, 11, 0, 0])
    m.check()
