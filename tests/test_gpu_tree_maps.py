"""Drafted trees: masks and positions, the accepted path, what stays in the cache and goes back to the free
list; against plain implementations."""
import random

import pytest
import torch

from tree_util import accept_reference, ancestors, pack, random_tree

pytestmark = pytest.mark.gpu

sfa = pytest.importorskip("indexer_selected_sparse_block_gb300")
DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def run_maps(trees, cached, words, pad=0, cu=None, total=None):
    parent = [p for t in trees for p in t] + [-1] * pad
    if cu is None:
        cu = [0]
        for t in trees:
            cu.append(cu[-1] + len(t))
    if total is None:
        total = [a + len(t) for a, t in zip(cached, trees)]
    n = len(parent)
    mask = i32([[7] * words] * n).reshape(n, words)
    q_pos, last, status = i32([9] * n), i32([9] * n), i32([0])
    sfa.sfa_build_tree_maps(i32(parent), i32(cu), i32(total), mask, q_pos, cached_pos=last, dev_status=status)
    return mask.tolist(), q_pos.tolist(), last.tolist(), sfa.sfa_read_device_status(status)


def want_maps(trees, cached, words, pad=0):
    mask, q_pos, last = [], [], []
    for t, a in zip(trees, cached):
        seen, depth = ancestors(t[:32 * words])
        cut = len(t) - len(seen)
        mask += pack(seen, words) + [[0] * words] * cut
        q_pos += [a + d for d in depth] + [-1] * cut
        last += [a - 1] * len(seen) + [-1] * cut
    return mask + [[0] * words] * pad, q_pos + [-1] * pad, last + [-1] * pad


@pytest.mark.parametrize("n_seq,n,words,pad,roots", [
    (1, 1, 1, 0, 1), (1, 2, 1, 3, 1), (3, 31, 1, 0, 1), (3, 32, 1, 1, 2), (2, 33, 2, 0, 1), (5, 64, 2, 7, 3),
    (4, 65, 3, 0, 1), (2, 100, 32, 5, 1), (2, 1024, 32, 0, 1), (300, 20, 1, 11, 1), (2, 257, 9, 0, 40)])
@pytest.mark.parametrize("chain", [0.0, 0.3, 1.0])
def test_maps(n_seq, n, words, pad, roots, chain):
    r = random.Random(n * 7 + n_seq)
    trees = [random_tree(r.choice([0, n, r.randint(1, n)]), r, roots, chain) for _ in range(n_seq)]
    trees[-1] = random_tree(n, r, roots, chain)
    cached = [r.choice([0, 1, r.randrange(100000)]) for _ in trees]
    assert run_maps(trees, cached, words, pad) == (*want_maps(trees, cached, words, pad), 0)


def test_maps_of_bad_trees():
    """Parents that are none make roots; nodes past the mask have none of it; flagged."""
    trees = [[-1, 1, 0, -2, 5, 3, 1 << 30, -(1 << 31)], [-1, 0]]
    got = run_maps(trees, [10, 0], 1)
    fixed = [[-1, -1, 0, -1, -1, 3, -1, -1], [-1, 0]]
    assert got == (*want_maps(fixed, [10, 0], 1), sfa.SFA_DEV_BAD_TREE)
    long = [random_tree(40, random.Random(1))]
    assert run_maps(long, [5], 1) == (*want_maps(long, [5], 1), sfa.SFA_DEV_BAD_TREE)


def test_maps_of_bad_offsets():
    trees, bad = [[-1, 0, 0], [-1, 0]], sfa.SFA_DEV_BAD_QUERY
    mask, q_pos, _, st = run_maps(trees, [4, 4], 1, cu=[0, 3, 99])
    want = want_maps(trees[:1], [4], 1)
    assert mask[:3] == want[0] and q_pos[:3] == want[1] and st == bad
    _, q_pos, last, st = run_maps(trees, [4, 4], 1, total=[2, 6])      # fewer positions than nodes
    assert q_pos == [0, 1, 1, 4, 5] and last == [-1, -1, -1, 3, 3] and st == bad
    _, q_pos, _, st = run_maps(trees, [4, 4], 1, cu=[-1, 3, 5])
    assert q_pos[3:] == [5 - 1, 5] and st == bad


def test_maps_of_nothing():
    assert run_maps([], [], 1, pad=4) == ([[0]] * 4, [-1] * 4, [-1] * 4, 0)
    assert run_maps([[], []], [3, 0], 1) == ([], [], [], 0)


def run_accept(trees, token, target, most, root=None, pad=0):
    cu = [0]
    for t in trees:
        cu.append(cu[-1] + len(t))
    flat = lambda v: i32([x for t in v for x in t] + [-1] * pad)
    n = len(trees)
    path, n_acc, nxt, status = i32([[9] * most] * n).reshape(n, most), i32([9] * n), i32([9] * n), i32([0])
    sfa.sfa_tree_accept(flat(trees), flat(token), flat(target), i32(cu), path, n_acc, nxt,
                        root_target=None if root is None else i32(root), dev_status=status)
    return path.tolist(), n_acc.tolist(), nxt.tolist(), sfa.sfa_read_device_status(status)


@pytest.mark.parametrize("n_seq,n,most,tokens,roots,chain", [
    (1, 1, 1, 5, 1, 0.0), (1, 16, 16, 2, 1, 0.3), (40, 64, 64, 3, 1, 0.2), (40, 64, 3, 1, 1, 0.6), (7, 1024, 1024, 2, 1, 0.5),
    (7, 200, 200, 1, 1, 1.0), (33, 33, 40, 4, 5, 0.3), (3, 1024, 1024, 1, 1, 1.0)])
@pytest.mark.parametrize("rooted", [False, True])
def test_accept(n_seq, n, most, tokens, roots, chain, rooted):
    """Few tokens, so that siblings share them and paths go deep; empty trees, roots that are not the
    model's."""
    r = random.Random(n + most)
    trees = [random_tree(r.choice([0, n, r.randint(1, n)]), r, roots, chain) for _ in range(n_seq)]
    trees[0] = random_tree(n, r, roots, chain)
    draw = lambda: [[r.randrange(tokens) for _ in t] for t in trees]
    token, target = draw(), draw()
    root = [r.randrange(tokens) for _ in trees] if rooted else None
    path, n_acc, nxt, st = run_accept(trees, token, target, most, root, pad=3)
    for s, t in enumerate(trees):
        p, k, w = accept_reference(t, token[s], target[s], root[s] if rooted else None, most)
        assert (path[s], n_acc[s], nxt[s]) == (p + [-1] * (most - k), k, w)
    assert st == 0


def test_accept_leaves_bad_nodes_out():
    got = run_accept([[-1, 5, 0, -3, 2]], [[1, 1, 1, 1, 1]], [[1, 1, 1, 1, 8]], 5)
    assert got == ([[0, 2, 4, -1, -1]], [3], [8], sfa.SFA_DEV_BAD_TREE)


class Commit:
    """Sequences with cached and drafted tokens on random pages; caches of several kinds."""

    def __init__(self, lens, page, kinds=("bf16",), seed=0, width=None, lost=()):
        r = random.Random(seed)
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.lens, self.page = lens, page
        need = [-(-(a + n) // page) for a, n in lens]
        self.n_pages = sum(need) + 3
        order = list(range(self.n_pages))
        r.shuffle(order)
        self.width = max(need) + 1 if width is None else width
        self.table, taken, k = [], [], 0
        for (a, _), c in zip(lens, need):
            row = order[k:k + c]
            self.table.append(row + [-1] * (self.width - c))
            taken += row[-(-a // page):]
            k += c
        self.free = [99] * 2 + taken + order[k:]         # two entries of no matter, this step's, what is left
        self.head = 2 + len(taken)
        self.cu = [0]
        self.slot = []
        for s, (a, n) in enumerate(lens):
            self.cu.append(self.cu[-1] + n)
            for pos in range(a, a + n):
                self.slot.append(self.table[s][pos // page] * page + pos % page)
        for i in lost:
            self.slot[i] = -1
        shapes = {"bf16": ((2, 64), torch.bfloat16), "f32": ((1, 30), torch.float32), "q8": ((2, 80), torch.uint8),
                  "odd": ((1, 51), torch.bfloat16), "wide": ((1, 576), torch.bfloat16)}
        self.caches = []
        for kind in kinds:
            shape, dt = shapes[kind]
            x = torch.randint(0, 255, (self.n_pages * page, *shape), generator=g, device=DEV)
            self.caches.append(x.to(dt))

    def run(self, path, n_acc, head=None, in_place=False, slot=None):
        n = len(self.lens)
        total = i32([a + b for a, b in self.lens])
        free, hd = i32(self.free), i32([self.head if head is None else head])
        out, ho = (total, hd) if in_place else (i32([9] * n), i32([9]))
        status, table = i32([0]), i32(self.table).reshape(n, self.width)
        most = max([len(p) for p in path] + [1])
        rows = i32([p + [-1] * (most - len(p)) for p in path]).reshape(n, most)
        got = [c.clone() for c in self.caches]
        sfa.sfa_tree_commit(got, i32(self.slot), i32(self.cu), rows, i32(n_acc), total, self.page, table, free, hd, out, ho,
                            dev_status=status)
        return got, out.tolist(), ho.tolist()[0], free.tolist(), table.tolist(), sfa.sfa_read_device_status(status)

    def want(self, path, head=None):
        """path: the valid part of each."""
        caches = [c.clone() for c in self.caches]
        length, back = [], []
        for s, ((a, n), p) in enumerate(zip(self.lens, path)):
            src = [self.slot[self.cu[s] + x] for x in p]
            dst = [self.slot[self.cu[s] + k] for k in range(len(p))]
            n_cells = self.n_pages * self.page
            pairs = [(i, j) for i, j in zip(src, dst) if 0 <= i < n_cells and 0 <= j < n_cells]
            for c, old in zip(caches, self.caches):
                for i, j in pairs:
                    c[j] = old[i]
            length.append(a + len(p))
            back += [e for e in self.table[s][-(-(a + len(p)) // self.page):-(-(a + n) // self.page)] if e >= 0]
        head = self.head if head is None else head
        free = list(self.free)
        for i, e in enumerate(back):
            if head - len(back) + i >= 0:
                free[head - len(back) + i] = e
        return caches, length, max(head - len(back), 0), free

    def check(self, path, n_acc=None, status=0, **kw):
        valid = [p[:m] for p, m in zip(path, [len(p) for p in path] if n_acc is None else n_acc)]
        got, length, head, free, table, st = self.run(path, [len(p) for p in path] if n_acc is None else n_acc, **kw)
        want = self.want(valid, head=kw.get("head"))
        for x, y in zip(got, want[0]):
            assert torch.equal(x, y)
        assert (length, head, free, table, st) == (*want[1:], self.table, status)


def random_path(n, r, most=None):
    k = r.randint(0, min(n, most or n))
    return sorted(r.sample(range(n), k))


@pytest.mark.parametrize("n_seq,old,new,page,most", [
    (1, 0, 1, 1, 1), (1, 63, 16, 64, 5), (5, 100, 64, 16, 9), (3, 40, 200, 7, 200), (40, 30, 33, 8, 6), (700, 20, 9, 4, 4),
    (2, 5, 1024, 48, 1024), (3, 0, 40, 1, 40)])
@pytest.mark.parametrize("in_place", [False, True])
def test_commit(n_seq, old, new, page, most, in_place):
    r = random.Random(old + new * 3 + page)
    lens = [(r.choice([0, old, r.randint(0, old)]), r.choice([0, new, r.randint(1, new)])) for _ in range(n_seq)]
    lens[0] = (old, new)
    c = Commit(lens, page, ("bf16", "f32", "q8", "odd"), seed=new)
    c.check([random_path(n, r, most) for _, n in lens], in_place=in_place)


@pytest.mark.parametrize("kinds", [(), ("wide",), ("odd",), ("wide", "wide", "bf16", "q8")])
def test_commit_of_any_caches(kinds):
    c = Commit([(50, 60), (3, 20)], 8, kinds)
    c.check([list(range(1, 60, 2)), [0, 1, 2, 19]])
    c.check([[], []])
    c.check([list(range(60)), list(range(20))])        # all of it: nothing moves or goes back


def test_commit_stops_at_bad_paths():
    c = Commit([(10, 8), (10, 8), (10, 8), (10, 8), (10, 8)], 4)
    bad = sfa.SFA_DEV_BAD_TREE
    paths = [[1, 3, 2, 5], [2, 8], [-1], [5, 5], [0, 7]]
    got = c.run(paths, [4, 2, 1, 2, 9])
    want = c.want([[1, 3], [2], [], [5], [0, 7]])
    assert all(torch.equal(x, y) for x, y in zip(got[0], want[0]))
    assert got[1:4] == want[1:] and got[5] == bad
    c.check([[1], [2], [], [], [4]], n_acc=[1, 1, -3, 0, 1], status=bad)


def test_commit_of_lost_nodes():
    """Nodes without a cell count, and their rows stay where they are; flagged."""
    c = Commit([(4, 8)], 4, lost=(6, 7))
    c.check([[1, 3, 6]], status=sfa.SFA_DEV_BAD_CELL)
    c.slot[2] = 1 << 30
    c.check([[1, 2, 5]], status=sfa.SFA_DEV_BAD_CELL)


def test_commit_with_a_head_that_took_nothing():
    c = Commit([(0, 16)], 4)
    c.check([[0]], head=1, status=sfa.SFA_DEV_BAD_LENGTH)
    c.check([[0]], head=-5, status=sfa.SFA_DEV_BAD_LENGTH)


def test_commit_of_no_sequence():
    free, head, out = i32([1, 2, 3]), i32([2]), i32([9])
    e = lambda *s: torch.empty(s, dtype=torch.int32, device=DEV)
    sfa.sfa_tree_commit([], e(0), i32([0]), e(0, 1), e(0), e(0), 4, e(0, 2), free, head, e(0), out)
    assert out.tolist() == [2] and free.tolist() == [1, 2, 3]


def test_offsets_past_32_bits():
    """Rows of a cache of more than 2^31 bytes and elements."""
    n_cells = (1 << 31) // 576 + 4096
    cache = torch.empty((n_cells, 1, 576), dtype=torch.bfloat16, device=DEV)
    slot = [n_cells - 9, 5, n_cells - 1, n_cells - 2]
    rows = torch.randn((4, 1, 576), device=DEV).to(torch.bfloat16)
    cache[slot] = rows
    table, free, head = i32([[0, 1]]), i32([0, 1]), i32([2])
    ln = i32([0])
    sfa.sfa_tree_commit([cache], i32(slot), i32([0, 4]), i32([[1, 2, 3]]), i32([3]), i32([4]), n_cells, table, free, head,
                        ln, head)
    assert torch.equal(cache[slot], rows[[1, 2, 3, 3]]) and ln.tolist() == [3]
