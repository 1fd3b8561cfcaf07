"""A sequence released while drafted trees wait for their commit: the cache's lists, with the page maps' and
the commit's rules of include/sfa.h in plain Python in the kernels' place; and how often a draft is committed."""
import random

import pytest
import torch

import indexer_selected_sparse_block_gb300 as sfa
from indexer_selected_sparse_block_gb300 import SfaPagedCache
from test_host_tree_streams import cache, i32, launches  # noqa: F401 (a fixture)

P, PAGES, WIDTH = 4, 10, 6


def make(n_seq):
    return sfa.SfaPagedCache(n_seq=n_seq, n_pages=PAGES, page_size=P, max_pages=WIDTH, n_tok_cap=32, h_kv=1, dkq=64, dv=64,
                             device="cpu", n_draft_max=16)


def pages(n):
    return -(-n // P)


def draft(c, new):
    """sfa_build_page_maps: cells for the nodes; the lengths stay."""
    at, cu = int(c.free_head), [0]
    for s, n in enumerate(new):
        a = int(c.length[s])
        for k in range(pages(a), pages(a + n)):
            c.page_table[s, k] = c.free_pages[at]
            at += 1
        c.len_total[s] = a + n
        cu.append(cu[-1] + n)
    c.cu_new.copy_(torch.tensor(cu))
    c._head_out.fill_(at)


def step(c, new):
    draft(c, new)
    c.length.copy_(c.len_total)
    c.free_head.copy_(c._head_out)


def commit(c, kept):
    """sfa_tree_commit: kept[s] nodes of each tree stay; nothing of a sequence that holds nothing any more."""
    back = []
    for s, m in enumerate(kept):
        n, total = int(c.cu_new[s + 1] - c.cu_new[s]), int(c.len_total[s])
        keep = 0 if total == 0 else max(total - n, 0) + min(m, n)
        back += [e for e in c.page_table[s, pages(keep):pages(total)].tolist() if e >= 0]
        c.length[s] = keep
    head = int(c._head_out)
    c.free_pages[head - len(back):head] = torch.tensor(back, dtype=torch.int32)
    c.free_head.fill_(head - len(back))


def check(c, lengths):
    assert c.length.tolist() == lengths
    held = [e for s, n in enumerate(lengths) for e in c.page_table[s, :pages(n)].tolist()]
    free = c.free_pages[int(c.free_head):].tolist()
    assert sorted(held + free) == list(range(PAGES))


@pytest.mark.parametrize("gone,lengths", [(1, [10, 0]), (0, [0, 10])])
def test_the_other_trees_are_committed(gone, lengths):
    c = make(2)
    step(c, [7, 8])
    draft(c, [3, 2])
    c.release(gone)
    commit(c, [3, 2])
    check(c, lengths)
    step(c, [5, 1])
    check(c, [n + k for n, k in zip(lengths, [5, 1])])


def test_a_tree_that_is_dropped_after_a_release():
    c = make(3)
    step(c, [7, 8, 1])
    draft(c, [3, 2, 9])
    c.release(1)
    c.release(2)
    step(c, [1, 1, 1])
    check(c, [8, 1, 1])


def test_release_after_a_commit_without_a_new_draft():
    c = make(3)
    step(c, [7, 8, 0])
    draft(c, [3, 2, 4])
    commit(c, [1, 0, 2])
    c.release(2)                                    # what is left looks like trees of no accepted node
    check(c, [8, 8, 0])
    c.release(1)
    check(c, [8, 0, 0])
    draft(c, [2, 3, 3])
    commit(c, [2, 1, 0])
    check(c, [10, 1, 0])


def test_release_after_a_commit_that_kept_nodes_of_one_prompt_alone():
    """Once that sequence is released, the others are as they were before the draft, but nothing is pending."""
    c = make(3)
    step(c, [0, 8, 3])
    draft(c, [5, 6, 2])
    commit(c, [4, 0, 0])
    c.release(0)
    check(c, [0, 8, 3])
    c.release(1)
    check(c, [0, 0, 3])
    c.release(2)
    check(c, [0, 0, 0])


def test_pages_of_an_earlier_draft_behind_the_end():
    """A table's row still names pages that went back and that another sequence's tree has now."""
    c = make(2)
    step(c, [4, 4])
    draft(c, [16, 0])                               # pages 2 to 5 of sequence 0, all given back
    commit(c, [0, 0])
    draft(c, [0, 9])                                # pages 2 to 4 of sequence 1
    c.release(0)
    commit(c, [0, 9])
    check(c, [0, 13])


@pytest.mark.parametrize("seed", range(40))
def test_any_order(seed):
    r = random.Random(seed)
    c, want = make(3), [0, 0, 0]
    for _ in range(30):
        room = PAGES - sum(pages(n) for n in want)
        new = [r.choice([0, 1, r.randint(0, 5)]) if pages(n) < WIDTH - 2 else 0 for n in want]
        if sum(pages(n + k) - pages(n) for n, k in zip(want, new)) > room:
            new = [0] * 3
        if r.random() < 0.4:
            step(c, new)
            want = [n + k for n, k in zip(want, new)]
        else:
            draft(c, new)
            for s in r.sample(range(3), r.choice([0, 0, 1, 1, 2, 3])):
                c.release(s)
                want[s] = new[s] = 0
            if r.random() < 0.7:
                kept = [r.randint(0, k) for k in new]
                commit(c, kept)
                want = [n + k for n, k in zip(want, kept)]
        check(c, want)
        if r.random() < 0.3:
            s = r.randrange(3)
            c.release(s)
            want[s] = 0
            check(c, want)
