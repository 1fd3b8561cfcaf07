"""The drafted-tree entry points on the host: refusals before anything is enqueued, the size query, the
binding's and the cache's checks."""
import ctypes

import pytest
import torch

from test_host_scratch import Fake, f32, i32

FAKE = ctypes.c_void_p(0x10000)     # never dereferenced: every call below is rejected first
ODD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def B():
    import __graft_entry__
    __graft_entry__.build()
    from indexer_selected_sparse_block_gb300 import _binding
    return _binding


@pytest.fixture(scope="module")
def L(B):
    return B.lib()


MAPS = dict(parent=FAKE, cu=FAKE, total=FAKE, n_seq=4, rows=32, mask=FAKE, words=2, q_pos=FAKE, cached=None,
            status=None, stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(n_seq=-1), 1), (dict(rows=-1), 1), (dict(rows=1 << 31), 1), (dict(words=0), 1), (dict(words=33), 2),
    (dict(parent=None), 1), (dict(cu=None), 1), (dict(total=None), 1), (dict(mask=None), 1), (dict(q_pos=None), 1),
    (dict(rows=0), 0)])
def test_maps_refuse(L, change, rc):
    assert L.sfa_build_tree_maps(*{**MAPS, **change}.values()) == rc


ACCEPT = dict(parent=FAKE, token=FAKE, target=FAKE, root=None, cu=FAKE, n_seq=4, rows=32, path=FAKE, stride=8, n_acc=FAKE,
              nxt=FAKE, status=None, stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(n_seq=-1), 1), (dict(rows=-1), 1), (dict(rows=1 << 31), 1), (dict(stride=0), 1), (dict(stride=1 << 31), 1),
    (dict(parent=None), 1), (dict(token=None), 1), (dict(target=None), 1), (dict(cu=None), 1), (dict(path=None), 1),
    (dict(n_acc=None), 1), (dict(nxt=None), 1), (dict(n_seq=0), 0)])
def test_accept_refuses(L, change, rc):
    assert L.sfa_tree_accept(*{**ACCEPT, **change}.values()) == rc


COMMIT = dict(n=1, caches=None, n_cells=640, slot=FAKE, cu=FAKE, total=FAKE, n_seq=4, rows=32, path=FAKE, stride=8,
              n_acc=FAKE, page=64, table=FAKE, width=8, free=FAKE, n_free=10, head=FAKE, len_out=FAKE, head_out=FAKE,
              status=None, stream=None)


@pytest.mark.parametrize("change,rows,rc", [
    (dict(n=-1), None, 1), (dict(n=5), None, 1), (dict(n_cells=-1), None, 1), (dict(n_cells=1 << 31), None, 1),
    (dict(n_seq=-1), None, 1), (dict(rows=-1), None, 1), (dict(stride=0), None, 1), (dict(page=0), None, 1),
    (dict(width=-1), None, 1), (dict(width=1 << 26), None, 1), (dict(n_free=-1), None, 1), (dict(n_free=1 << 31), None, 1),
    (dict(slot=None), None, 1), (dict(cu=None), None, 1), (dict(total=None), None, 1), (dict(path=None), None, 1),
    (dict(n_acc=None), None, 1), (dict(table=None), None, 1), (dict(free=None), None, 1), (dict(head=None), None, 1),
    (dict(len_out=None), None, 1), (dict(head_out=None), None, 1),
    ({}, (0, 128), 1), ({}, (0x10008, 128), 1), ({}, (0x10000, 0), 1), ({}, (0x10000, 3), 1), ({}, (0x10000, 1 << 25), 1)])
def test_commit_refuses(B, L, change, rows, rc):
    packed = B._CELL_ROWS.pack(*(rows or (0x10000, 128))) * 5
    assert L.sfa_tree_commit(*{**COMMIT, "caches": packed, **change}.values()) == rc
    assert L.sfa_tree_commit(*{**COMMIT, "caches": None}.values()) == 1


ATTEND = dict(Q=FAKE, K=FAKE, V=None, dtype=0, n_cells=640, table=FAKE, width=8, page=64, n_seq=2, n_q=20, h_q=16, h_kv=1,
              dkq=576, dv=512, scale=ctypes.c_float(0.04), cu=FAKE, total=FAKE, mask=FAKE, words=1, part=0, new_max=16,
              kv_max=500, O=FAKE, o_dtype=1, lse=None, ws=FAKE, ws_bytes=1 << 40, status=None, stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(part=1), 1), (dict(part=2), 1), (dict(part=4), 1), (dict(part=-1), 1), (dict(mask=None), 1), (dict(words=0), 1),
    (dict(new_max=33), 1), (dict(words=33, new_max=1025), 2), (dict(words=33), 2), (dict(dtype=3), 1), (dict(o_dtype=2), 1),
    (dict(Q=ODD), 1), (dict(K=None), 1), (dict(table=None), 1), (dict(cu=None), 1), (dict(total=None), 1),
    (dict(dkq=640), 2), (dict(h_q=15, h_kv=2), 1), (dict(h_q=65), 2), (dict(page=0), 1), (dict(kv_max=-1), 1),
    (dict(scale=ctypes.c_float(float("nan"))), 1), (dict(n_cells=1 << 31), 1),
    (dict(ws=None, ws_bytes=0, n_seq=1, n_q=16, width=4096, n_cells=1 << 20, kv_max=262144), 4),
    (dict(n_seq=0), 0), (dict(n_q=0), 0), (dict(new_max=0), 0)])
def test_attend_refuses(L, change, rc):
    assert L.sfa_tree_attend_paged(*{**ATTEND, **change}.values()) == rc


def test_workspace(B):
    size = lambda part, kv: B.sfa_tree_attend_workspace_bytes(B.SFA_BF16, 1, 16, 16, 1, 576, 512, False, 16, kv, part=part)
    assert size(B.SFA_PART_ALL, 262144) > size(B.SFA_PART_ALL, 128) == 0
    assert size(B.SFA_PART_DRAFTED, 262144) == 0           # one piece whatever is cached
    assert size(B.SFA_PART_WINDOW, 262144) == 0            # no part of this call


def test_binding_checks(B):
    def no(f, *a, **k):
        with pytest.raises(ValueError):
            f(*a, **k)

    maps = dict(parent=i32(9), cu_new=i32(3), len_total=i32(2), mask=i32(9, 1), q_pos=i32(9))
    for k, v in [("parent", torch.zeros(9, dtype=torch.int32)), ("parent", Fake(9, dtype=torch.int64)), ("cu_new", i32(2)),
                 ("mask", i32(8, 1)), ("mask", Fake(9, 1, dtype=torch.int64)), ("mask", i32(9)), ("q_pos", i32(8))]:
        no(B.sfa_build_tree_maps, **{**maps, k: v})
    no(B.sfa_build_tree_maps, **maps, cached_pos=i32(8))
    acc = dict(parent=i32(9), token=i32(9), target=i32(9), cu_new=i32(3), path=i32(2, 4), n_acc=i32(2), next_token=i32(2))
    for k, v in [("token", i32(8)), ("target", Fake(9, dtype=torch.int64)), ("cu_new", i32(4)), ("path", i32(3, 4)),
                 ("next_token", i32(1)), ("parent", torch.zeros(9, dtype=torch.int32))]:
        no(B.sfa_tree_accept, **{**acc, k: v})
    no(B.sfa_tree_accept, **acc, root_target=i32(1))
    com = dict(caches=[Fake(64, 1, 576)], slot=i32(9), cu_new=i32(3), path=i32(2, 4), n_acc=i32(2), len_total=i32(2),
               page_size=16, page_table=i32(2, 4), free_pages=i32(4), free_head=i32(1), len_out=i32(2), free_head_out=i32(1))
    for k, v in [("caches", [Fake(64, 1, 576)] * 5), ("caches", [Fake(64, 1, 576), Fake(63, 1, 576)]), ("cu_new", i32(2)),
                 ("caches", [Fake(64)]), ("path", i32(3, 4)), ("page_table", i32(3, 4)), ("len_out", i32(3)),
                 ("free_head", i32(2))]:
        no(B.sfa_tree_commit, **{**com, k: v})
    att = dict(Q=Fake(9, 16, 576), K=Fake(64, 1, 576), V=None, page_table=i32(2, 4), page_size=16, cu_new=i32(3),
               len_total=i32(2), tree_mask=i32(9, 1), n_new_max=5, n_kv_max=64, scale=0.1, O=f32(9, 16, 512))
    for k, v in [("tree_mask", i32(8, 1)), ("tree_mask", Fake(9, 1, dtype=torch.int64)), ("cu_new", i32(2)),
                 ("O", f32(8, 16, 512)), ("K", Fake(64, 1, 512)), ("Q", f32(9, 16, 576))]:
        no(B.sfa_tree_attend_paged, **{**att, k: v})


def test_cache_checks():
    import indexer_selected_sparse_block_gb300 as sfa
    kw = dict(n_seq=1, n_pages=4, page_size=4, max_pages=4, n_tok_cap=4, h_kv=1, dkq=64, dv=64, device="cpu")
    with pytest.raises(ValueError):
        sfa.SfaPagedCache(**kw, n_draft_max=1025)
    t = torch.zeros(4, dtype=torch.int32)
    c = sfa.SfaPagedCache(**kw)
    with pytest.raises(ValueError):
        c.draft(t[:1], t)                       # made without trees
    with pytest.raises(ValueError):
        c.commit(t, t)                          # no tree
    with pytest.raises(ValueError):
        c.step(t[:1], Q=torch.zeros(4, 1, 64))  # queries, and nothing to turn them by
    with pytest.raises(ValueError):
        sfa.SfaPagedCache(**kw, q8_0=True).step(t[:1], K=torch.zeros(4, 1, 64), rope=sfa.SfaRope(64))
    c = sfa.SfaPagedCache(**kw, n_draft_max=33)
    assert c.tree_mask.shape == (4, 2) and c.path.shape == (1, 33)
