"""The paged-serving entry points on the host: refusals before anything is enqueued, the size
query, and the binding's checks."""
import ctypes

import pytest
import torch

FAKE = ctypes.c_void_p(0x10000)     # never dereferenced: every call below is rejected first
FAKE2 = ctypes.c_void_p(0x20000)
ODD = ctypes.c_void_p(0x10008)      # not 16-byte aligned


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    from indexer_selected_sparse_block_gb300 import _binding
    return _binding.lib()


MAPS = dict(old=FAKE, new=FAKE, n_seq=4, page=64, free=FAKE, n_free=10, head=FAKE, n_pages=20,
            table=FAKE, width=8, cu=FAKE, total=FAKE2, q_seq=FAKE, q_pos=FAKE, slot=FAKE, cap=32,
            cells=None, n_pos=0, out=FAKE2, status=None, stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(n_seq=-1), 1), (dict(page=0), 1), (dict(n_free=-1), 1), (dict(n_pages=-1), 1),
    (dict(width=-1), 1), (dict(cap=-1), 1), (dict(cap=1 << 31), 1), (dict(n_free=1 << 31), 1),
    (dict(n_pos=-1), 1), (dict(cu=None), 1), (dict(head=None), 1), (dict(out=None), 1),
    (dict(out=FAKE), 1),                       # the head may not be read and written in place
    (dict(total=FAKE), 1),                     # nor the lengths
    (dict(old=None), 1), (dict(new=None), 1), (dict(total=None), 1), (dict(table=None), 1),
    (dict(free=None), 1), (dict(q_seq=None), 1), (dict(q_pos=None), 1), (dict(slot=None), 1),
    (dict(n_pages=1 << 26), 1),                # cells beyond 2^31
    (dict(width=1 << 26), 1),                  # positions beyond 2^31
    (dict(width=1 << 40), 1),
    (dict(n_seq=16385), 2),
])
def test_maps_refuse(L, change, rc):
    assert L.sfa_build_page_maps(*{**MAPS, **change}.values()) == rc


def _write(**kw):
    from indexer_selected_sparse_block_gb300._binding import _CellWrite
    d = dict(src=0x10000, src_stride=128, dst=0x20000, src_dtype=0, dst_dtype=0, n_inner=2, d=64)
    d.update(kw)
    return _CellWrite(*d.values())


@pytest.mark.parametrize("change,rc", [
    (dict(src=None), 1), (dict(dst=None), 1), (dict(dst=0x20008), 1), (dict(src=0x10001), 1),
    (dict(src_dtype=2), 1), (dict(src_dtype=-1), 1), (dict(dst_dtype=3), 1), (dict(n_inner=0), 1),
    (dict(d=0), 1), (dict(src_stride=127), 1), (dict(n_inner=1 << 20, d=1 << 20), 1),
    (dict(dst_dtype=1), 2),                    # bf16 rows into an fp32 cache
    (dict(dst_dtype=2, n_inner=1, d=96), 2),   # a q8_0 row length without a format
])
def test_write_refuses(L, change, rc):
    from indexer_selected_sparse_block_gb300._binding import _CellWrite
    arr = (_CellWrite * 2)(_write(), _write(**change))
    assert L.sfa_write_cells(2, ctypes.cast(arr, ctypes.c_void_p), FAKE, 5, 100, None, None) == rc


def test_write_refuses_lists(L):
    from indexer_selected_sparse_block_gb300._binding import SFA_MAX_CELL_WRITES, _CellWrite
    arr = ctypes.cast((_CellWrite * 1)(_write()), ctypes.c_void_p)
    f = L.sfa_write_cells
    assert f(-1, arr, FAKE, 5, 100, None, None) == 1
    assert f(SFA_MAX_CELL_WRITES + 1, arr, FAKE, 5, 100, None, None) == 1
    assert f(1, None, FAKE, 5, 100, None, None) == 1
    assert f(1, arr, None, 5, 100, None, None) == 1
    assert f(1, arr, FAKE, -1, 100, None, None) == 1
    assert f(1, arr, FAKE, 5, 1 << 31, None, None) == 1
    assert f(1, arr, FAKE, 0, 100, None, None) == 0           # no rows: no work
    assert f(0, None, None, 5, 100, None, None) == 0


ATT = dict(Q=FAKE, K=FAKE, V=None, dtype=0, n_cells=6400, table=FAKE, width=100, page=64, n_seq=2,
           n_q=10, h_q=16, h_kv=1, dkq=576, dv=512, scale=ctypes.c_float(0.04), cu=FAKE, total=FAKE,
           new_max=10, kv_max=6000, O=FAKE, o_dtype=0, lse=None, ws=FAKE, ws_bytes=1 << 40,
           status=None, stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(dtype=3), 1), (dict(o_dtype=2), 1), (dict(n_seq=-1), 1), (dict(n_q=-1), 1),
    (dict(h_q=12, h_kv=5), 1), (dict(h_kv=0), 1), (dict(new_max=-1), 1), (dict(kv_max=-1), 1),
    (dict(kv_max=1 << 31), 1), (dict(page=0), 1), (dict(width=-1), 1), (dict(width=1 << 26), 1),
    (dict(n_cells=-1), 1), (dict(n_cells=1 << 31), 1),
    (dict(scale=ctypes.c_float(float("nan"))), 1), (dict(scale=ctypes.c_float(float("inf"))), 1),
    (dict(Q=None), 1), (dict(K=None), 1), (dict(table=None), 1), (dict(cu=None), 1),
    (dict(total=None), 1), (dict(O=None), 1), (dict(Q=ODD), 1), (dict(K=ODD), 1), (dict(O=ODD), 1),
    (dict(lse=ODD), 1), (dict(ws=ODD), 1),
    (dict(dkq=576, dv=576), 2), (dict(dkq=320, dv=256), 2), (dict(V=FAKE), 2),
    (dict(dkq=64, dv=128), 1),                 # V = K with more value dims than K has
    (dict(h_q=65, h_kv=1), 2),
    (dict(ws=None), 4), (dict(ws_bytes=100), 4),
    (dict(n_seq=0), 0), (dict(n_q=0), 0), (dict(new_max=0), 0),      # nothing to do
])
def test_attend_refuses(L, change, rc):
    assert L.sfa_chunk_attend_paged(*{**ATT, **change}.values()) == rc


def test_workspace_query(L):
    from indexer_selected_sparse_block_gb300 import sfa_chunk_attend_workspace_bytes as ws
    assert ws(0, 1, 1, 16, 1, 576, 512, False, 1, 4097) > 0           # a split decode list
    assert ws(0, 1, 1, 16, 1, 576, 512, False, 1, 1) == 0             # one key: no split
    assert ws(0, 0, 0, 16, 1, 576, 512, False, 1, 100) == 0
    assert ws(0, 1, 1, 16, 1, 100, 100, False, 1, 100) == 0           # a refused shape


def test_binding_refuses(L):
    """What the binding checks before the library is called (CPU tensors never get there)."""
    import indexer_selected_sparse_block_gb300 as sfa
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    args = lambda **k: {**dict(len_old=i(2), len_new=i(2), page_size=4, free_pages=i(3),
                               free_head=i(1), n_pages=8, page_table=i(2, 5), cu_new=i(3),
                               len_total=i(2), q_seq=i(6), q_pos=i(6), slot=i(6),
                               free_head_out=i(1)), **k}
    for bad in (dict(len_new=i(3)), dict(cu_new=i(2)), dict(q_seq=i(5)), dict(free_head=i(2)),
                dict(page_table=i(3, 5)), dict(slot=torch.zeros(6)), dict(cell_of=i(3, 9)),
                dict(len_old=i(4)[::2]), {}):
        with pytest.raises(ValueError):
            sfa.sfa_build_page_maps(**args(**bad))
    x, y = torch.zeros(6, 2, 64), torch.zeros(12, 2, 64)
    for pairs in ([(x, y[:, :1])], [(x[:5], y)], [(x.transpose(1, 2), y)], [(x, y[:, :, :32])],
                  [(x, y)] * 5, [(x, y)]):
        with pytest.raises(ValueError):
            sfa.sfa_write_cells(pairs, i(6))
    b = torch.bfloat16
    att = lambda **k: {**dict(Q=torch.zeros(6, 16, 64, dtype=b), K=torch.zeros(32, 2, 64, dtype=b),
                              V=None, page_table=i(2, 4), page_size=4, cu_new=i(3), len_total=i(2),
                              n_new_max=3, n_kv_max=16, scale=0.1, O=torch.zeros(6, 16, 64)), **k}
    for bad in (dict(K=torch.zeros(32, 2, 128, dtype=b)), dict(K=torch.zeros(32, 2, 64)),
                dict(V=torch.zeros(31, 2, 64, dtype=b)), dict(cu_new=i(2)), dict(page_table=i(3, 4)),
                dict(O=torch.zeros(5, 16, 64)), dict(O=torch.zeros(6, 16, 64, dtype=torch.float16)),
                dict(lse=torch.zeros(6, 15)), dict(len_total=torch.zeros(2)), {}):
        with pytest.raises(ValueError):
            sfa.sfa_chunk_attend_paged(**att(**bad))
