"""Page maps and cell writes on the GPU against plain implementations, and a paged cache's whole
step: maps, writes, attention, over several steps, captured and replayed."""
import math
import random

import pytest
import torch

from paged_util import UBF, attend_reference, check_close, maps_reference

pytestmark = pytest.mark.gpu

sfa = pytest.importorskip("indexer_selected_sparse_block_gb300")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    return torch.device("cuda:0")


def run_maps(dev, old, new, page, free, head, n_pages, table, cap, n_pos=0):
    """The call on a copy of table; its outputs as lists, and the status word."""
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev).reshape(-1)
    n = len(old)
    width = len(table[0]) if table else 0
    t = torch.tensor(table, dtype=torch.int32, device=dev).reshape(n, width)
    cells = torch.full((n, n_pos), -7, dtype=torch.int32, device=dev) if n_pos else None
    out = dict(cu=i32([9] * (n + 1)), total=i32([9] * n), q_seq=i32([9] * cap), q_pos=i32([9] * cap),
               slot=i32([9] * cap), head=i32([9]))
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    sfa.sfa_build_page_maps(i32(old), i32(new), page, i32(free), i32([head]), n_pages, t, out["cu"],
                            out["total"], out["q_seq"], out["q_pos"], out["slot"], out["head"],
                            cell_of=cells, dev_status=status)
    got = {k: v.tolist() for k, v in out.items()}
    return got, t.tolist(), cells, sfa.sfa_read_device_status(status)


def check_maps(dev, old, new, page, free, head, n_pages, table, cap, status=0, n_pos=0):
    got, t, cells, st = run_maps(dev, old, new, page, free, head, n_pages, table, cap, n_pos)
    want = [list(r) for r in table]
    cu, total, q_seq, q_pos, slot, out = maps_reference(old, new, page, free, head, n_pages, want, cap)
    assert got == dict(cu=cu, total=total, q_seq=q_seq, q_pos=q_pos, slot=slot, head=[out])
    assert t == want
    if n_pos:
        expect = torch.full((len(old), n_pos), -7, dtype=torch.int32)
        for s, p, c in zip(q_seq, q_pos, slot):
            if s >= 0 and p < n_pos:
                expect[s, p] = c
        assert torch.equal(cells.cpu(), expect)
    assert st == status
    return t


def filled_table(old, page, width, order):
    table, k = [], 0
    for a in old:
        n = min(-(-a // page), width)
        table.append(order[k:k + n] + [-1] * (width - n))
        k += n
    return table, order[k:]


@pytest.mark.parametrize("n_seq,old,new,page,pad", [
    (1, 0, 1, 1, 0), (1, 0, 1, 64, 0), (1, 63, 1, 64, 3), (1, 64, 1, 64, 0), (1, 1000, 513, 16, 5),
    (3, 40, 70, 7, 0), (32, 500, 1, 64, 0), (32, 500, 40, 24, 100), (33, 0, 9, 8, 1),
    (257, 90, 20, 16, 0), (700, 30, 5, 3, 11), (1500, 12, 3, 128, 2), (6001, 9, 2, 5, 0),
    (16384, 3, 1, 2, 0), (2, 100, 20000, 48, 77),
])
def test_maps(dev, n_seq, old, new, page, pad):
    """Ragged lengths, some of them zero, from sequences of every table state."""
    r = random.Random(n_seq * 7 + old + new * 3 + page)
    a = [r.randint(0, old) for _ in range(n_seq)]
    b = [r.choice([0, new, r.randint(0, new)]) for _ in range(n_seq)]
    a[0], b[-1] = old, new
    width = max(-(-(x + y) // page) for x, y in zip(a, b)) + 1
    n_pages = sum(-(-(x + y) // page) for x, y in zip(a, b)) + 9
    order = list(range(n_pages))
    r.shuffle(order)
    table, free = filled_table(a, page, width, order)
    check_maps(dev, a, b, page, free, 0, n_pages, table, sum(b) + pad, n_pos=width * page)
    check_maps(dev, a, b, page, [0, 1] + free, 2, n_pages, table, sum(b) + pad)


def test_maps_nothing(dev):
    check_maps(dev, [], [], 16, [3], 0, 8, [], 0)
    check_maps(dev, [], [], 16, [3], 1, 8, [], 5)              # padding only
    check_maps(dev, [5, 0], [0, 0], 4, [7], 0, 8, [[1, 2], [-1, -1]], 3)
    check_maps(dev, [5, 0], [0, 0], 4, [], 0, 8, [[1, 2], [-1, -1]], 0)


def test_maps_free_list_runs_out(dev):
    """Sequence 0 takes two pages of three, sequence 1 lacks one; what it has is used."""
    no = sfa.SFA_DEV_NO_PAGES
    t = check_maps(dev, [0, 3], [7, 10], 4, [5, 6, 7], 0, 8, [[-1] * 4, [0] + [-1] * 3], 20,
                   status=no)
    assert t == [[5, 6, -1, -1], [0, 7, -1, -1]]
    check_maps(dev, [0], [9], 4, [5, 6, 7], 3, 8, [[-1] * 4], 9, status=no)
    check_maps(dev, [0], [9], 4, [], 0, 8, [[-1] * 4], 9, status=no)
    check_maps(dev, [0], [9], 4, [2, -1, 3], 0, 8, [[-1] * 4], 9, status=no)   # a hole in the list


def test_maps_bad_entries(dev):
    bad = sfa.SFA_DEV_BAD_CELL
    check_maps(dev, [0], [9], 4, [2, 8, 3], 0, 8, [[-1] * 4], 9, status=bad)   # a free page beyond
    check_maps(dev, [5], [2], 4, [2], 0, 8, [[1, 8]], 2, status=bad)           # the partly filled page
    check_maps(dev, [5], [2], 4, [2], 0, 8, [[1, -3]], 2, status=bad)


def test_maps_lengths_beyond(dev):
    bad = sfa.SFA_DEV_BAD_LENGTH
    check_maps(dev, [-4, 2], [3, -1], 4, [0, 1, 2], 0, 8, [[-1] * 2, [5, -1]], 6, status=bad)
    check_maps(dev, [3, 0], [9, 2], 4, [0, 1, 2], 0, 8, [[6, -1], [-1, -1]], 12, status=bad)   # table
    check_maps(dev, [0, 0, 0], [4, 5, 6], 4, [0, 1, 2, 3, 4], 0, 8, [[-1] * 3] * 3, 6, status=bad)
    check_maps(dev, [0], [2 ** 31 - 1], 4, [0], 0, 8, [[-1]], 3, status=bad)
    check_maps(dev, [2 ** 31 - 1], [0], 4, [0], 0, 8, [[-1]], 3, status=bad)
    check_maps(dev, [0], [6], 4, [0, 1], 0, 8, [[-1, -1]], 6, n_pos=5, status=bad)             # map
    check_maps(dev, [0], [6], 4, [0, 1], -3, 8, [[-1, -1]], 6)                 # a head before the list


# -------------------------------------------------------------------------------------- writes
def plain_q8(x):
    """q8_0 rows of x [..][d] (fp32), by the rule in include/sfa.h."""
    d = x.shape[-1]
    b = x.reshape(x.shape[:-1] + (d // 32, 32))
    delta = b.abs().amax(-1) / 127.0
    q = torch.where(delta[..., None] == 0, torch.zeros_like(b), b / delta[..., None])
    q = (torch.sign(q) * torch.floor(q.abs() + 0.5)).to(torch.int8)
    rb = sfa.sfa_q8_0_row_bytes(d)
    out = torch.zeros(x.shape[:-1] + (rb,), dtype=torch.uint8)
    out[..., :d] = q.reshape(x.shape).view(torch.uint8)
    out[..., d:d + d // 16] = delta.to(torch.float16).view(torch.uint8)
    return out


def as_cache(x, dst):
    return plain_q8(x.float()) if dst == "q8" else x.to(dst)


@pytest.mark.parametrize("src,dst", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                     (torch.float32, torch.bfloat16), (torch.bfloat16, "q8"),
                                     (torch.float32, "q8")])
@pytest.mark.parametrize("rows,h,d", [(1, 1, 576), (9, 2, 64), (200, 1, 512), (3001, 4, 128),
                                      (33, 1, 5), (17, 3, 100), (64, 1, 1)])
def test_write(dev, src, dst, rows, h, d):
    if dst == "q8" and d not in (64, 128, 512, 576):
        pytest.skip("no q8_0 row of this length")
    g = torch.Generator().manual_seed(rows + d)
    n_cells = rows + 40
    x = torch.randn((rows, h, d), generator=g).to(src)
    if dst == "q8":
        x[0] = 0                                     # a zero block
    slot = torch.randperm(n_cells, generator=g)[:rows].to(torch.int32)
    slot[rows // 2] = -1                             # a token without a cell
    base = as_cache(torch.randn((n_cells, h, d), generator=g), dst)
    for stride in (1, 2):                            # packed rows, and rows apart
        wide = torch.full((rows, stride * h, d), 3.0, dtype=src)
        wide[:, :h] = x
        xs = wide.to(dev)[:, :h]
        cache = base.to(dev)
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        sfa.sfa_write_cells([(xs, cache)], slot.to(dev), dev_status=status)
        want = base.clone()
        live = slot >= 0
        want[slot[live].long()] = as_cache(x, dst)[live]
        assert torch.equal(cache.cpu(), want)
        assert sfa.sfa_read_device_status(status) == 0


def test_write_several_caches(dev):
    """K, V and the index keys of a step in one launch, two-dimensional rows among them, and an
    unaligned source."""
    g = torch.Generator().manual_seed(5)
    n, cells = 77, 130
    slot = torch.randperm(cells, generator=g)[:n].to(torch.int32)
    K = torch.randn((n, 2, 512), generator=g)
    V = torch.randn((n, 2, 512), generator=g).to(torch.bfloat16)
    X = torch.randn((n + 1, 129), generator=g)[:, 1:]          # rows 4 bytes off a boundary
    Y = torch.randn((n, 64), generator=g)
    caches = [torch.zeros((cells, 2, 512), dtype=torch.bfloat16), torch.zeros((cells, 2, 512), dtype=torch.bfloat16),
              torch.zeros((cells, 128)), torch.zeros((cells, 64), dtype=torch.bfloat16)]
    c = [t.to(dev) for t in caches]
    xd = torch.zeros((n + 1, 129), device=dev)
    xd[:, 1:] = X.to(dev)
    sfa.sfa_write_cells([(K.to(dev), c[0]), (V.to(dev), c[1]), (xd[:, 1:], c[2]), (Y.to(dev), c[3])],
                        slot.to(dev))
    for got, want, rows in zip(c, caches, (K, V, X[:n], Y)):
        want[slot.long()] = rows.to(want.dtype)
        assert torch.equal(got.cpu(), want)


def test_write_bad_slots(dev):
    x = torch.ones((4, 1, 64), device=dev)
    cache = torch.zeros((8, 1, 64), device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    slot = torch.tensor([8, -2 ** 31, 3, 2 ** 31 - 1], dtype=torch.int32, device=dev)
    sfa.sfa_write_cells([(x, cache)], slot, dev_status=status)
    assert cache.sum(dim=(1, 2)).tolist() == [0, 0, 0, 64, 0, 0, 0, 0]
    assert sfa.sfa_read_device_status(status) == sfa.SFA_DEV_BAD_CELL
    big = torch.full((1, 1, 64), 1e10, device=dev)
    q8 = torch.zeros((8, 1, 80), dtype=torch.uint8, device=dev)
    status.zero_()
    sfa.sfa_write_cells([(big, q8)], slot[2:3], dev_status=status)
    assert sfa.sfa_read_device_status(status) == sfa.SFA_DEV_FP16_RANGE


# -------------------------------------------------------------------------- the step as a whole
def host_table(cache):
    return cache.page_table.tolist()


@pytest.mark.parametrize("dkq,dv,h_q,h_kv,sep,page", [(576, 512, 16, 1, False, 8), (128, 128, 8, 2, True, 6)])
def test_cache_steps(dev, dkq, dv, h_q, h_kv, sep, page):
    """Prefill, mixed and decode steps of a paged cache: after each, the attention of the new
    tokens over everything written so far against the plain one on the host's own record."""
    g = torch.Generator().manual_seed(dkq)
    n_seq, cap = 3, 40
    steps = [[13, 0, 7], [1, 9, 1], [1, 1, 1], [0, 22, 1]]
    c = sfa.SfaPagedCache(n_seq=n_seq, n_pages=40, page_size=page, max_pages=16, n_tok_cap=cap,
                          h_kv=h_kv, dkq=dkq, dv=dv, separate_v=sep, d_idx=64)
    c.K.fill_(float("nan"))                          # cells no token was written to
    perm = torch.randperm(40, generator=g).to(torch.int32)
    c.free_pages.copy_(perm)
    rows = {s: ([], []) for s in range(n_seq)}
    scale = 1 / math.sqrt(dkq)
    for new in steps:
        K = torch.randn((cap, h_kv, dkq), generator=g).to(torch.bfloat16)
        V = torch.randn((cap, h_kv, dv), generator=g).to(torch.bfloat16) if sep else None
        X = torch.randn((cap, 64), generator=g).to(torch.bfloat16)
        Q = torch.randn((cap, h_q, dkq), generator=g).to(torch.bfloat16)
        c.step(torch.tensor(new, dtype=torch.int32, device=dev), K.to(dev),
               None if V is None else V.to(dev), X.to(dev))
        O = torch.full((cap, h_q, dv), 5.0, device=dev)
        c.attend(Q.to(dev), cap, 100, scale, O)
        at = 0
        for s, n in enumerate(new):
            for j in range(at, at + n):
                rows[s][0].append(K[j])
                rows[s][1].append(V[j] if sep else K[j][:, :dv])
            at += n
        # the plain form on the host's rows: one page a sequence
        lens = [len(rows[s][0]) for s in range(n_seq)]
        P = max(lens)
        zero = torch.zeros((h_kv, dkq), dtype=torch.bfloat16)
        Kh = torch.stack([x for s in range(n_seq) for x in rows[s][0] + [zero] * (P - lens[s])])
        Vh = torch.stack([x for s in range(n_seq) for x in rows[s][1] + [zero[:, :dv]] * (P - lens[s])])
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        ref, _, tol, _ = attend_reference(Q[:at], Kh, Vh, [[s] for s in range(n_seq)], P, cu, lens,
                                          scale, dv, p_round=UBF ** 2)
        check_close(O[:at], ref, tol, f"step {new}")
        assert bool((O[at:] == 5.0).all())           # rows of no chunk
        assert c.length.tolist() == lens
        # the index keys and the per-position map: position t of every sequence
        m, t = c.cell_of.cpu(), torch.tensor(host_table(c))
        for s in range(n_seq):
            for pos in range(lens[s]):
                assert int(m[s, pos]) == int(t[s, pos // page]) * page + pos % page
    assert sfa.sfa_read_device_status(c.status) == 0
    used = {p for r in host_table(c) for p in r if p >= 0}
    c.release(1)
    assert host_table(c)[1] == [-1] * 16 and int(c.length[1]) == 0
    free = c.free_pages[int(c.free_head):].tolist()
    held = {p for r in host_table(c) for p in r if p >= 0}
    assert sorted(free) == sorted(set(range(40)) - held) and held < used


def test_cell_map_feeds_the_sparse_step(dev):
    """SfaStep on the cache's cells through its cell_of: bit for bit what it gives on a cell map
    made on the host."""
    n_seq, n_tok, page = 2, 700, 16
    w = sfa.WORKLOADS["decode_1x4096"].with_(n_seq=n_seq, depth=n_tok - 1, seed=3)
    case = sfa.make_case(w, device=dev)
    c = sfa.SfaPagedCache(n_seq=n_seq, n_pages=200, page_size=page, max_pages=44, n_tok_cap=n_seq * n_tok,
                          h_kv=1, dkq=576, dv=512, d_idx=64)
    c.free_pages.copy_(torch.randperm(200, generator=torch.Generator().manual_seed(1)).to(torch.int32))
    c.step(torch.full((n_seq,), n_tok, dtype=torch.int32, device=dev),
           case["K"].reshape(-1, 1, 576), None, case["X"].reshape(-1, 64))
    cell_of = c.cell_of[:, :n_tok].contiguous()
    outs = []
    host_map, n_cells = sfa.make_cell_map(n_seq, n_tok, page, seed=9, device=dev)
    for m, X, K in ((cell_of, c.X, c.K),
                    (host_map, sfa.to_cells(case["X"], host_map, n_cells),
                     sfa.to_cells(case["K"], host_map, n_cells))):
        step = sfa.SfaStep(n_seq=n_seq, n_tok_cap=n_tok, n_q=n_seq, h_q=16, h_kv=1, dkq=576, dv=512,
                           h_idx=4, d_idx=64, compress_ratio=4, indexer_top_k=32, n_blk_max=n_tok // 4,
                           cell_of=m)
        O = step.run(X, K, None, case["Q"], case["q_idx"], case["w"], case["q_seq"], case["q_pos"],
                     w.scale, new_blocks=(0, n_tok // 4))
        outs.append((O.clone(), step.blk_idx.clone()))
        assert sfa.sfa_read_device_status(step.status) == 0
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert sfa.sfa_read_device_status(c.status) == 0


def test_step_replays_as_a_graph(dev):
    """A captured step (maps, writes, attention) replayed with other lengths and rows gives what
    the eager step gives, bit for bit; two caches' graphs of one shape do not disturb each other."""
    g = torch.Generator().manual_seed(8)
    n_seq, cap, kvm = 4, 24, 200
    scale = 1 / math.sqrt(576)
    lens = [[5, 0, 9, 1], [1, 1, 1, 1], [0, 12, 3, 2], [1, 1, 1, 1]]
    data = [(torch.randn((cap, 1, 576), generator=g).to(torch.bfloat16).to(dev),
             torch.randn((cap, 16, 576), generator=g).to(torch.bfloat16).to(dev)) for _ in lens]

    def make():
        return sfa.SfaPagedCache(n_seq=n_seq, n_pages=64, page_size=8, max_pages=25, n_tok_cap=cap,
                                 h_kv=1, dkq=576, dv=512, cell_map=False)

    need = sfa.sfa_chunk_attend_workspace_bytes(sfa.SFA_BF16, n_seq, cap, 16, 1, 576, 512, False,
                                                cap, kvm)
    eager, want = make(), []
    for new, (K, Q) in zip(lens, data):
        O = torch.zeros((cap, 16, 512), device=dev)
        eager.step(torch.tensor(new, dtype=torch.int32, device=dev), K)
        eager.attend(Q, cap, kvm, scale, O)
        want.append(O)
    graphs = []
    for _ in range(2):
        c = make()
        buf = dict(n=torch.zeros(n_seq, dtype=torch.int32, device=dev), K=torch.zeros_like(data[0][0]),
                   Q=torch.zeros_like(data[0][1]), O=torch.zeros((cap, 16, 512), device=dev),
                   ws=torch.empty(max(need, 16), dtype=torch.uint8, device=dev))

        def one(c=c, buf=buf):
            c.step(buf["n"], buf["K"])
            c.attend(buf["Q"], cap, kvm, scale, buf["O"], workspace=buf["ws"])

        graphs.append((sfa.SfaStep.graphed(one), c, buf))   # warm-up: no tokens, nothing moves
    for i, (new, (K, Q)) in enumerate(zip(lens, data)):
        for graph, c, buf in graphs:
            buf["n"].copy_(torch.tensor(new, dtype=torch.int32))
            buf["K"].copy_(K)
            buf["Q"].copy_(Q)
            buf["O"].zero_()
            graph.replay()
        for graph, c, buf in graphs:
            assert torch.equal(buf["O"], want[i]), i
            assert sfa.sfa_read_device_status(c.status) == 0
            assert c.page_table.tolist() == graphs[0][1].page_table.tolist()
