"""Attention of chunks of new tokens over a paged cache, against the plain 64-bit form within
bounds that follow from the arithmetic (paged_util.attend_reference)."""
import math
import random

import pytest
import torch

from paged_util import UBF, attend_reference, check_close

pytestmark = pytest.mark.gpu

sfa = pytest.importorskip("indexer_selected_sparse_block_gb300")

# Weights reach the value products as two bf16 halves for fp32 results (half a step of the second
# half: UBF^2) and as one bf16 value for bf16 results; fp32 caches keep them in fp32.
P_ROUND = {("bf16", "f32"): UBF ** 2, ("bf16", "bf16"): UBF, ("f32", "f32"): 0.0, ("f32", "bf16"): 0.0,
           ("q8", "f32"): 0.0, ("q8", "bf16"): 0.0}
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    return torch.device("cuda:0")


class Case:
    """lens: (cached before, new) per sequence; the cells that hold no token are NaN."""

    def __init__(self, dev, lens, page, shape, dtype="bf16", out="f32", seed=0, spare_q=0, kscale=1.0,
                 scale=None, spare_pages=3):
        self.dkq, self.dv, self.sep, self.h_q, self.h_kv = shape
        self.lens, self.page, self.dtype, self.out, self.dev = lens, page, dtype, out, dev
        g = torch.Generator().manual_seed(seed)
        self.total = [a + n for a, n in lens]
        self.cu = [0]
        for _, n in lens:
            self.cu.append(self.cu[-1] + n)
        pages = [-(-t // page) for t in self.total]
        n_pages = sum(pages) + spare_pages
        order = torch.randperm(n_pages, generator=g).tolist()
        width = max(pages + [1]) + 1
        self.table, k = [], 0
        for n in pages:
            self.table.append(order[k:k + n] + [-1] * (width - n))
            k += n
        dt = TYPES.get(dtype, torch.float32)
        draw = lambda d, f=1.0: (torch.randn((n_pages * page, self.h_kv, d), generator=g) * f).to(torch.bfloat16).to(dt)
        self.K, self.V = draw(self.dkq, kscale), draw(self.dv) if self.sep else None
        live = torch.zeros(n_pages * page, dtype=torch.bool)
        for s, t in enumerate(self.total):
            for pos in range(t):
                live[self.table[s][pos // page] * page + pos % page] = True
        n_q = self.cu[-1] + spare_q
        self.Q = torch.randn((n_q, self.h_q, self.dkq), generator=g).to(torch.bfloat16)
        self.Q[self.cu[-1]:] = float("nan")
        self.scale = 1 / math.sqrt(self.dkq) if scale is None else scale
        if dtype == "q8":
            self.Kc, self.K = self._q8(self.K)
            if self.sep:
                self.Vc, self.V = self._q8(self.V)
            else:
                self.Vc = None
        else:
            if dtype == "f32":
                self.Q = self.Q.float()
            for t in (self.K, self.V):
                if t is not None:
                    t[~live] = float("nan")
            self.Kc, self.Vc = self.K.to(dev), None if self.V is None else self.V.to(dev)

    def _q8(self, x):
        """The q8_0 rows of x on the device and the values they stand for."""
        x = x.to(self.dev)
        d = x.shape[-1]
        y = torch.zeros(x.shape[:-1] + (sfa.sfa_q8_0_row_bytes(d),), dtype=torch.uint8, device=self.dev)
        sfa.sfa_quantize_kv_q8_0(x, y)
        codes = y[..., :d].contiguous().view(torch.int8).float()
        sc = y[..., d:d + d // 16].contiguous().view(torch.float16).float()
        return y, (codes * sc.repeat_interleave(32, -1)).cpu()

    def call(self, n_new_max=None, n_kv_max=None, stream=None, table=None, cu=None, total=None, lse=True,
             workspace=None):
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=self.dev)
        n_q = self.Q.shape[0]
        self.O = torch.full((n_q, self.h_q, self.dv), 7.0, dtype=TYPES[self.out], device=self.dev)
        self.lse = torch.full((n_q, self.h_q), 7.0, device=self.dev) if lse else None
        status = torch.zeros(1, dtype=torch.int32, device=self.dev)
        args = (self.Q.to(self.dev), self.Kc, self.Vc, i32(table or self.table), self.page, i32(cu or self.cu),
                i32(total or self.total))
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        sfa.sfa_chunk_attend_paged(*args,
                                   max([n for _, n in self.lens] + [1]) if n_new_max is None else n_new_max,
                                   max(self.total + [1]) if n_kv_max is None else n_kv_max, self.scale,
                                   self.O, lse=self.lse, dev_status=status, stream=stream,
                                   workspace=workspace)
        if stream is not None:
            torch.cuda.current_stream().wait_stream(stream)
        torch.cuda.synchronize()
        return sfa.sfa_read_device_status(status)

    def check(self, table=None, kv_max=None, cu=None, total=None):
        cu = cu or self.cu
        ref, ref_l, tol, tol_l = attend_reference(
            self.Q, self.K, self.V, table or self.table, self.page, cu, total or self.total, self.scale,
            self.dv, kv_max=kv_max, p_round=P_ROUND[self.dtype, self.out],
            o_round=UBF if self.out == "bf16" else 0.0)
        n = self.cu[-1]
        check_close(self.O[:n], ref[:n], tol[:n], "O")
        if self.lse is not None:
            check_close(self.lse[:n], ref_l[:n], tol_l[:n], "lse")
            assert bool((self.lse[n:] == 7.0).all())
        assert bool((self.O[n:].float() == 7.0).all())


WIDE, W512, W512K = (576, 512, False, 16, 1), (512, 512, True, 16, 2), (512, 512, False, 16, 1)
N128, N128K, N64, N64K = (128, 128, True, 16, 4), (128, 128, False, 4, 4), (64, 64, True, 8, 1), (64, 64, False, 8, 2)
SHAPES = [WIDE, W512, W512K, N128, N128K, N64, N64K]
RAGGED = [(0, 1), (0, 17), (5, 3), (127, 1), (128, 40), (0, 0), (255, 2), (300, 0), (61, 70)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("dtype", ["bf16", "f32", "q8"])
@pytest.mark.parametrize("shape", SHAPES)
def test_ragged(dev, shape, dtype, out):
    """Every shape and type: one to many new tokens, empty chunks, sequences of one token, lengths
    on and off the tiles' and pages' edges, unused rows of Q."""
    c = Case(dev, RAGGED, 16, shape, dtype, out, seed=shape[0], spare_q=5)
    assert c.call() == 0
    c.check()


@pytest.mark.parametrize("shape", [WIDE, N128])
@pytest.mark.parametrize("page", [1, 2, 3, 8, 24, 40, 64, 96, 100, 128, 192, 256, 1000])
def test_page_sizes(dev, shape, page):
    """Pages smaller and larger than a tile, ending inside one or not, odd ones."""
    c = Case(dev, [(0, 3), (190, 20), (500, 1), (130, 9)], page, shape, seed=page)
    assert c.call() == 0
    c.check()


@pytest.mark.parametrize("shape", [WIDE, W512, N128, N64])
@pytest.mark.parametrize("length", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 193, 255, 256, 257, 511, 900])
def test_single_tokens(dev, shape, length):
    """Decode: one new token behind every length around a tile's edges."""
    c = Case(dev, [(length - 1, 1)], 64, shape, seed=length)
    assert c.call() == 0
    c.check()


@pytest.mark.parametrize("shape", [(576, 512, False, h, k) for h, k in
                                   [(1, 1), (3, 1), (12, 1), (15, 3), (33, 1), (64, 1), (32, 2)]]
                         + [(128, 128, True, h, k) for h, k in [(1, 1), (5, 1), (48, 1), (6, 2), (7, 7), (64, 1)]]
                         + [(64, 64, True, 20, 2), (64, 64, True, 63, 1), (512, 512, True, 24, 2)])
def test_head_groups(dev, shape):
    """Query heads per KV head that do and do not divide a tile's rows."""
    c = Case(dev, [(70, 19), (3, 1), (0, 45)], 16, shape, seed=shape[3])
    assert c.call() == 0
    c.check()


@pytest.mark.parametrize("shape,new", [(WIDE, 1), (WIDE, 3), (N128, 1), (N64, 2), (W512, 1)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_long_split_lists(dev, shape, new, out):
    """Few rows against a long list: it is cut over the SMs and merged; the same on every run."""
    c = Case(dev, [(6000, new), (37, new), (2049, new)], 32, shape, out=out, seed=new)
    need = sfa.sfa_chunk_attend_workspace_bytes(sfa.SFA_BF16, 3, 3 * new, shape[3], shape[4], shape[0],
                                                shape[1], shape[2], new, 6000 + new)
    assert need > 0                       # the plan really splits
    assert c.call() == 0
    c.check()
    O, lse = c.O, c.lse
    ws = torch.full((need,), 255, dtype=torch.uint8, device=dev)       # NaN everywhere
    assert c.call(workspace=ws) == 0
    assert torch.equal(c.O, O) and torch.equal(c.lse, lse)


@pytest.mark.parametrize("shape,dtype", [(WIDE, "bf16"), (N128, "bf16"), (N64, "bf16"), (W512, "bf16"), (N128, "f32")])
def test_rising_scores(dev, shape, dtype):
    """Each key scores higher than all before it, by much: every tile moves the running maximum."""
    c = Case(dev, [(700, 40)], 64, shape, dtype, seed=4)
    g = shape[3] // shape[4]
    q = torch.sign(c.Q[:, ::g].float().mean(0, keepdim=True)) + 0.0
    q[q == 0] = 1.0
    c.Q = q.repeat_interleave(g, 1).expand(c.Q.shape).contiguous().to(c.Q.dtype)
    ramp = torch.arange(740).float() / 740 * 4
    for pos in range(740):
        cell = c.table[0][pos // 64] * 64 + pos % 64
        c.K[cell] = (q[0, :, :] * ramp[pos]).to(c.K.dtype)
    c.Kc = c.K.to(dev)
    c.scale = 1.0                         # scores up to 4 dkq in steps of dkq / 185
    assert c.call() == 0
    c.check()


def test_large_and_negative_scores(dev):
    """Scores of hundreds, a negative scale, and a zero one (a plain mean)."""
    for scale in (3.0, -0.5, 0.0):
        for shape in (WIDE, N128):
            c = Case(dev, [(150, 20), (0, 1)], 16, shape, seed=6, scale=scale)
            assert c.call() == 0
            c.check()


@pytest.mark.parametrize("shape", [WIDE, W512, N128, N64])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_pages(dev, shape, dtype):
    """Page table entries that are no page: their positions are left out, a query that sees no
    other gets zeros, and the status says so."""
    c = Case(dev, [(0, 20), (150, 30), (64, 1)], 16, shape, dtype, seed=2)
    t = [list(r) for r in c.table]
    t[0][0] = -1                      # the first 16 queries of sequence 0 see nothing
    t[1][3] = len(c.K) // 16          # one past the last page
    t[1][9], t[2][4] = -2 ** 31, 2 ** 31 - 1
    assert c.call(table=t) == sfa.SFA_DEV_BAD_CELL
    c.check(table=t)
    assert bool((c.O[:16] == 0).all()) and bool(torch.isneginf(c.lse[:16]).all())


@pytest.mark.parametrize("shape,dtype", [(WIDE, "bf16"), (N128, "bf16"), (N64, "f32")])
def test_bounds_that_do_not_hold(dev, shape, dtype):
    """Host bounds and offsets that the device data breaks: flagged, what fits is computed, no row
    outside is touched."""
    bad = sfa.SFA_DEV_BAD_QUERY
    c = Case(dev, [(100, 30), (20, 4)], 16, shape, dtype, seed=3)
    assert c.call(n_kv_max=64) == bad                 # longer lists: their first 64 keys
    c.check(kv_max=64)
    assert c.call(n_new_max=8) == bad                 # a longer chunk: its first 8 queries
    ref, _, tol, _ = attend_reference(c.Q, c.K, c.V, c.table, 16, c.cu, c.total, c.scale, c.dv,
                                      p_round=P_ROUND[dtype, "f32"])
    for r in (slice(0, 8), slice(30, 34)):
        check_close(c.O[r], ref[r], tol[r], "O")
    assert bool((c.O[8:30] == 7.0).all())
    assert c.call(cu=[0, 30, 35]) == bad              # past the last row: an empty chunk
    check_close(c.O[:30], ref[:30], tol[:30], "O")
    assert bool((c.O[30:] == 7.0).all())
    assert c.call(cu=[0, 30, 29]) == bad
    check_close(c.O[:30], ref[:30], tol[:30], "O")
    assert bool((c.O[30:] == 7.0).all())
    assert c.call(total=[10, 24]) == bad              # fewer tokens than the chunk: 20 queries before 0
    c.check(total=[10, 24])
    assert bool((c.O[:20] == 0).all()) and bool(torch.isneginf(c.lse[:20]).all())
    short = [r[:5] for r in c.table]                  # 80 positions of 130
    assert c.call(table=short) == bad
    c.check(table=short)


def test_nonfinite_values(dev):
    """NaN and infinities in attended cells reach the rows that attend them and no others."""
    for shape, dtype in ((WIDE, "f32"), (N128, "f32")):
        c = Case(dev, [(100, 30), (5, 3)], 16, shape, dtype, seed=9)
        cell = c.table[0][110 // 16] * 16 + 110 % 16          # query 10 of the chunk: a later key
        v = c.K if c.V is None else c.V
        v[cell, :, 3] = float("inf")
        c.Kc, c.Vc = c.K.to(dev), None if c.V is None else c.V.to(dev)
        assert c.call() == 0
        O = c.O.float()
        assert bool(torch.isfinite(O[:10]).all()) and bool(torch.isfinite(O[30:]).all())
        # where V is K's first dims the key's score is +-inf with the sign of q[3]: -inf is weight
        # exp(-inf) = 0, an unattended key; +inf (and any score with V apart) attends it
        seen = (c.Q[10:30, :, 3] > 0) if c.V is None else torch.ones(20, c.h_q, dtype=torch.bool)
        assert not bool(torch.isfinite(O[10:30, :, 3].cpu()[seen]).any())


def test_streams_and_no_lse(dev):
    c = Case(dev, RAGGED, 16, WIDE, out="bf16", seed=1)
    assert c.call(stream=torch.cuda.Stream(), lse=False) == 0
    c.check()


def test_nothing_to_do(dev):
    c = Case(dev, [(5, 0), (0, 0)], 16, WIDE, seed=1, spare_q=4)
    assert c.call() == 0
    assert bool((c.O == 7.0).all())


def test_agrees_with_the_dense_call(dev):
    """The same queries through sfa_dense_attend_paged (a position map instead of the table)."""
    for shape in (WIDE, W512, N128, N64):
        c = Case(dev, [(300, 20), (77, 5)], 16, shape, seed=8)
        assert c.call() == 0
        n_pos = max(c.total)
        cell_of = torch.tensor([[max(r[t // 16], 0) * 16 + t % 16 for t in range(n_pos)] for r in c.table],
                               dtype=torch.int32, device=dev)
        q_seq = torch.tensor([0] * 20 + [1] * 5, dtype=torch.int32, device=dev)
        q_pos = torch.tensor(list(range(300, 320)) + list(range(77, 82)), dtype=torch.int32, device=dev)
        O = torch.empty_like(c.O)
        if shape[3] // shape[4] > 16:
            continue
        sfa.sfa_dense_attend_paged(c.Q.to(dev), c.Kc, c.Vc, cell_of, q_seq, q_pos, n_pos, c.scale, O)
        ref, _, tol, _ = attend_reference(c.Q, c.K, c.V, c.table, 16, c.cu, c.total, c.scale, c.dv,
                                          p_round=UBF ** 2)
        check_close(c.O, O.double().cpu(), 2 * tol, "chunk against dense")


def dealt_out(need, part_rows, dv):
    """The workspace of work dealt out to s CTAs: two row tiles of partial results and notes each."""
    return any(need == 2 * s * part_rows * (dv + 2) * 4 + 32 * s for s in range(1, 161))


def many_lens(n, seed, longest=400):
    r = random.Random(seed)
    return [(r.choice([0, 1, 15, 16, 127, 128, r.randrange(longest)]), r.choice([0, 1, 1, 1, 2, 5])) for _ in range(n)]


@pytest.mark.parametrize("shape,dtype", [(WIDE, "bf16"), (W512, "bf16"), (N128, "bf16"), (N64, "bf16"), (N64K, "bf16"),
                                         (N128, "f32"), (WIDE, "q8")])
@pytest.mark.parametrize("n_seq", [32, 33, 100])
def test_many_sequences(dev, shape, dtype, n_seq):
    """More sequences than lanes, empty chunks and lists among them, the last ones too."""
    c = Case(dev, many_lens(n_seq - 2, n_seq) + [(40, 2), (3, 0)], 16, shape, dtype, "bf16", seed=n_seq)
    assert c.call() == 0
    c.check()


DEALT = [(3000, 3), (0, 0), (0, 90), (700, 1), (2300, 60), (5, 0), (1, 1), (1500, 2), (0, 3), (2900, 100)]


@pytest.mark.parametrize("shape", [N128, N64, N64K, N128K])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_dealt_out(dev, shape, out):
    """Narrow heads with ragged lists: slots that hold several lists, lists that take several
    slots, empty ones between; the same bits on every run, whatever the workspace held; bad pages."""
    c = Case(dev, DEALT, 32, shape, "bf16", out, seed=shape[0])
    need = sfa.sfa_chunk_attend_workspace_bytes(sfa.SFA_BF16, len(DEALT), c.cu[-1], shape[3], shape[4], shape[0], shape[1],
                                                shape[2], 100, 3003, sfa.SFA_BF16 if out == "bf16" else sfa.SFA_F32)
    assert dealt_out(need, min(100 * shape[3] // shape[4], 256), shape[1])
    ws = torch.full((need,), 255, dtype=torch.uint8, device=dev)
    assert c.call(workspace=ws) == 0
    c.check()
    O, lse = c.O, c.lse
    assert c.call(workspace=ws) == 0                    # what the first call left in it
    assert torch.equal(c.O, O) and torch.equal(c.lse, lse)
    t = [list(r) for r in c.table]
    t[0][40], t[4][0], t[9][70] = -1, len(c.K) // 32, 2 ** 31 - 1
    assert c.call(table=t, workspace=ws) == sfa.SFA_DEV_BAD_CELL
    c.check(table=t)


@pytest.mark.parametrize("shape,dtype", [(WIDE, "bf16"), (N128, "bf16"), (N64, "bf16"), (N128, "f32")])
def test_captured_and_replayed(dev, shape, dtype):
    """One captured call, replayed with other lengths (within the host bounds) and other queries."""
    c = Case(dev, [(900, 20), (300, 33), (64, 1), (0, 10)], 16, shape, dtype, seed=5)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
    Q, cu, total, table = c.Q.to(dev), i32(c.cu), i32(c.total), i32(c.table)
    c.O = torch.full((c.cu[-1], c.h_q, c.dv), 7.0, device=dev)
    c.lse = torch.full((c.cu[-1], c.h_q), 7.0, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    need = sfa.sfa_chunk_attend_workspace_bytes({"bf16": sfa.SFA_BF16, "f32": sfa.SFA_F32}[dtype], 4, c.cu[-1], c.h_q,
                                                c.h_kv, c.dkq, c.dv, c.sep, 40, 950)
    ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device=dev)
    run = lambda: sfa.sfa_chunk_attend_paged(Q, c.Kc, c.Vc, table, 16, cu, total, 40, 950, c.scale, c.O, lse=c.lse,
                                             workspace=ws, dev_status=status)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for new_cu, new_total in ((c.cu, c.total), ([0, 1, 41, 54, 64], [40, 333, 65, 10]), ([0, 20, 20, 60, 64], [920, 7, 65, 9])):
        cu.copy_(i32(new_cu))
        total.copy_(i32(new_total))
        c.Q = torch.randn(c.Q.shape, generator=torch.Generator().manual_seed(new_cu[1])).to(torch.bfloat16).to(c.Q.dtype)
        Q.copy_(c.Q)
        c.O.fill_(7.0)
        c.lse.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert sfa.sfa_read_device_status(status) == 0
        c.check(cu=new_cu, total=new_total)


def test_two_calls_at_once(dev):
    """Two streams, a workspace each: calls that overlap do not meet."""
    cases = [Case(dev, [(4000, 1), (2500, 1)], 32, s, seed=i) for i, s in enumerate((WIDE, N128, N64, W512))]
    alone = []
    for c in cases:
        assert c.call() == 0
        alone.append((c.O, c.lse))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
    streams = [torch.cuda.Stream() for _ in cases]
    runs = []
    for c in cases:
        runs.append((c.Q.to(dev), i32(c.table), i32(c.cu), i32(c.total), torch.empty_like(c.O), torch.empty_like(c.lse),
                     torch.zeros(1 << 24, dtype=torch.uint8, device=dev)))
    torch.cuda.synchronize()
    for _ in range(20):
        for c, st, (Q, table, cu, total, O, lse, ws) in zip(cases, streams, runs):
            sfa.sfa_chunk_attend_paged(Q, c.Kc, c.Vc, table, 32, cu, total, 1, 4001, c.scale, O, lse=lse,
                                       workspace=ws, stream=st)
    torch.cuda.synchronize()
    for (O, lse), run in zip(alone, runs):
        assert torch.equal(O, run[4]) and torch.equal(lse, run[5])


@pytest.mark.parametrize("shape,dtype", [(WIDE, "bf16"), (N128, "bf16"), (N64, "f32")])
def test_caches_past_32_bit_offsets(dev, shape, dtype):
    """Pages whose elements lie more than 2^32 into the cache."""
    c = Case(dev, [(300, 5), (0, 40)], 64, shape, dtype, seed=7)
    row = c.h_kv * min(c.dkq, c.dv)
    shift = (2 ** 32 // row) // 64 + 3                 # pages
    n = len(c.K)
    if torch.cuda.mem_get_info()[0] < 3 * (shift * 64 + n) * c.h_kv * c.dkq * c.Kc.element_size():
        pytest.skip("not enough device memory")

    def far(x):
        big = torch.empty((shift * 64 + n,) + x.shape[1:], dtype=x.dtype, device=dev)
        big[shift * 64:] = x
        return big

    c.Kc, c.Vc = far(c.Kc), None if c.Vc is None else far(c.Vc)
    assert c.call(table=[[e if e < 0 else e + shift for e in r] for r in c.table]) == 0
    c.check()


def test_infinite_keys(dev):
    """A key with an infinity scores +-inf: -inf is no weight at all, as the formula has it."""
    for shape, dtype in ((N128, "f32"), (N128, "bf16"), (W512, "bf16")):
        c = Case(dev, [(100, 30)], 16, shape, dtype, seed=11)
        c.Q[..., 3] = c.Q[..., 3].abs() + 0.5
        cell = c.table[0][50 // 16] * 16 + 50 % 16
        c.K[cell, :, 3] = -math.inf
        c.Kc = c.K.to(dev)
        assert c.call() == 0
        t = c.table
        c.K[cell, :, 3] = -1e4                         # a weight of zero in 64 bits too
        ref, _, _, _ = attend_reference(c.Q, c.K, c.V, t, 16, c.cu, c.total, c.scale, c.dv)
        c.K[cell, :, 3] = 0.0                          # the bound, without the far score
        _, _, tol, _ = attend_reference(c.Q, c.K, c.V, t, 16, c.cu, c.total, c.scale, c.dv, p_round=P_ROUND[dtype, "f32"])
        check_close(c.O, ref, tol, "O")


@pytest.mark.parametrize("shape,dtype,n_seq,length", [(N128, "bf16", 40, 30000), (N64, "bf16", 160, 30000),
                                                      (WIDE, "bf16", 80, 20000), (W512, "bf16", 40, 20000),
                                                      (W512K, "bf16", 80, 2100), (N128, "f32", 40, 20000)])
def test_long_sums_keep_fp32(dev, shape, dtype, n_seq, length):
    """fp32 results of long lists: hi + lo weights lose at most 2^-17, and a sum that is cut at each of
    its additions half a step a time on average, 2^-24 of a running sum that is two thirds of its end
    on average: 384 of them between sums that are rounded, so 256 2^-24.  (Sequences that share their pages, so that every list is long and whole.)"""
    dkq, dv, sep, h_q, h_kv = shape
    g = torch.Generator(device=dev).manual_seed(length)
    n_pages = -(-length // 64)
    randn = lambda *s: torch.randn(s, generator=g, device=dev).to(torch.bfloat16).to(TYPES[dtype])
    K, V, Q = randn(n_pages * 64, h_kv, dkq), randn(n_pages * 64, h_kv, dv) if sep else None, randn(n_seq + 1, h_q, dkq)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
    table = torch.arange(n_pages, dtype=torch.int32, device=dev).repeat(n_seq, 1)
    O = torch.empty((n_seq + 1, h_q, dv), device=dev)
    # the last sequence has two new tokens
    sfa.sfa_chunk_attend_paged(Q, K, V, table, 64, i32(list(range(n_seq)) + [n_seq + 1]), i32([length] * n_seq), 2, length,
                               1 / math.sqrt(dkq), O)
    G = h_q // h_kv
    for rows, keys in ((slice(0, n_seq - 1), length), (slice(n_seq - 1, n_seq), length - 1), (slice(n_seq, None), length)):
        k = K[:keys].double()
        v = k[..., :dv] if V is None else V[:keys].double()
        q = Q[rows].double().view(-1, h_kv, G, dkq)
        ref = torch.empty_like(O[rows], dtype=torch.float64)
        for i in range(h_kv):
            p = torch.softmax(q[:, i].reshape(-1, dkq) @ k[:, i].T / math.sqrt(dkq), -1)
            ref[:, i * G:(i + 1) * G] = (p @ v[:, i]).view(-1, G, dv)
        err = float((O[rows].double() - ref).norm() / ref.norm())
        assert err <= 256 * 2.0 ** -24 + 2.0 ** -17, f"{err:.3g}"


@pytest.mark.parametrize("shape,n_seq", [(N128, 40), (N64, 160), (WIDE, 80), (W512, 40)])
@pytest.mark.parametrize("bad_pages", [0, 56])
def test_long_sums_with_moving_maxima(dev, shape, n_seq, bad_pages):
    """Long whole lists whose scores rise and fall by tens, by other amounts in other heads, so that
    sums that were set aside are scaled again; and lists whose first 28 tiles hold no key at all.
    Bound: weights off by twice the scores' error (dkq / 16 additions cut by at most a step, 2^-23 of
    the score), and what test_long_sums_keep_fp32 allows."""
    dkq, dv, sep, h_q, h_kv = shape
    length, page = 9000, 64
    g = torch.Generator(device=dev).manual_seed(dkq + bad_pages)
    n_pages = -(-length // page)
    randn = lambda *s: torch.randn(s, generator=g, device=dev)
    # a walk of the scores, a step every 100 keys: about +-30 over the list
    steps = torch.randn(-(-n_pages * page // 100), generator=g, device=dev) * 4
    walk = steps.cumsum(0).repeat_interleave(100)[:n_pages * page]
    u = torch.sign(randn(h_kv, dkq))
    K = (randn(n_pages * page, h_kv, dkq) * 0.1 + walk.view(-1, 1, 1) * u / dkq ** 0.5).to(torch.bfloat16)
    V = randn(n_pages * page, h_kv, dv).to(torch.bfloat16) if sep else None
    G = h_q // h_kv
    gain = torch.linspace(-1, 1, G, device=dev).view(1, 1, G, 1)
    Q = (u.view(1, h_kv, 1, dkq) * gain + randn(n_seq, h_kv, G, dkq) * 0.05).reshape(n_seq, h_q, dkq).to(torch.bfloat16)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
    table = torch.arange(n_pages, dtype=torch.int32, device=dev).repeat(n_seq, 1)
    table[:, :bad_pages] = -1
    O = torch.empty((n_seq, h_q, dv), device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    sfa.sfa_chunk_attend_paged(Q, K, V, table, page, i32(list(range(n_seq + 1))), i32([length] * n_seq), 1, length,
                               1 / math.sqrt(dkq), O, dev_status=status)
    assert sfa.sfa_read_device_status(status) == (sfa.SFA_DEV_BAD_CELL if bad_pages else 0)
    k = K[bad_pages * page:length].double()
    v = k[..., :dv] if V is None else V[bad_pages * page:length].double()
    q = Q.double().view(n_seq, h_kv, G, dkq)
    ref = torch.empty_like(O, dtype=torch.float64)
    most = 0.0
    for i in range(h_kv):
        x = q[:, i].reshape(-1, dkq) @ k[:, i].T / math.sqrt(dkq)
        most = max(most, float(x.abs().max()))
        ref[:, i * G:(i + 1) * G] = (torch.softmax(x, -1) @ v[:, i]).view(n_seq, G, dv)
    assert most > 10
    err = float((O.double() - ref).norm() / ref.norm())
    assert err <= 2 * dkq / 16 * 2.0 ** -23 * most + 256 * 2.0 ** -24 + 2.0 ** -17, f"{err:.3g}"


@pytest.mark.parametrize("shape", [N128, N64, WIDE, W512, (128, 128, True, 12, 4), (576, 512, False, 12, 1)])
def test_long_chunks_keep_fp32(dev, shape):
    """The same with chunks: tiles full of rows and ones that are not (203 queries; 12 heads)."""
    dkq, dv, sep, h_q, h_kv = shape
    n_seq, new, length, page = 6, 203, 9000, 64
    g = torch.Generator(device=dev).manual_seed(h_q + dkq)
    n_pages = -(-length // page)
    randn = lambda *s: torch.randn(s, generator=g, device=dev).to(torch.bfloat16)
    K, V, Q = randn(n_pages * page, h_kv, dkq), randn(n_pages * page, h_kv, dv) if sep else None, randn(n_seq * new, h_q, dkq)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
    table = torch.arange(n_pages, dtype=torch.int32, device=dev).repeat(n_seq, 1)
    O = torch.empty((n_seq * new, h_q, dv), device=dev)
    sfa.sfa_chunk_attend_paged(Q, K, V, table, page, i32([s * new for s in range(n_seq + 1)]), i32([length] * n_seq), new,
                               length, 1 / math.sqrt(dkq), O)
    G = h_q // h_kv
    k = K[:length].double()
    v = k[..., :dv] if V is None else V[:length].double()
    hidden = torch.arange(length, device=dev)[None, :] > torch.arange(length - new, length, device=dev)[:, None]
    for s in range(n_seq):
        rows = slice(s * new, (s + 1) * new)
        ref = torch.empty_like(O[rows], dtype=torch.float64)
        for h in range(h_q):
            x = (Q[rows, h].double() @ k[:, h // G].T / math.sqrt(dkq)).masked_fill(hidden, -math.inf)
            ref[:, h] = torch.softmax(x, -1) @ v[:, h // G]
        err = float((O[rows].double() - ref).norm() / ref.norm())
        assert err <= 256 * 2.0 ** -24 + 2.0 ** -17, f"{err:.3g}"


@pytest.mark.parametrize("shape,dtype", [(N128, "bf16"), (N64, "bf16"), (WIDE, "bf16"), (N128, "f32")])
def test_lengths_at_the_ends_of_int32(dev, shape, dtype):
    """Device lengths that cannot be, the largest and smallest ones: flagged; the largest attends what
    its pages hold, the smallest and negative ones nothing, the others are right."""
    lens = [(3000, 3), (0, 90), (1566, 2), (2300, 60), (100, 7), (64, 1), (1500, 2), (0, 3)]   # the third: whole pages
    c = Case(dev, lens, 32, shape, dtype, seed=3)
    total = list(c.total)
    total[2], total[4], total[5] = 2 ** 31 - 1, -2 ** 31, -1
    assert c.call(total=total) == sfa.SFA_DEV_BAD_QUERY | sfa.SFA_DEV_BAD_CELL
    c.check(total=total, kv_max=max(c.total))
    for s in (4, 5):
        assert bool((c.O[c.cu[s]:c.cu[s + 1]] == 0).all())


def test_two_graphs_share_a_workspace(dev):
    """Captured calls of two shapes on one workspace, replayed in turn on one stream."""
    cases = [Case(dev, lens, 32, s, seed=i) for i, (s, lens) in enumerate(((WIDE, [(4000, 1), (2500, 1)]), (N128, DEALT)))]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
    ws = torch.full((1 << 26,), 255, dtype=torch.uint8, device=dev)
    graphs, kept = [], []
    for c in cases:
        assert c.call() == 0
        Q, table, cu, total = c.Q.to(dev), i32(c.table), i32(c.cu), i32(c.total)
        O, lse = torch.empty_like(c.O), torch.empty_like(c.lse)
        most = max(n for _, n in c.lens)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            sfa.sfa_chunk_attend_paged(Q, c.Kc, c.Vc, table, 32, cu, total, most, max(c.total), c.scale, O, lse=lse, workspace=ws)
        graphs.append(graph)
        kept.append((Q, table, cu, total, O, lse))
    for _ in range(3):
        for c, graph, (_, _, _, _, O, lse) in zip(cases, graphs, kept):
            O.fill_(5.0)
            graph.replay()
    torch.cuda.synchronize()
    for c, (_, _, _, _, O, lse) in zip(cases, kept):
        n = c.cu[-1]
        assert torch.equal(O[:n], c.O[:n]) and torch.equal(lse[:n], c.lse[:n])
