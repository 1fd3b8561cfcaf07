"""Attention of drafted trees over a paged cache against the plain 64-bit form, within bounds that follow
from the arithmetic (tree_util.tree_attend_exact)."""
import math
import random

import pytest
import torch

from paged_util import UBF, check_close
from test_gpu_chunk import N64, N64K, N128, N128K, SHAPES, W512, W512K, WIDE
from tree_util import ancestors, pack, random_tree, tree_attend_exact

pytestmark = pytest.mark.gpu

sfa = pytest.importorskip("indexer_selected_sparse_block_gb300")
DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def q8_values(y, d):
    codes = y[..., :d].contiguous().view(torch.int8).float()
    return codes * y[..., d:d + d // 16].contiguous().view(torch.float16).float().repeat_interleave(32, -1)


class Trees:
    """lens: (cached, drafted) of each sequence on random pages; the cells that hold no token are NaN."""

    def __init__(self, lens, page, shape, dtype="bf16", out="f32", seed=0, spare_q=0, words=None, seen=None, odd=(),
                 scale=None, kscale=1.0, lost=()):
        self.dkq, self.dv, self.sep, self.h_q, self.h_kv = shape
        self.lens, self.page, self.dtype, self.out = lens, page, dtype, out
        self.halves = 0.0
        r, g = random.Random(seed), torch.Generator(device=DEV).manual_seed(seed)
        n_pg = [-(-(a + n) // page) for a, n in lens]
        order = torch.randperm(sum(n_pg) + 2, generator=g, device=DEV)
        self.table = torch.full((len(lens), max(n_pg + [1]) + 1), -1, dtype=torch.int32, device=DEV)
        self.cu, self.total, self.cells, at = [0], [a + n for a, n in lens], [], 0
        for s, k in enumerate(n_pg):
            self.table[s, :k] = order[at:at + k].to(torch.int32)
            t = torch.arange(self.total[s], device=DEV)
            self.cells.append(order[at:at + k][t // page] * page + t % page)
            at += k
            self.cu.append(self.cu[-1] + lens[s][1])
        for s, pg in lost:
            self.table[s, pg] = -1
            self.cells[s][pg * page:(pg + 1) * page] = -1
        n_cells = order.numel() * page
        live = torch.zeros(n_cells, dtype=torch.bool, device=DEV)
        for c in self.cells:
            live[c[c >= 0]] = True
        dt = torch.float32 if dtype == "f32" else torch.bfloat16
        n_q = self.cu[-1] + spare_q
        randn = lambda n, h, d: torch.randn((n, h, d), generator=g, device=DEV).to(dt)
        self.Q = randn(n_q, self.h_q, self.dkq)
        self.Q[self.cu[-1]:] = math.nan
        K, V = randn(n_cells, self.h_kv, self.dkq) * kscale, randn(n_cells, self.h_kv, self.dv) if self.sep else None
        if dtype == "q8":
            def quant(x):
                if x is None:
                    return None, None
                y = torch.zeros(x.shape[:-1] + (sfa.sfa_q8_0_row_bytes(x.shape[-1]),), dtype=torch.uint8, device=DEV)
                sfa.sfa_quantize_kv_q8_0(x, y)
                return y, q8_values(y, x.shape[-1])
            (self.K, self.Kv), (self.V, self.Vv) = quant(K), quant(V)
        else:
            self.Kv, self.Vv = K.clone(), None if V is None else V.clone()
            for x in (K, V):
                if x is not None:
                    x[~live] = math.nan
            for s, pos, i, d, x in odd:
                (K if V is None else V)[self.cells[s][pos], i, d] = x
            self.K, self.V = K, V
        if seen is None:
            seen = [ancestors(random_tree(n, r))[0] for _, n in lens]
        self.seen = seen
        self.words = words or max(1, -(-max([n for _, n in lens] + [1]) // 32))
        rows = [w for v in seen for w in pack(v, self.words)] + [[-1] * self.words] * spare_q
        self.mask = i32(rows).reshape(n_q, self.words)
        self.scale = 1 / math.sqrt(self.dkq) if scale is None else scale

    def call(self, part=None, n_new_max=None, n_kv_max=None, lse=True, stream=None):
        dt = torch.float32 if self.out == "f32" else torch.bfloat16
        n_q = self.Q.shape[0]
        self.part = sfa.SFA_PART_ALL if part is None else part
        self.O = torch.full((n_q, self.h_q, self.dv), 7.0, dtype=dt, device=DEV)
        self.lse = torch.full((n_q, self.h_q), 7.0, device=DEV) if lse else None
        status = i32([0])
        new_max = max([n for _, n in self.lens] + [1]) if n_new_max is None else n_new_max
        kv_max = max(self.total + [1]) if n_kv_max is None else n_kv_max
        code = {"bf16": sfa.SFA_BF16, "f32": sfa.SFA_F32, "q8": sfa.SFA_Q8_0}[self.dtype]
        need = sfa.sfa_tree_attend_workspace_bytes(code, len(self.lens), n_q, self.h_q, self.h_kv, self.dkq, self.dv, self.sep,
                                                   new_max, kv_max, sfa.SFA_F32 if self.out == "f32" else sfa.SFA_BF16,
                                                   part=self.part)
        ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device=DEV)     # NaN
        cu, total = i32(self.cu), i32(self.total)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        sfa.sfa_tree_attend_paged(self.Q, self.K, self.V, self.table, self.page, cu, total, self.mask, new_max, kv_max,
                                  self.scale, self.O, lse=self.lse, part=self.part, workspace=ws, dev_status=status,
                                  stream=stream)
        if stream is not None:
            torch.cuda.current_stream().wait_stream(stream)
        torch.cuda.synchronize()
        self.need = need
        return sfa.sfa_read_device_status(status)

    def exact(self, seen=None, twice=False):
        bf16 = self.dtype == "bf16"
        return tree_attend_exact(self.Q, self.Kv, self.Vv, self.cells, self.cu, self.total, seen or self.seen, self.scale,
                                 self.dv, drafted=self.part == sfa.SFA_PART_DRAFTED,
                                 # other caches: three tf32 products, 2^-19 of a product at most
                                 product=0.0 if bf16 else 2.0 ** -19,
                                 p_round=self.halves if not bf16 else UBF if self.out == "bf16" else UBF ** 2,
                                 o_round=(2 if twice else 1) * UBF if self.out == "bf16" else 0.0)

    def check(self, seen=None):
        ref, ref_l, tol, tol_l = self.exact(seen)
        n = self.cu[-1]
        check_close(self.O[:n], ref[:n], tol[:n], "O")
        if self.lse is not None:
            check_close(self.lse[:n], ref_l[:n], tol_l[:n], "lse")
            assert bool((self.lse[n:] == 7.0).all())
        assert bool((self.O[n:].float() == 7.0).all())

    def check_odd(self, odd):
        """Elements that no odd value reaches are those of a cache without any; what attends one has it."""
        ref, ref_l, tol, tol_l = self.exact(twice=True)
        hit = torch.zeros(ref.shape, dtype=torch.bool)
        any_hit = torch.zeros(ref_l.shape, dtype=torch.bool)
        G = self.h_q // self.h_kv
        for s, pos, i, d, _ in odd:
            a, n = self.lens[s]
            for j in range(n):
                if (pos < a and self.part == sfa.SFA_PART_ALL) or (pos >= a and self.seen[s][j][pos - a]):
                    if self.sep:
                        hit[self.cu[s] + j, i * G:(i + 1) * G, d] = True
                    else:
                        any_hit[self.cu[s] + j, i * G:(i + 1) * G] = True
        O, lse = self.O.double().cpu(), self.lse.double().cpu()
        assert not bool(torch.isfinite(O[hit]).any())
        keep = ~hit & ~any_hit[..., None]
        check_close(torch.where(keep, O, ref), ref, tol, "O")
        check_close(torch.where(any_hit, ref_l, lse), ref_l, tol_l, "lse")


DRAFTED = sfa.SFA_PART_DRAFTED
RAGGED = [(0, 1), (0, 17), (5, 3), (127, 1), (128, 40), (0, 0), (255, 2), (300, 0), (61, 70), (1, 33)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("dtype", ["bf16", "f32", "q8"])
@pytest.mark.parametrize("shape", SHAPES)
def test_ragged(shape, dtype, out):
    """Every shape and type: trees of one to many nodes, none, behind nothing or much, on and off the tiles'
    and pages' edges, unused rows of Q."""
    c = Trees(RAGGED, 16, shape, dtype, out, seed=shape[0], spare_q=5)
    assert c.call() == 0
    c.check()
    assert c.call(DRAFTED, lse=dtype != "f32") == 0
    c.check()


@pytest.mark.parametrize("shape", [WIDE, N128])
@pytest.mark.parametrize("page", [1, 3, 8, 24, 64, 100, 128, 256])
def test_page_sizes(shape, page):
    c = Trees([(190, 20), (0, 130), (64, 64), (127, 66)], page, shape, "bf16", "f32", seed=page)
    assert c.call() == 0
    c.check()
    assert c.call(DRAFTED) == 0
    c.check()


@pytest.mark.parametrize("shape,out", [(WIDE, "bf16"), (WIDE, "f32"), (W512, "f32"), (N128, "bf16"), (N64, "f32"), (N64K, "bf16")])
@pytest.mark.parametrize("lens", [[(9000, 16)], [(20000, 7), (17, 5), (4000, 63)], [(5000, 200), (1, 1)]])
def test_split_lists(shape, out, lens):
    """Long lists in pieces, their last one with the nodes or some of them."""
    c = Trees(lens, 64, shape, "bf16", out, seed=len(lens))
    assert c.call() == 0 and c.need > 0
    c.check()


@pytest.mark.parametrize("shape,out,n_seq,old,n", [
    (WIDE, "bf16", 7, 6000, 63),        # 56 lists on 76 pairs, whole
    (WIDE, "bf16", 7, 16000, 63),       # long first pieces, the ends on the other pairs
    (WIDE, "f32", 10, 3000, 63),        # 80 lists: a wave of whole ones, the last few cut
    (WIDE, "bf16", 20, 2000, 61),
    (W512, "bf16", 12, 2500, 63)])      # two KV heads: lists in the order of both
def test_last_waves(shape, out, n_seq, old, n):
    lens = [(old - 17 * s, n - (s % 3 == 2)) for s in range(n_seq)]
    odd = [(1, lens[1][0] + 5, 0, 3, math.nan), (n_seq - 1, old - 17 * (n_seq - 1), 0, 8, math.inf)]
    c = Trees(lens, 64, shape, "bf16", out, seed=n_seq)
    assert c.call() == 0 and (c.need > 0) == (old != 6000)
    c.check()
    if shape[2]:                         # V apart: an odd value is no odd score
        c = Trees(lens, 64, shape, "bf16", out, seed=n_seq, odd=odd)
        assert c.call() == 0
        c.check_odd(odd)


@pytest.mark.parametrize("shape", [WIDE, W512K, N128, N128K, N64])
@pytest.mark.parametrize("n", [129, 500, 1024])
def test_large_trees(shape, n):
    """Several row tiles and mask words; nodes in more than one key tile."""
    c = Trees([(70, n), (0, 31)], 32, shape, "bf16", "bf16", seed=n)
    assert c.call() == 0
    c.check()
    assert c.call(DRAFTED) == 0
    c.check()


@pytest.mark.parametrize("shape", [(576, 512, False, 48, 1), (576, 512, False, 12, 4), (512, 512, True, 40, 2),
                                   (512, 512, False, 64, 1), (128, 128, True, 64, 1), (128, 128, False, 15, 3),
                                   (64, 64, True, 21, 3), (64, 64, True, 16, 16)])
def test_groups_of_heads(shape):
    """Groups that leave tiles with rows to spare, and more heads than a node's tile has."""
    c = Trees([(300, 11), (0, 5), (77, 19)], 16, shape, "bf16", "f32", seed=shape[3])
    assert c.call() == 0
    c.check()
    assert c.call(DRAFTED) == 0
    c.check()


@pytest.mark.parametrize("shape", [WIDE, N128, N64])
@pytest.mark.parametrize("n_seq", [33, 300])
def test_many_sequences(shape, n_seq):
    """More sequences than a warp counts at a time, of a few nodes each, some without any."""
    r = random.Random(n_seq)
    lens = [(r.choice([0, 3, 130, r.randrange(300)]), r.choice([0, 1, 2, 5, 9])) for _ in range(n_seq)]
    c = Trees(lens, 8, shape, "bf16", "bf16", seed=n_seq, spare_q=3)
    assert c.call() == 0
    c.check()
    assert c.call(DRAFTED) == 0
    c.check()


def test_two_calls_at_once():
    """On two streams, each with a workspace from its stream's pool."""
    a, b = Trees([(30000, 20)], 64, WIDE, seed=3), Trees([(20000, 31), (9000, 4)], 64, N128, seed=4)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    args = [(c.Q, c.K, c.V, c.table, c.page, i32(c.cu), i32(c.total), c.mask, 31, 30031, c.scale) for c in (a, b)]
    for c in (a, b):
        c.part = sfa.SFA_PART_ALL
        c.O = torch.full((c.Q.shape[0], c.h_q, c.dv), 7.0, device=DEV)
        c.lse = torch.full((c.Q.shape[0], c.h_q), 7.0, device=DEV)
    torch.cuda.synchronize()
    for _ in range(5):
        for c, x, s in zip((a, b), args, streams):
            sfa.sfa_tree_attend_paged(*x, c.O, lse=c.lse, stream=s)
    torch.cuda.synchronize()
    a.check()
    b.check()


@pytest.mark.parametrize("shape,dtype", [(WIDE, "bf16"), (N128, "bf16"), (N64, "bf16"), (WIDE, "f32"), (N64, "q8")])
def test_any_mask(shape, dtype):
    """Masks that are no tree's: rows that attend nothing, later nodes, not themselves; bits behind the last
    node."""
    r = random.Random(3)
    lens = [(0, 40), (130, 35), (0, 3)]
    seen = [[[r.random() < 0.4 for _ in range(n)] for _ in range(n)] for _, n in lens]
    seen[0][5] = seen[0][39] = seen[1][0] = [False] * 40
    seen[2] = [[False] * 3] * 3
    c = Trees(lens, 16, shape, dtype, "f32", seen=seen, words=3)
    full = c.mask.clone()
    for s, (_, n) in enumerate(lens):                      # bits that no node has
        for w in range(3):
            junk = sum(1 << b for b in range(32) if 32 * w + b >= n)
            full[c.cu[s]:c.cu[s + 1], w] |= junk - (1 << 32) if junk >> 31 else junk
    c.mask = full
    for part in (sfa.SFA_PART_ALL, DRAFTED):
        assert c.call(part) == 0
        c.check(seen=[[v[:n] for v in x[:n]] for x, (_, n) in zip(seen, lens)])
    empty = c.lse[5].cpu()
    assert bool((empty == -math.inf).all()) and not bool(c.O[5].any())


def test_a_chain_is_the_causal_chunk():
    """A tree that is one path: the chunk attention's results, within both bounds."""
    for shape in (WIDE, N128):
        lens = [(300, 50), (0, 20)]
        c = Trees(lens, 16, shape, seen=[ancestors([j - 1 for j in range(n)])[0] for _, n in lens])
        assert c.call() == 0
        O, lse = torch.empty_like(c.O), torch.empty_like(c.lse)
        sfa.sfa_chunk_attend_paged(c.Q, c.K, c.V, c.table, c.page, i32(c.cu), i32(c.total), 50, 350, c.scale, O, lse=lse)
        _, _, tol, tol_l = c.exact()
        check_close(O, c.O.double().cpu(), 2 * tol, "O")
        check_close(lse, c.lse.double().cpu(), 2 * tol_l, "lse")


@pytest.mark.parametrize("shape", [WIDE, N128, N64])
@pytest.mark.parametrize("scale,kscale", [(-0.2, 1.0), (0.0, 1.0), (1.0, 4.0)])
def test_scales(shape, scale, kscale):
    c = Trees([(200, 30), (0, 9)], 16, shape, scale=scale, kscale=kscale)
    assert c.call() == 0
    c.check()


ODD = [math.nan, math.inf, -math.inf]


@pytest.mark.parametrize("dtype", ["f32", "q8"])
@pytest.mark.parametrize("shape", [WIDE, W512, N128, N64])
@pytest.mark.parametrize("scale,kscale", [(-0.2, 1.0), (0.0, 1.0), (1.0, 4.0), (0.05, 2.0 ** -40)])
def test_scales_of_other_caches(shape, dtype, scale, kscale):
    if dtype == "q8" and kscale < 1:
        kscale = 2.0 ** -10      # scales of blocks are binary16
    c = Trees([(300, 20), (1000, 40), (0, 9)], 16, shape, dtype, "f32", scale=scale, kscale=kscale)
    if dtype == "q8":
        # p v with both in two bf16 halves, x = hi + lo + r: of x in [1, 2) lo is 2^-8 at most, r half a step of that,
        # 2^-17; what is left out, r_p v, p r_v and lo_p lo_v, is 2^-17 + 2^-17 + 2^-16 of |p v| at most, 2 UBF^2; the
        # bound takes a weight's rounding twice.  (Of scores near zero; elsewhere the scores' own bound is above it.)
        c.halves = UBF ** 2
    assert c.call() == 0
    c.check()


@pytest.mark.parametrize("dtype,out", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("shape", [WIDE, W512, W512K, N128, N128K, N64])
def test_odd_values_stay_in_their_branch(shape, dtype, out):
    """NaN and infinities in nodes' values: in whole lists, in pieces, first and last nodes, two of them in
    rows that attend one, both or neither; and none where only a cached token has them."""
    lens = [(150, 40), (0, 33), (7000, 20), (64, 64), (300, 12)]
    dv, h_kv = shape[1], shape[4]
    odd = [(0, 155, 0, 3, ODD[0]), (0, 189, h_kv - 1, dv - 1, ODD[1]), (1, 7, 0, 0, ODD[2]), (1, 32, 0, 5, ODD[0]),
           (2, 7003, 0, 9, ODD[1]), (3, 64 + 63, h_kv - 1, 40, ODD[0]), (4, 17, 0, 7, ODD[0])]
    c = Trees(lens, 16, shape, dtype, out, seed=5, odd=odd)
    assert c.call() == 0
    c.check_odd(odd)
    assert c.call(DRAFTED) == 0
    c.check_odd(odd)


@pytest.mark.parametrize("gap", [50.0, 200.0])
@pytest.mark.parametrize("dtype,out", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("shape", [W512, N128, N64])
def test_odd_values_of_small_weights(shape, dtype, out, gap):
    """A value that is not finite shows in what attends it by however small a weight (scores `gap` below others)."""
    lens = [(150, 40), (0, 33), (64, 64)]
    odd = [(0, 155, 0, 3, math.nan), (1, 7, 0, 0, math.inf), (2, 64, 0, 40, -math.inf)]
    c = Trees(lens, 16, shape, dtype, out, seed=6, odd=odd)
    c.Q[..., 0] = 16.0
    for s, pos, i, _, _ in odd:
        for x in (c.K, c.Kv):
            x[c.cells[s][pos], i, 0] = -gap / (16.0 * c.scale)
    assert c.call() == 0
    c.check_odd(odd)
    assert c.call(DRAFTED) == 0
    c.check_odd(odd)


@pytest.mark.parametrize("scale", [b"\x00\x7c", b"\x01\x7e"])     # an infinity, a NaN
@pytest.mark.parametrize("shape", [WIDE, W512, N128, N64])
def test_odd_scales_of_q8_rows_stay_in_their_branch(shape, scale):
    """A block's scale that is not finite: of the values (apart, its 32 dims; where V is K, whatever attends it, but
    by a score of minus infinity, whose weight is zero)."""
    a, n, node, blk = 70, 30, 4, 1
    c = Trees([(a, n), (5, 9)], 16, shape, "q8", "f32", seed=9)
    rows, d = (c.V, c.dv) if c.sep else (c.K, c.dkq)
    rows[c.cells[0][a + node], 0, d + 2 * blk:d + 2 * blk + 2] = torch.tensor(list(scale), dtype=torch.uint8, device=DEV)
    assert c.call() == 0
    ref, ref_l, tol, tol_l = c.exact()
    hit = torch.tensor([v[node] for v in c.seen[0]] + [False] * 9)
    heads = torch.arange(c.h_q) < c.h_q // c.h_kv           # of KV head 0
    odd = hit[:, None] & heads[None]
    O, lse = c.O.double().cpu(), c.lse.double().cpu()
    dims = torch.zeros(c.dv, dtype=torch.bool)
    dims[32 * blk:32 * blk + 32] = True
    if not c.sep:
        dims[:] = True
    bad = odd[..., None] & dims
    assert bool(hit.any())
    if c.sep or scale == b"\x01\x7e":
        assert not bool(torch.isfinite(O[bad]).any())
    check_close(torch.where(bad, ref, O), ref, tol, "O")
    check_close(lse if c.sep else torch.where(odd, ref_l, lse), ref_l, tol_l, "lse")


@pytest.mark.parametrize("gap", [50.0, 200.0])
@pytest.mark.parametrize("shape", [W512, N128, N64])
def test_odd_scales_of_small_weights(shape, gap):
    """An infinite scale of values shows in what attends it by however small a weight."""
    a, n, node, blk = 70, 30, 4, 1
    c = Trees([(a, n), (5, 9)], 16, shape, "q8", "f32", seed=9)
    d = c.dkq
    c.Q[..., 0] = 16.0
    cell = c.cells[0][a + node]
    # the key's first block: its first code -127 by the scale that gives the score, zeros otherwise
    row = c.K[cell, 0]
    row[:32] = 0
    row[0] = 129                                                        # -127
    row[d:d + 2] = torch.tensor([gap / (16.0 * c.scale * 127)], dtype=torch.float16, device=DEV).view(torch.uint8)
    c.V[cell, 0, c.dv + 2 * blk:c.dv + 2 * blk + 2] = torch.tensor(list(b"\x00\x7c"), dtype=torch.uint8, device=DEV)
    assert c.call() == 0
    hit = torch.tensor([v[node] for v in c.seen[0]] + [False] * 9)
    odd = hit[:, None] & (torch.arange(c.h_q) < c.h_q // c.h_kv)[None]
    O = c.O.double().cpu()
    dims = torch.zeros(c.dv, dtype=torch.bool)
    dims[32 * blk:32 * blk + 32] = True
    bad = odd[..., None] & dims
    assert bool(hit.any()) and not bool(torch.isfinite(O[bad]).any())
    assert bool(torch.isfinite(O[~bad]).all())


@pytest.mark.parametrize("shape", [WIDE, N128])
def test_odd_values_of_the_cached_tokens_stay_out_of_the_drafted_part(shape):
    c = Trees([(130, 10)], 16, shape, "bf16", "f32", odd=[(0, 129, 0, 1, math.nan), (0, 128, 0, 2, math.inf)])
    assert c.call(DRAFTED) == 0
    c.check()


def test_missing_pages():
    """Pages that are none are left out and flagged, of the cached tokens and of the nodes."""
    for shape, dtype in ((WIDE, "bf16"), (N128, "bf16"), (WIDE, "f32")):
        c = Trees([(100, 30), (16, 5), (3, 20)], 8, shape, dtype, lost=[(0, 2), (0, 14), (1, 0), (1, 1), (1, 2), (2, 0)])
        assert c.call() == sfa.SFA_DEV_BAD_CELL
        c.check()


def test_bounds_cut_trees_and_lists():
    c = Trees([(100, 30), (50, 9)], 16, N128)
    assert c.call(n_new_max=12) == sfa.SFA_DEV_BAD_QUERY
    ref, ref_l, tol, tol_l = c.exact(seen=[[[on and x < 12 for x, on in enumerate(v)] for v in c.seen[0]], c.seen[1]])
    rows = list(range(12)) + list(range(30, 39))
    check_close(c.O[rows], ref[rows], tol[rows], "O")
    check_close(c.lse[rows], ref_l[rows], tol_l[rows], "lse")
    assert bool((c.O[12:30] == 7.0).all())
    assert c.call(n_kv_max=110) == sfa.SFA_DEV_BAD_QUERY
    ref, _, tol, _ = c.exact(seen=[[[on and x < 10 for x, on in enumerate(v)] for v in c.seen[0]], c.seen[1]])
    check_close(c.O[:39], ref[:39], tol[:39], "O")


def test_bad_lengths():
    """Offsets that do not ascend: no tree; fewer positions than nodes: the nodes that have one."""
    c = Trees([(40, 10), (30, 8)], 16, WIDE)
    cu = list(c.cu)
    c.cu = [0, 10, 5]
    assert c.call() == sfa.SFA_DEV_BAD_QUERY
    c.cu = [0, 10, 10]
    ref, _, tol, _ = c.exact()
    check_close(c.O[:10], ref[:10], tol[:10], "O")
    assert bool((c.O[10:] == 7.0).all())
    c.cu, c.total = cu, [6, 38]
    assert c.call() == sfa.SFA_DEV_BAD_QUERY
    c2 = Trees([(40, 10), (30, 8)], 16, WIDE)
    assert c2.call() == 0
    assert torch.equal(c.O[10:], c2.O[10:])


def test_no_cells_and_no_rows():
    c = Trees([(0, 4)], 16, N64)
    c.table.fill_(-1)
    c.cells = [torch.full((4,), -1, device=DEV)]
    assert c.call() == sfa.SFA_DEV_BAD_CELL
    assert not bool(c.O.any()) and bool((c.lse == -math.inf).all())
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=DEV)
    sfa.sfa_tree_attend_paged(e(0, 8, 64), c.K, c.V, c.table, 16, i32([0, 0]), i32([0]), i32([]).reshape(0, 1), 4, 9, 1.0,
                              e(0, 8, 64))


def test_another_stream_and_host_results():
    c = Trees([(500, 20), (31, 9)], 16, W512)
    side = torch.cuda.Stream()
    assert c.call(stream=side) == 0
    c.check()
    O = torch.zeros(c.O.shape, dtype=torch.float32).pin_memory()
    sfa.sfa_tree_attend_paged(c.Q, c.K, c.V, c.table, c.page, i32(c.cu), i32(c.total), c.mask, 20, 520, c.scale, O)
    torch.cuda.synchronize()
    assert torch.equal(O, c.O.cpu())


@pytest.mark.parametrize("power", [20, 60, 100])
@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("shape", [W512, N128, N64])
def test_large_values_where_they_weigh_little(shape, dtype, out, power):
    """Values 2^power times the others': of a node that few attend, of a node and a cached token whose scores are as
    much lower, and of a node that its descendants attend as any other."""
    lens = [(150, 40), (20, 33), (5000, 20), (64, 64)]
    c = Trees(lens, 16, shape, dtype, out, seed=8)
    c.Q[..., 0] = 16.0
    large = [(0, 155, False), (1, 20 + 7, True), (1, 3, True), (2, 4000, True), (3, 64 + 40, False)]
    for s, pos, low in large:
        cell = c.cells[s][pos]
        for x in (c.V, c.Vv):
            x[cell] = x[cell] * 2.0 ** power
        if low:
            for x in (c.K, c.Kv):
                x[cell, :, 0] = -math.log(2.0) * power / (16.0 * c.scale)
    assert c.call() == 0
    c.check()


@pytest.mark.parametrize("shape", [WIDE, W512, N128, N64])
@pytest.mark.parametrize("dtype", ["q8", "f32", "bf16"])
def test_long_sums_are_rounded_not_cut(shape, dtype):
    """Queries of zero: every weight is one, and the results are means of many positive values, to which a sum
    cut towards zero at every step would be short by its steps.  Off by: the values' two parts, 2^-17 at most
    each way (q8_0 ones; bf16 and fp32 ones less); sums of what tiles of at least 16 keys give, rounded or,
    of bf16 caches, cut for 24 tiles of 128 keys at a time: 2.2e-7 a tile; the result's rounding."""
    n_keys = 30000
    c = Trees([(n_keys, 4)], 64, shape, dtype, "f32", seed=2)
    c.Q.zero_()
    for x, v in ((c.K, c.Kv), (c.V, c.Vv)):
        if x is None:
            continue
        if dtype == "q8":                       # the codes' signs
            d = v.shape[-1]
            codes = x[..., :d].contiguous().view(torch.int8)
            x[..., :d] = codes.abs().view(torch.uint8)
            v.copy_(q8_values(x, d))
        else:
            x.abs_()
            v.abs_()
    assert c.call() == 0
    ref, ref_l, _, _ = c.exact()
    steps = n_keys / 16
    off = 2.0 ** -16 + 6 * math.sqrt(steps) * 2.0 ** -24 + 24 * 2.2e-7 + 2.0 ** -22
    err = (c.O.double().cpu() - ref).abs() / ref
    assert float(err.max()) <= off, (float(err.max()), off)
    assert float((c.lse.double().cpu() - ref_l).abs().max()) <= 6 * math.sqrt(n_keys) * 2.0 ** -24


def test_results_do_not_change_from_run_to_run():
    for shape, lens in ((WIDE, [(9000, 16), (100, 30)]), (N128, [(9000, 16), (100, 61), (3000, 2)])):
        c = Trees(lens, 16, shape, "bf16", "f32")
        assert c.call() == 0
        O, lse = c.O.clone(), c.lse.clone()
        for _ in range(3):
            assert c.call() == 0
            assert torch.equal(O, c.O) and torch.equal(lse, c.lse)


def test_two_captured_calls_with_a_workspace_each():
    """Replayed in turn, with lengths and masks changed between."""
    a, b = Trees([(4000, 20)], 16, WIDE), Trees([(3000, 31)], 16, WIDE, seed=1)
    graphs = []
    for c in (a, b):
        c.call()
        ws = torch.empty(max(c.need, 16), dtype=torch.uint8, device=DEV)
        c.d = (i32(c.cu), i32(c.total), ws)
        graphs.append(sfa.SfaStep.graphed(lambda c=c: sfa.sfa_tree_attend_paged(
            c.Q, c.K, c.V, c.table, c.page, c.d[0], c.d[1], c.mask, c.lens[0][1], c.total[0], c.scale, c.O, lse=c.lse,
            workspace=c.d[2])))
    for c, cut in ((a, 5), (b, 9)):
        n = c.lens[0][1]
        c.seen = [[[x == j for x in range(n)] for j in range(n)]]
        c.mask.copy_(i32(pack(c.seen[0], c.words)))
        c.d[1].sub_(cut)                                  # fewer cached tokens: other keys for every node
        c.total[0] -= cut
        c.lens[0] = (c.lens[0][0] - cut, n)
        c.O.zero_()
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    a.check()
    b.check()
