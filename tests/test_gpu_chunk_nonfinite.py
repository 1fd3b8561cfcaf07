"""Values that are not finite in new tokens: they reach the queries that attend them, and no
earlier query of their chunk."""
import math

import pytest
import torch

from paged_util import UBF, attend_exact, check_close
from test_gpu_chunk import N64, N128, W512, W512K, WIDE

pytestmark = pytest.mark.gpu

sfa = pytest.importorskip("indexer_selected_sparse_block_gb300")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    return torch.device("cuda:0")


class Chunks:
    """lens: (cached before, new) of each sequence, on random pages; `odd` of them, (sequence,
    position, KV head, value dim, value), are set in V (or K, where it is V)."""

    def __init__(self, dev, shape, lens, odd, out="f32", dtype="bf16", page=16, seed=0, full=False):
        self.dkq, self.dv, self.sep, self.h_q, self.h_kv = shape
        self.lens, self.page, self.out, self.odd = lens, page, out, odd
        g = torch.Generator(device=dev).manual_seed(seed)
        n_pg = [-(-(a + n) // page) for a, n in lens]
        order = torch.randperm(sum(n_pg) + 2, generator=g, device=dev)
        self.table = torch.full((len(lens), max(n_pg)), -1, dtype=torch.int32, device=dev)
        self.cu, self.total, at = [0], [a + n for a, n in lens], 0
        self.cells = []
        for s, k in enumerate(n_pg):
            self.table[s, :k] = order[at:at + k].to(torch.int32)
            t = torch.arange(self.total[s], device=dev)
            self.cells.append(order[at:at + k][t // page] * page + t % page)
            at += k
            self.cu.append(self.cu[-1] + lens[s][1])
        self.dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
        held = torch.float32 if full else torch.bfloat16      # full: fp32 values with all their bits
        randn = lambda n, h, d: torch.randn((n, h, d), generator=g, device=dev).to(held).to(self.dt)
        n_cells = order.numel() * page
        self.Q = randn(self.cu[-1], self.h_q, self.dkq)
        self.K, self.V = randn(n_cells, self.h_kv, self.dkq), randn(n_cells, self.h_kv, self.dv) if self.sep else None
        self.clean = (self.K.clone(), None if self.V is None else self.V.clone())
        for s, pos, i, d, x in odd:
            (self.K if self.V is None else self.V)[self.cells[s][pos], i, d] = x
        self.scale, self.dev = 1 / math.sqrt(self.dkq), dev

    def call(self):
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=self.dev)
        self.O = torch.full((self.cu[-1], self.h_q, self.dv), 7.0, device=self.dev,
                            dtype=torch.float32 if self.out == "f32" else torch.bfloat16)
        self.lse = torch.full((self.cu[-1], self.h_q), 7.0, device=self.dev)
        status = torch.zeros(1, dtype=torch.int32, device=self.dev)
        most = max(n for _, n in self.lens)
        need = sfa.sfa_chunk_attend_workspace_bytes(
            sfa.SFA_BF16 if self.dt is torch.bfloat16 else sfa.SFA_F32, len(self.lens), self.cu[-1], self.h_q, self.h_kv,
            self.dkq, self.dv, self.sep, most, max(self.total), sfa.SFA_F32 if self.out == "f32" else sfa.SFA_BF16)
        ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device=self.dev)
        sfa.sfa_chunk_attend_paged(self.Q, self.K, self.V, self.table, self.page, i32(self.cu), i32(self.total), most,
                                   max(self.total), self.scale, self.O, lse=self.lse, workspace=ws, dev_status=status)
        assert sfa.sfa_read_device_status(status) == 0
        return need

    def check(self):
        """Elements that no odd value reaches are those of a cache without any; the others are not
        finite.  (With V apart: an odd value has no part in the scores.  Where V is K, what attends an
        odd key is not looked at: its score is odd too.)"""
        K, V = self.clean
        p_round = UBF ** 2 if self.out == "f32" else UBF
        if self.dt is torch.float32:
            p_round = 0.0
        ref, ref_l, tol, tol_l = attend_exact(self.Q, K, V, self.cells, self.cu, self.total, self.scale, self.dv,
                                              p_round=p_round, o_round=UBF if self.out == "bf16" else 0.0)
        G = self.h_q // self.h_kv
        row, reached = torch.zeros(ref.shape[:2], dtype=torch.bool), torch.zeros(ref.shape, dtype=torch.bool)
        for s, pos, i, d, _ in self.odd:
            first = self.cu[s] + max(pos - self.lens[s][0], 0)
            row[first:self.cu[s + 1], i * G:(i + 1) * G] = True
            reached[first:self.cu[s + 1], i * G:(i + 1) * G, d] = True
        O, lse = self.O.double().cpu(), self.lse.cpu()
        if self.sep:
            assert not bool(torch.isfinite(O[reached]).any())
            row[:] = False
        skip = reached if self.sep else row[..., None].expand_as(reached)
        check_close(torch.where(skip, ref, O), ref, tol, "O")
        check_close(torch.where(row, ref_l.float(), lse), torch.where(row, ref_l.float().double(), ref_l), tol_l, "lse")


@pytest.mark.parametrize("shape", [WIDE, W512, N128, N64])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("many", [False, True])
def test_pieces_that_a_row_does_not_attend(dev, shape, out, many):
    """A list is cut so that its last piece holds the last token alone, whose values are not finite:
    the other queries of its chunk have no key there.  Few pieces, and many (another merge)."""
    dkq, dv, sep, h_q, h_kv = shape
    for tiles in range(3, 60):
        total = 128 * tiles + 1
        need = sfa.sfa_chunk_attend_workspace_bytes(sfa.SFA_BF16, 1, 3, h_q, h_kv, dkq, dv, sep, 3, total,
                                                    sfa.SFA_F32 if out == "f32" else sfa.SFA_BF16)
        rows = 3 * (h_q // h_kv)
        split, rest = divmod(need, h_kv * rows * (dv + 2) * 4)
        if rest == 0 and split > 1 and (split >= 8) == many and tiles % -(-(tiles + 1) // split) == 0:
            break
    else:
        pytest.skip("no such length found for this device")
    odd = [(0, total - 1, i, 5 + i, x) for i in range(h_kv) for x in [math.nan]]
    c = Chunks(dev, shape, [(total - 3, 3)], odd, out=out, seed=dkq)
    assert c.call() == need
    c.check()


N128K, N64K, G1 = (128, 128, False, 4, 4), (64, 64, False, 8, 2), (512, 512, True, 2, 2)
SHAPES = [WIDE, W512, W512K, G1, N128, N128K, N64, N64K]
NAN, INF = math.nan, math.inf


def odd_tokens(shape, lens):
    """In every sequence's chunk: its second token, one in the middle and the last, other values and KV
    heads each; in the first sequence every token from the sixth on."""
    odd = []
    for s, (a, n) in enumerate(lens):
        for k, pos in enumerate(sorted({a + min(1, n - 1), a + n // 2, a + n - 1})):
            odd.append((s, pos, (s + k) % shape[4], (7 * k + s) % shape[1], (NAN, INF, -INF)[k % 3]))
    odd += [(0, lens[0][0] + j, 0, j % shape[1], NAN) for j in range(5, lens[0][1])]
    return odd


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype,out", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
def test_later_tokens(dev, shape, dtype, out):
    """Chunks of one to 150 tokens behind none to 700, odd tokens all over them."""
    lens = [(100, 30), (5, 3), (0, 40), (127, 2), (700, 150), (64, 1), (0, 1), (300, 129)]
    c = Chunks(dev, shape, lens, odd_tokens(shape, lens), out=out, dtype=dtype, seed=shape[0])
    c.call()
    c.check()


@pytest.mark.parametrize("shape", [WIDE, W512, N128, N64])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_later_tokens_of_cut_lists(dev, shape, out):
    """Long lists in pieces, each looked at for itself; a chunk that lies across two of them."""
    lens = [(6000, 5), (4090, 12), (37, 8)]
    c = Chunks(dev, shape, lens, odd_tokens(shape, lens), out=out, page=32, seed=shape[0] + 1)
    assert c.call() > 0
    c.check()


@pytest.mark.parametrize("shape,n_seq", [(WIDE, 80), (W512, 40), (N128, 40), (N64, 160)])
def test_later_tokens_behind_moved_sums(dev, shape, n_seq):
    """Whole lists of more than 24 tiles with fp32 results, whose sums were set aside on the way."""
    lens = [(4000, 4)] * n_seq
    odd = [(s, 4000 + s % 4, s % shape[4], s % shape[1], NAN) for s in range(0, n_seq, 3)]
    c = Chunks(dev, shape, lens, odd, page=64, seed=shape[0] + 2)
    c.call()
    c.check()


@pytest.mark.parametrize("shape", [WIDE, W512, N128, N64, N64K])
def test_positions_below_zero(dev, shape):
    """More new tokens than cached ones: queries below position 0 attend nothing, whatever the tokens
    from 0 on hold."""
    c = Chunks(dev, shape, [(0, 12)], [(0, 0, 0, 3, NAN), (0, 5, 0, 4, NAN)], seed=3)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
    O = torch.full((12, c.h_q, c.dv), 7.0, device=dev)
    lse = torch.full((12, c.h_q), 7.0, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    sfa.sfa_chunk_attend_paged(c.Q, c.K, c.V, c.table, 16, i32([0, 12]), i32([8]), 12, 12, c.scale, O, lse=lse,
                               dev_status=status)
    assert sfa.sfa_read_device_status(status) == sfa.SFA_DEV_BAD_QUERY
    G = c.h_q // c.h_kv
    assert bool((O[:4] == 0).all()) and bool(torch.isneginf(lse[:4]).all())
    # queries 4 to 8 are at positions 0 to 4: the odd token at 5 is not theirs
    if c.sep:
        assert bool(torch.isfinite(O[4:9, :G, 4]).all()) and not bool(torch.isfinite(O[9:, :G, 4]).any())
        assert not bool(torch.isfinite(O[4:, :G, 3]).any())
    assert bool(torch.isfinite(O[:, G:]).all())


@pytest.mark.parametrize("shape", [WIDE, W512, N128, N64])
def test_old_odd_values(dev, shape):
    """Odd values in cached tokens, which every query attends: nothing is done again, all are odd."""
    lens = [(300, 20), (50, 9)]
    c = Chunks(dev, shape, lens, [(0, 250, 0, 3, NAN), (1, 3, 0, 5, NAN)], seed=5)
    c.call()
    c.check()
