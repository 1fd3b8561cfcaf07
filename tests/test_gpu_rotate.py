"""sfa_rotate_rows against plain 64-bit rotation: layouts, parts of a head, types, strides, far positions,
rows into cells, in place, gradients, streams and graphs."""
import math

import pytest
import torch

from paged_util import check_close
from rotate_util import rotate_reference

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def sfa():
    import indexer_selected_sparse_block_gb300 as s
    return s


def _rows(n, h, d, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn((n, h, d), generator=g, device=DEV).to(dtype)


def _pos(n, far, seed):
    g = torch.Generator(device=DEV).manual_seed(seed + 77)
    return torch.randint(0, far, (n,), generator=g, device=DEV, dtype=torch.int64).to(torch.int32)


def _check(x, got, pos, rope, begin, what, inverse=False):
    ref, tol = rotate_reference(x, pos, rope.freqs, rope.magnitude, begin, rope.pairs, got.dtype, inverse)
    check_close(got, ref, tol, what)


TYPES = [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.bfloat16), (torch.float32, torch.float32)]


@pytest.mark.parametrize("src,dst", TYPES)
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("n,h,d,rot,begin", [
    (1, 16, 576, 64, 512), (33, 1, 576, 64, 512), (7, 3, 128, 128, 0), (5, 2, 64, 32, 16),
    (300, 16, 128, 64, 64), (9, 2, 512, 512, 0),
    (4, 3, 50, 6, 3), (3, 1, 2, 2, 0), (6, 5, 71, 70, 1),          # nothing aligned
    (5, 2, 64, 24, 8), (5, 2, 64, 40, 8),                          # adjacent pairs in 16 bytes, halves not
    (2500, 4, 64, 64, 0),                                          # several rows a block
])
def test_rotates(sfa, n, h, d, rot, begin, pairs, src, dst):
    x = _rows(n, h, d, src, n + d)
    pos = _pos(n, 131072, n)
    rope = sfa.SfaRope(rot, pairs=pairs)
    out = torch.full((n, h, d), 7.0, dtype=dst, device=DEV)
    sfa.sfa_rotate_rows([(x, out, begin)], pos, rope)
    _check(x, out, pos, rope, begin, "out")


@pytest.mark.parametrize("kw", [dict(factor=8.0), dict(factor=32.0, original_len=4096, magnitude=1.34657),
                                dict(base=5e6), dict(freqs=[(-1) ** j * 0.3 * j for j in range(32)])])
@pytest.mark.parametrize("pairs", [False, True])
def test_scaled_frequencies_at_far_positions(sfa, kw, pairs):
    x = _rows(64, 2, 64, torch.float32, 3)
    pos = torch.tensor([0, 1, 2, 4095, 4096, 1 << 20, (1 << 30) + 1, (1 << 31) - 1] * 8, dtype=torch.int32, device=DEV)
    rope = sfa.SfaRope(64, pairs=pairs, **kw)
    out = torch.empty_like(x)
    sfa.sfa_rotate_rows([(x, out, 0)], pos, rope)
    _check(x, out, pos, rope, 0, "out")


def test_quarter_turns(sfa):
    """Angles on and next to the quadrants' borders: frequencies of n / 8 turns a position."""
    freqs = [2 * math.pi * (k / 8 + e) for k in range(8) for e in (-1e-9, 0.0, 1e-9, 2.0 ** -40)]
    rope = sfa.SfaRope(64, freqs=freqs)
    x = _rows(40, 1, 64, torch.float32, 5)
    pos = torch.arange(40, dtype=torch.int32, device=DEV)
    out = torch.empty_like(x)
    sfa.sfa_rotate_rows([(x, out, 0)], pos, rope)
    _check(x, out, pos, rope, 0, "out")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,rot,begin", [(576, 64, 512), (96, 32, 32), (51, 10, 2)])
def test_in_place_leaves_the_other_dims(sfa, d, rot, begin, dtype):
    x = _rows(37, 3, d, dtype, 1)
    x[:, :, 0 if begin else -1] = float("nan")      # a dim that does not turn: its bits stay
    pos = _pos(37, 5000, 1)
    y = x.clone()
    rope = sfa.SfaRope(rot)
    sfa.sfa_rotate_rows([(y, y, begin)], pos, rope)
    keep = [k for k in range(d) if not begin <= k < begin + rot]
    bits = torch.int16 if dtype == torch.bfloat16 else torch.int32
    assert torch.equal(y[..., keep].view(bits), x[..., keep].view(bits))
    z = torch.nan_to_num(x)
    _check(z, torch.nan_to_num(y), pos, rope, begin, "in place")


def test_padding_rows_and_slots(sfa):
    n, n_cells = 40, 64
    x, q = _rows(n, 1, 576, torch.bfloat16, 2), _rows(n, 4, 64, torch.bfloat16, 3)
    pos, slot = _pos(n, 9000, 2), torch.randperm(n_cells, device=DEV)[:n].to(torch.int32)
    pos[5], pos[39], slot[7], slot[8], slot[9] = -1, -7, -1, n_cells, 2 ** 31 - 1
    cache = _rows(n_cells, 1, 576, torch.bfloat16, 4)
    Q = _rows(n, 4, 576, torch.bfloat16, 5)
    before, Qb = cache.clone(), Q.clone()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    rope = sfa.SfaRope(64, pairs=True)
    # the rotated part of the queries straight behind their other dims: a view
    sfa.sfa_rotate_rows([(q, Q[..., 512:], 0)], pos, rope, cells=[(x, cache, 512)], slot=slot, dev_status=status)
    assert sfa.sfa_read_device_status(status) == sfa.SFA_DEV_BAD_CELL
    live = [i for i in range(n) if i not in (5, 39, 7, 8, 9)]
    at = slot[live].long()
    _check(x[live], cache[at], pos[live], rope, 512, "cells")
    rest = torch.ones(n_cells, dtype=torch.bool, device=DEV)
    rest[at] = False
    assert torch.equal(cache[rest], before[rest])
    rows = [i for i in range(n) if i not in (5, 39)]
    _check(q[rows], Q[rows][..., 512:], pos[rows], rope, 0, "Q")
    assert torch.equal(Q[..., :512], Qb[..., :512]) and torch.equal(Q[[5, 39]], Qb[[5, 39]])


def test_strided_rows_and_heads(sfa):
    """Rows apart, heads outermost, a broadcast source and an odd offset."""
    n, h, d = 21, 4, 64
    pos, rope = _pos(n, 700, 8), sfa.SfaRope(32)
    x = _rows(h, n, 2 * d, torch.bfloat16, 6).transpose(0, 1)[..., :d]
    out = torch.zeros((h, n + 3, d + 8), dtype=torch.bfloat16, device=DEV).transpose(0, 1)[..., 8:]
    odd = torch.zeros(n * h * d + 1, dtype=torch.bfloat16, device=DEV)[1:].view(n, h, d)
    one = _rows(n, 1, d, torch.bfloat16, 7).expand(n, h, d)
    many = torch.empty((n, h, d), dtype=torch.bfloat16, device=DEV)
    flat = _rows(n, 1, d, torch.bfloat16, 9)[:, 0]
    flat_out = torch.empty_like(flat)
    sfa.sfa_rotate_rows([(x, out, 16), (x, odd, 16), (one, many, 0), (flat, flat_out, 32)], pos, rope)
    _check(x, out[:n], pos, rope, 16, "heads outermost")
    _check(x, odd, pos, rope, 16, "odd offset")
    _check(one, many, pos, rope, 0, "broadcast")
    _check(flat[:, None], flat_out[:, None], pos, rope, 32, "one head")
    assert not bool(out[n:].any())


def test_rows_of_one_stay_in_bounds(sfa):
    """A single row and head whose strides say nothing."""
    x = _rows(1, 1, 64, torch.bfloat16, 6)
    out = torch.empty((1, 1, 64), dtype=torch.bfloat16, device=DEV).as_strided((1, 1, 64), (3, 5, 1))
    pos, rope = _pos(1, 700, 8), sfa.SfaRope(32)
    sfa.sfa_rotate_rows([(x, out, 16)], pos, rope)
    _check(x, out, pos, rope, 16, "one")
    sfa.sfa_rotate_rows([(x[:0], out[:0], 16)], pos[:0], rope)
    sfa.sfa_rotate_rows([], pos, rope)


@pytest.mark.parametrize("pairs", [False, True])
def test_inverse_is_the_gradient_and_the_way_back(sfa, pairs):
    n, h, d = 19, 2, 96
    rope = sfa.SfaRope(64, pairs=pairs, magnitude=1.2)
    x, g = _rows(n, h, d, torch.float32, 1), _rows(n, h, d, torch.float32, 2)
    pos = _pos(n, 100000, 3)
    gx = torch.empty_like(g)
    sfa.sfa_rotate_rows([(g, gx, 32)], pos, rope, inverse=True)
    _check(g, gx, pos, rope, 32, "gradient", inverse=True)
    # the formula's gradient, by autograd in double
    xd = x.double().cpu().requires_grad_()
    ang = torch.outer(pos.double().cpu(), torch.tensor(rope.freqs, dtype=torch.float64))
    c, s = ang.cos()[:, None] * rope.magnitude, ang.sin()[:, None] * rope.magnitude
    z = xd[..., 32:]
    u, v = (z[..., 0::2], z[..., 1::2]) if pairs else (z[..., :32], z[..., 32:])
    a, b = u * c - v * s, u * s + v * c
    rot = torch.stack([a, b], -1).flatten(-2) if pairs else torch.cat([a, b], -1)
    torch.cat([xd[..., :32], rot], -1).backward(g.double().cpu())
    _, tol = rotate_reference(g, pos, rope.freqs, rope.magnitude, 32, pairs, torch.float32, True)
    check_close(gx, xd.grad, tol, "autograd")
    # and by differences of the call itself, which is linear
    y0, y1 = torch.empty_like(x), torch.empty_like(x)
    sfa.sfa_rotate_rows([(x, y0, 32)], pos, rope)
    step = _rows(n, h, d, torch.float32, 4)
    sfa.sfa_rotate_rows([(x + step, y1, 32)], pos, rope)
    lhs = ((y1.double() - y0.double()) * g.double()).sum()
    rhs = (step.double() * gx.double()).sum()
    size = ((y1.abs() + y0.abs()).double() * g.abs().double()).sum()
    assert abs(float(lhs - rhs)) <= 2.0 ** -18 * float(size)


def test_values_that_are_not_finite_stay_in_their_pair(sfa):
    x = _rows(4, 1, 64, torch.float32, 1)
    x[0, 0, 3], x[1, 0, 40], x[2, 0, 9] = math.inf, math.nan, -math.inf
    pos, rope = _pos(4, 999, 1), sfa.SfaRope(64)
    out = torch.empty_like(x)
    sfa.sfa_rotate_rows([(x, out, 0)], pos, rope)
    bad = ~torch.isfinite(out[:, 0])
    assert {tuple(t) for t in torch.nonzero(bad).tolist()} <= {(0, 3), (0, 35), (1, 8), (1, 40), (2, 9), (2, 41)}
    assert bad[0, 3] and bad[1, 8] and bad[1, 40] and bad[2, 41]


def test_stream_and_graph(sfa):
    n = 50
    x, pos, rope = _rows(n, 4, 128, torch.bfloat16, 1), _pos(n, 4000, 1), sfa.SfaRope(128)
    out, again = torch.empty_like(x), torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    sfa.sfa_rotate_rows([(x, out, 0)], pos, rope, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    _check(x, out, pos, rope, 0, "stream")
    g = sfa.SfaStep.graphed(lambda: sfa.sfa_rotate_rows([(x, again, 0)], pos, rope))
    del rope                                        # the call has read it
    x.copy_(_rows(n, 4, 128, torch.bfloat16, 2))
    pos.add_(1000)
    again.zero_()
    g.replay()
    torch.cuda.synchronize()
    _check(x, again, pos, sfa.SfaRope(128), 0, "replayed")


def test_offsets_past_32_bits(sfa):
    """The last rows of a cache of more than 2^31 elements."""
    n_cells, d = 2 ** 31 // 512 + 1000, 512
    cache = torch.empty((n_cells, 1, d), dtype=torch.bfloat16, device=DEV)
    x, pos, rope = _rows(5, 1, d, torch.bfloat16, 1), _pos(5, 4000, 1), sfa.SfaRope(64)
    slot = torch.tensor([n_cells - 1, 2 ** 31 // 512, 2 ** 31 // 512 - 1, n_cells - 17, 0], dtype=torch.int32, device=DEV)
    sfa.sfa_rotate_rows([], pos, rope, cells=[(x, cache, 448)], slot=slot)
    _check(x, cache[slot.long()], pos, rope, 448, "cells")
