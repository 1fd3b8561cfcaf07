"""Rotary positions on the host: frequencies and their scaling, the phase table, refusals before anything
is enqueued, and the binding's checks."""
import ctypes
import math

import pytest
import torch

FAKE = ctypes.c_void_p(0x10000)     # never dereferenced: every call below is rejected first


@pytest.fixture(scope="module")
def B():
    import __graft_entry__
    __graft_entry__.build()
    from indexer_selected_sparse_block_gb300 import _binding
    return _binding


@pytest.mark.parametrize("n_rot,base", [(2, 10000.0), (64, 10000.0), (128, 5e6), (512, 1.5)])
def test_plain_and_divided_frequencies(B, n_rot, base):
    plain = [base ** (-2.0 * j / n_rot) for j in range(n_rot // 2)]
    got = B.SfaRope(n_rot, base=base).freqs
    assert all(abs(x - y) <= 1e-14 * y for x, y in zip(got, plain))
    got = B.SfaRope(n_rot, base=base, factor=8.0).freqs
    assert all(abs(x - y / 8) <= 1e-14 * y for x, y in zip(got, plain))


def test_frequencies_scaled_by_parts(B):
    base, orig, fast, slow, factor = 10000.0, 4096, 32.0, 1.0, 16.0
    got = B.SfaRope(64, base=base, factor=factor, original_len=orig, beta_fast=fast, beta_slow=slow).freqs
    kept = divided = between = 0
    for j, f in enumerate(got):
        p = base ** (-2.0 * j / 64)
        turns = orig * p / (2 * math.pi)
        if turns >= fast:
            assert abs(f - p) <= 1e-14 * p
            kept += 1
        elif turns <= slow:
            assert abs(f - p / factor) <= 1e-14 * p
            divided += 1
        else:
            k = (turns - slow) / (fast - slow)
            assert abs(f - (k * p + (1 - k) * p / factor)) <= 1e-14 * p
            between += 1
    assert kept and divided and between


def test_given_frequencies_and_phase_table(B):
    freqs = [0.0, 1.0, 2 * math.pi, -0.25, 123.456, 1e-9]
    r = B.SfaRope(12, freqs=freqs, pairs=True, magnitude=1.25)
    assert r.freqs == freqs and r._rope.pairs == 1 and r._rope.magnitude == 1.25
    for f, t in zip(freqs, r._rope.turns):
        frac = math.fmod(f / (2 * math.pi), 1.0) % 1.0
        # 2^-52 of the quotient, and a unit of the table
        off = abs(t / 2.0 ** 64 - frac)
        assert min(off, 1 - off) <= abs(f) * 2.0 ** -52 + 2.0 ** -63
    assert r._rope.turns[0] == 0 and r._rope.turns[2] == 0


@pytest.mark.parametrize("kw", [dict(n_rot=0), dict(n_rot=3), dict(n_rot=514), dict(n_rot=-2),
                                dict(n_rot=4, freqs=[1.0])])
def test_rope_refuses_sizes(B, kw):
    with pytest.raises(ValueError):
        B.SfaRope(**kw)


@pytest.mark.parametrize("kw", [dict(base=0.0), dict(base=-1.0), dict(base=math.nan), dict(base=math.inf),
                                dict(factor=0.0), dict(factor=math.nan), dict(original_len=-1.0),
                                dict(original_len=math.inf), dict(original_len=4096.0, beta_fast=1.0),
                                dict(original_len=4096.0, beta_fast=math.nan), dict(magnitude=math.inf),
                                dict(magnitude=1e39), dict(magnitude=math.nan),
                                dict(freqs=[math.nan] * 4), dict(freqs=[math.inf] * 4)])
def test_rope_refuses_values(B, kw):
    with pytest.raises(B.SfaError) as e:
        B.SfaRope(8, **kw)
    assert e.value.status == B.SFA_ERR_INVALID_ARG


ROW = dict(src=0x10000, src_stride=256, src_head_stride=128, dst=0x90000, dst_stride=256, dst_head_stride=128,
           src_dtype=0, dst_dtype=0, n_heads=2, d=128, rot_begin=64, to_cells=0)


def _call(B, n=1, rope=None, inverse=0, pos=FAKE, n_rows=5, slot=FAKE, n_cells=100, **row):
    if rope is None:
        rope = B.SfaRope(64)._rope
    packed = B._ROTATION.pack(*{**ROW, **row}.values())
    return B.lib().sfa_rotate_rows(n, packed * max(n, 1), ctypes.addressof(rope), inverse, pos, n_rows, slot,
                                   n_cells, None, None)


@pytest.mark.parametrize("change,rc", [
    (dict(src=0), 1), (dict(dst=0), 1), (dict(src=0x10001), 1), (dict(dst=0x90001), 1),
    (dict(src_dtype=2), 1), (dict(dst_dtype=2), 1), (dict(src_dtype=-1), 1),
    (dict(dst_dtype=1), 2),                                    # bf16 rows into fp32
    (dict(src_dtype=1, src=0x10002), 1),                       # aligned to its type
    (dict(n_heads=0), 1), (dict(d=0), 1), (dict(n_heads=1 << 20, d=1 << 20), 1),
    (dict(rot_begin=-1), 1), (dict(rot_begin=65), 1), (dict(d=63), 1),
    (dict(to_cells=2), 1), (dict(to_cells=1, slot=None), 1),
    (dict(src_stride=-1), 1), (dict(src_head_stride=-1), 1), (dict(dst_stride=-1), 1),
    (dict(dst_stride=127), 1), (dict(dst_head_stride=127), 1), (dict(dst_stride=0), 1),
    (dict(dst_stride=255), 1),                                 # rows overlap the heads of the next
    (dict(dst_stride=128, dst_head_stride=5 * 128 - 1), 1),    # heads overlap the rows of the next
    (dict(dst_stride=1 << 41), 1),
    (dict(dst=0x10000, to_cells=1), 1),                        # in place into cells
    (dict(dst=0x10000, dst_stride=384), 1),                    # in place, moved
    (dict(dst=0x10000, src_dtype=1), 1),                       # in place, another type
    (dict(n=-1), 1), (dict(n=5), 1), (dict(inverse=2), 1), (dict(pos=None), 1), (dict(n_rows=-1), 1),
    (dict(n_rows=1 << 31), 1), (dict(n_cells=-1), 1), (dict(n_cells=1 << 31), 1),
    (dict(n=0), 0), (dict(n_rows=0), 0),
])
def test_rotate_refuses(B, change, rc):
    assert _call(B, **change) == rc


@pytest.mark.parametrize("field,value", [("n_rot", 0), ("n_rot", 3), ("n_rot", 514), ("pairs", 2),
                                         ("magnitude", math.nan), ("magnitude", math.inf)])
def test_rotate_refuses_a_rope_that_is_none(B, field, value):
    r = B.SfaRope(64)._rope
    setattr(r, field, value)
    assert _call(B, rope=r) == 1


def test_binding_checks():
    from test_host_scratch import Fake, i32
    from indexer_selected_sparse_block_gb300 import _binding as B
    rope = B.SfaRope(64)
    pos = i32(4)
    x = Fake(4, 2, 128)

    def no(*a, **k):
        with pytest.raises(ValueError):
            B.sfa_rotate_rows(*a, **k)

    no([(x, x, 0)], torch.zeros(4, dtype=torch.int32), rope)             # positions on the host
    no([(x, x, 0)] * 5, pos, rope)
    no([], pos, rope, cells=[(x, Fake(9, 2, 128), 0)])                   # no slots
    no([(Fake(3, 2, 128), x, 0)], pos, rope)                             # too few rows
    no([(x, Fake(4, 1, 128), 0)], pos, rope)                             # other heads
    no([(x, Fake(4, 256), 0)], pos, rope)
    no([(x, Fake(4, 2, 128, dtype=torch.float16), 0)], pos, rope)
    no([(Fake(4, 2, 128, dtype=torch.uint8), x, 0)], pos, rope)
    no([(x, x, 0)], Fake(4, dtype=torch.int64), rope)
    no([(x, x, 0)], pos, rope, cells=[(x, Fake(9, 2, 128), 0), (x, Fake(8, 2, 128), 0)], slot=i32(4))
    no([(x, x, 0)], pos, rope, cells=[(x, Fake(9, 2, 128), 0)], slot=i32(3))
