"""The phase table of a rotation against exact arithmetic: frequencies of either sign and any size."""
from fractions import Fraction

import pytest

PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803")


@pytest.fixture(scope="module")
def B():
    import __graft_entry__
    __graft_entry__.build()
    from indexer_selected_sparse_block_gb300 import _binding
    return _binding


def small():
    """Frequencies over 40 powers of ten, of both signs."""
    f = [x * 10.0 ** -k for k in range(36) for x in (1.0, 3.7, 6.123456789)]
    return [s * x for x in f for s in (1, -1)]


@pytest.mark.parametrize("freqs", [small(), [10000.0 ** (-j / 32) for j in range(32)], [-(5e6 ** (-j / 64)) for j in range(64)],
                                   [0.5 * k - 11 for k in range(46)]])
def test_turns(B, freqs):
    """Of f / 2 pi turns a position, in units of 2^-64: off by the double quotient's rounding, 2^-53 of it, by
    2 pi's own, 2^-54.5, and by half a unit; together |f| 2^-55 + 2^-65."""
    r = B.SfaRope(2 * len(freqs), freqs=freqs)
    for f, t in zip(freqs, r._rope.turns):
        off = (Fraction(t, 1 << 64) - Fraction(f) / (2 * PI)) % 1
        assert min(off, 1 - off) <= abs(Fraction(f)) / (1 << 55) + Fraction(1, 1 << 65), f


def test_opposite_frequencies_turn_alike(B):
    f = small()[::2]
    a, b = B.SfaRope(2 * len(f), freqs=f)._rope.turns, B.SfaRope(2 * len(f), freqs=[-x for x in f])._rope.turns
    assert all((x + y) % (1 << 64) == 0 for x, y in zip(a, b))
