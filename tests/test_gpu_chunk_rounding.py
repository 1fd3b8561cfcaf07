"""What the chunk attention's roundings come to where they count most: one key with nearly all the
weight, and fp32 operands with all their bits."""
import math

import pytest
import torch

from paged_util import UBF, attend_exact, check_close, g_sum
from test_gpu_chunk import N64, N128, W512, W512K, WIDE
from test_gpu_chunk_nonfinite import Chunks

pytestmark = pytest.mark.gpu

sfa = pytest.importorskip("indexer_selected_sparse_block_gb300")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    return torch.device("cuda:0")


@pytest.mark.parametrize("shape", [WIDE, W512, N128, N64])
@pytest.mark.parametrize("above", [5.3, 6.6, 7.4])
def test_one_key_has_the_weight(dev, shape, above):
    """bf16 results: a key of a later tile scores `above` (base 2) over all of the first tile's, less
    than what the running maximum moves for, and 14 over its own tile's: its weight is no power of two.
    O is that key's values but for weights of at most 2^-8 each, and all of one row's elements are off by
    the one rounding of the large weight.
    Bound: that rounding and the result's own, UBF |O| each; the other weights' UBF of their share of
    A = sum p |v|, twice (in the sum and against the whole); the scores' and sums' as ever."""
    dkq, dv, sep, h_q, h_kv = shape
    c = Chunks(dev, shape, [(299, 1)], [], out="bf16", seed=int(above * 10))
    G = h_q // h_kv
    u = torch.sign(torch.randn((h_kv, dkq), device=dev, generator=torch.Generator(device=dev).manual_seed(1)))
    c.Q[:] = u.repeat_interleave(G, 0).to(c.dt)
    base = torch.randn((300, h_kv, dkq), device=dev, generator=torch.Generator(device=dev).manual_seed(2)) * 0.02
    step = math.log(2) / (c.scale * dkq)             # along u: one of base 2
    high = 200                                       # in the second tile of 128
    t = torch.arange(300, device=dev)
    level = torch.where(t < 128, -9.0, above - 14.0)     # of the scores, base 2
    level[5], level[high] = 0.0, above
    c.K[c.cells[0]] = (base + (level * step)[:, None, None] * u).to(c.dt)
    c.clean = (c.K.clone(), c.clean[1])
    c.call()
    K, V = c.clean
    ref, ref_l, _, tol_l = attend_exact(c.Q, K, V, c.cells, c.cu, c.total, c.scale, dv)
    for i in range(h_kv):
        k = K[c.cells[0], i].double()
        v = k[:, :dv] if V is None else V[c.cells[0], i].double()
        q = c.Q[0, i * G:(i + 1) * G].double()
        x = q @ k.t() * c.scale
        p = torch.softmax(x, -1)
        rest = p.clone()
        rest[:, high] = 0
        size = (q.abs() @ k.abs().t()).amax(-1) * c.scale
        d = size * g_sum(dkq) + 2.0 ** -20 * (1 + size)
        heads = slice(i * G, (i + 1) * G)
        O = ref[0, heads].abs()
        tol = 2 * UBF * O + (2 * UBF * (rest @ v.abs()) + (2 * d + g_sum(300))[:, None] * (p @ v.abs())).cpu() + 1e-30
        # UBF of the large weight's share, which is O but for the others'
        tol += UBF * (rest @ v.abs()).cpu()
        check_close(c.O[0, heads], ref[0, heads], tol, f"O of KV head {i}")
    check_close(c.lse, ref_l, tol_l, "lse")


@pytest.mark.parametrize("shape", [WIDE, W512, W512K, N128, N64])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_fp32_operands_with_all_their_bits(dev, shape, out):
    """Queries, keys and values of fp32 that bf16 does not hold: the second halves of all three count.
    (The first halves alone would leave 2^-11 of a product.)"""
    c = Chunks(dev, shape, [(700, 20), (0, 33), (2500, 1), (90, 1)], [], out=out, dtype="f32", seed=shape[0], full=True)
    c.call()
    K, V = c.clean
    ref, ref_l, tol, tol_l = attend_exact(c.Q, K, V, c.cells, c.cu, c.total, c.scale, c.dv, product=2.0 ** -19,
                                          o_round=UBF if out == "bf16" else 0.0)
    check_close(c.O, ref, tol, "O")
    check_close(c.lse, ref_l, tol_l, "lse")
    if out == "f32":
        # What an element's bound leaves room for, the whole does not: with operands of size one a score,
        # sum of dkq products times dkq^-1/2, is off by 2^-19 (products, either sign) and, of 3 dkq / 64
        # additions that cut at most a step of a running sum of size one, by 27 2^-23 at most; a result
        # by as much of its size, its keys' errors being of either sign as its values are, and by 2^-19
        # for the products with V and their additions again: below 2^-16 in all.
        def off(x):
            return float((x.double() - ref).norm() / ref.norm())
        assert off(c.O.cpu()) <= 2.0 ** -16
        # without the second half of Q, or K, or V it is not
        hi = lambda x: ((x.view(torch.int32) + 0x1000) & -0x2000).view(torch.float32)
        for q, k, v in ((hi(c.Q), K, V), (c.Q, hi(K), K[..., :c.dv] if V is None else V),
                        (c.Q, K, hi(K[..., :c.dv] if V is None else V))):
            low = attend_exact(q, k, v, c.cells, c.cu, c.total, c.scale, c.dv)[0]
            assert off(low) > 2.0 ** -14
