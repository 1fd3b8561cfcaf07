"""Queries of q8_0 trees over all of bf16's range: a row is binary16 times a power of two of its own, its largest
value brought to 2^14 .. 2^15.  A bf16 value of 2^-17 or more there is exact (eight bits, the last at 2^-24 at
least), a smaller one off by half of binary16's smallest step, 2^-25, which is 2^-39 of the row's largest."""
import math

import pytest
import torch

from paged_util import check_close
from test_gpu_chunk import N64, N128, W512, WIDE
from test_gpu_tree_attend import Trees, q8_values
from tree_util import tree_attend_exact

pytestmark = pytest.mark.gpu

sfa = pytest.importorskip("indexer_selected_sparse_block_gb300")
DEV = "cuda"

LENS = [(300, 20), (0, 40), (64, 1)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("power", [-124, -100, -20, 100, 117, 124])
@pytest.mark.parametrize("shape", [WIDE, W512, N128, N64])
def test_queries_of_any_size(shape, power, out):
    """Queries times 2^power, scores as ever by the scale."""
    c = Trees(LENS, 16, shape, "q8", out, seed=1)
    ok = c.cu[-1]
    c.Q[:ok] = (c.Q[:ok].double() * 2.0 ** power).to(torch.bfloat16)
    assert bool(torch.isfinite(c.Q[:ok].float()).all())
    c.scale = 2.0 ** -power / math.sqrt(c.dkq)
    assert c.call() == 0
    c.check()


@pytest.mark.parametrize("shape", [WIDE, W512, N128, N64])
@pytest.mark.parametrize("below", [8, 24, 30])
def test_one_large_dim(shape, below):
    """A dim 2^below times the others', against which the keys have nothing: the others decide, and are exact."""
    c = Trees(LENS, 16, shape, "q8", "f32", seed=2)
    c.Q[:, :, 1:] = torch.where(c.Q[:, :, 1:].abs() < 0.5, 0.5, c.Q[:, :, 1:])
    c.Q[:, :, 0] = 2.0 ** (below - 1)
    c.K[..., 0] = 0                                     # its code
    c.Kv = q8_values(c.K, c.dkq)
    if not c.sep:
        assert float(c.Kv[..., 0].abs().max()) == 0.0
    c.scale = 4.0 / math.sqrt(c.dkq)                     # scores of several units
    assert c.call() == 0
    # scores are sums of exact products, so their bound is that of the dims that count: of Q without dim 0
    Q = c.Q.clone()
    Q[..., 0] = 0
    ref, ref_l, tol, tol_l = tree_attend_exact(Q, c.Kv, c.Vv, c.cells, c.cu, c.total, c.seen, c.scale, c.dv, product=2.0 ** -15)
    n = c.cu[-1]
    check_close(c.O[:n], ref[:n], tol[:n], "O")
    check_close(c.lse[:n], ref_l[:n], tol_l[:n], "lse")
