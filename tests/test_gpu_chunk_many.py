"""Batches of many sequences whose chunks have several row tiles, dealt out or not, and lists in more
than 32 pieces: the ways through the work list that few sequences do not take."""
import random

import pytest
import torch

from share_util import slots_of
from test_gpu_chunk import N64, N128, W512, WIDE
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


def mixed(n_seq, seed, longest):
    """Mostly decodes, some empty chunks, every ninth sequence a chunk of up to 150 tokens, the last
    two a chunk and a decode."""
    r = random.Random(seed)
    lens = [(r.choice([0, 1, 127, 128, r.randrange(longest)]), r.choice([0, 1, 1, 1, 2])) for _ in range(n_seq - 2)]
    for s in range(7, n_seq - 2, 9):
        lens[s] = (r.randrange(longest), r.choice([33, 64, 65, 150]))
    return lens + [(100, 70), (longest, 1)]


@pytest.mark.parametrize("shape", [WIDE, W512, N128, N64])
@pytest.mark.parametrize("n_seq,longest", [(33, 3000), (65, 900), (170, 400), (300, 260)])
def test_mixed_batches(dev, shape, n_seq, longest):
    c = Chunks(dev, shape, mixed(n_seq, n_seq, longest), [], out="bf16", seed=n_seq)
    need = c.call()
    c.check()
    if not shape[2] or shape[0] == 512:      # 512 value dims: not dealt out
        return
    assert slots_of(need, min(150 * (c.h_q // c.h_kv), 256), c.dv)


@pytest.mark.parametrize("shape,out", [(WIDE, "bf16"), (WIDE, "f32"), (W512, "bf16")])
def test_more_than_32_pieces(dev, shape, out):
    """One token behind a long list: 64 pieces or so, the merge's second 32 among them; and three."""
    for new in (1, 3):
        c = Chunks(dev, shape, [(40000, new)], [], out=out, page=64, seed=new)
        need = c.call()
        piece = c.h_kv * new * (c.h_q // c.h_kv) * (c.dv + 2) * 4
        assert need % piece == 0 and need // piece > 32
        c.check()


def test_prompts_of_grouped_heads(dev):
    """Whole prompts of several row tiles each, from nothing, with one query head a KV head."""
    for shape in ((128, 128, True, 3, 3), (512, 512, True, 2, 2)):
        c = Chunks(dev, shape, [(0, 700), (0, 257), (0, 1), (0, 0), (0, 400)], [], seed=2)
        c.call()
        c.check()
