"""The merge of dealt-out lists (chunk attention of 128- and 64-wide heads) that many slots have a
part of: around 32, 64 and 128 of them, where the merge looks at the next 32 slots or does not."""
import math
import random

import pytest
import torch

from paged_util import UBF, check_close, g_sum
from share_util import pieces, slots_of

pytestmark = pytest.mark.gpu

sfa = pytest.importorskip("indexer_selected_sparse_block_gb300")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    return torch.device("cuda:0")


def workspace(lens, h_q, h_kv, d):
    most = max(n for _, n in lens)
    return sfa.sfa_chunk_attend_workspace_bytes(sfa.SFA_BF16, len(lens), sum(n for _, n in lens), h_q, h_kv, d, d,
                                                True, most, max(a + n for a, n in lens), sfa.SFA_F32)


def run_and_check(dev, lens, h_q, h_kv, d, page=64):
    """The call on random pages against softmax in 64 bits, within the bounds of
    paged_util.attend_reference (two bf16 halves of a weight).  Returns each list's slots."""
    g = torch.Generator(device=dev).manual_seed(sum(a for a, _ in lens) + d)
    G, total = h_q // h_kv, [a + n for a, n in lens]
    n_pg = [-(-t // page) for t in total]
    order = torch.randperm(sum(n_pg) + 2, generator=g, device=dev).to(torch.int32)
    table = torch.full((len(lens), max(n_pg)), -1, dtype=torch.int32, device=dev)
    at, cu = 0, [0]
    for s, k in enumerate(n_pg):
        table[s, :k] = order[at:at + k]
        at += k
        cu.append(cu[-1] + lens[s][1])
    randn = lambda n, h: torch.randn((n, h, d), generator=g, device=dev).to(torch.bfloat16)
    K, V, Q = randn(order.numel() * page, h_kv), randn(order.numel() * page, h_kv), randn(cu[-1], h_q)
    O = torch.full((cu[-1], h_q, d), 7.0, device=dev)
    lse = torch.full((cu[-1], h_q), 7.0, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    need = workspace(lens, h_q, h_kv, d)
    most = max(n for _, n in lens)
    slots = slots_of(need, min(most * G, 256), d)
    assert slots                                            # the work is dealt out
    ws = torch.full((need,), 255, dtype=torch.uint8, device=dev)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
    scale = 1 / math.sqrt(d)
    sfa.sfa_chunk_attend_paged(Q, K, V, table, page, i32(cu), i32(total), most, max(total), scale, O, lse=lse,
                               workspace=ws, dev_status=status)
    assert sfa.sfa_read_device_status(status) == 0
    for s, (a, n) in enumerate(lens):
        t = torch.arange(total[s], device=dev)
        cell = table[s].long()[t // page] * page + t % page
        for i in range(h_kv):
            k, v = K[cell, i].double(), V[cell, i].double()
            q = Q[cu[s]:cu[s + 1], i * G:(i + 1) * G].double()          # [n][G][d]
            x = torch.einsum("ngd,td->ngt", q, k) * scale
            x.masked_fill_((t[None, :] > a + torch.arange(n, device=dev)[:, None])[:, None], -math.inf)
            p = torch.softmax(x, -1)
            ref, ref_l = p @ v, torch.logsumexp(x, -1)
            size = torch.einsum("ngd,td->ngt", q.abs(), k.abs()).amax(-1) * scale
            dd = size * g_sum(d) + 2.0 ** -20 * (1 + size)
            tol = (2 * dd + 2 * UBF ** 2 + g_sum(total[s]))[..., None] * (p @ v.abs()) + 1e-30
            rows, heads = slice(cu[s], cu[s + 1]), slice(i * G, (i + 1) * G)
            check_close(O[rows, heads], ref.cpu(), tol.cpu(), f"O of sequence {s}, KV head {i}")
            check_close(lse[rows, heads], ref_l.cpu(), (dd + g_sum(total[s]) + 2.0 ** -22 * ref_l.abs()).cpu(),
                        f"lse of sequence {s}, KV head {i}")
    return [c for c, _ in pieces(lens, h_q, h_kv, slots)]


@pytest.mark.parametrize("length", [15896, 16000, 16024, 16128, 16152, 16256, 16280, 16384])
def test_one_token_of_grouped_heads(dev, length):
    """One token, four KV heads: lists of 31 to 33 slots each, one behind the other."""
    counts = run_and_check(dev, [(length - 1, 1)], 16, 4, 128)
    if torch.cuda.get_device_properties(dev).multi_processor_count == 152 and length <= 16128:
        assert 32 in counts[:-1]


@pytest.mark.parametrize("h_q,h_kv,d,slots", [(q, k, d, n) for q, k, d in [(16, 2, 64), (16, 4, 128), (8, 1, 64), (16, 1, 128)]
                                               for n in (31, 32, 33, 63, 64, 65, 95, 96, 97, 127, 128, 129) if n * k < 140])
def test_lists_of_slots(dev, h_q, h_kv, d, slots):
    """A few decodes and short chunks of which one list, not the last, has parts in `slots` slots."""
    r = random.Random(slots * 100 + d + h_kv)
    for _ in range(5000):
        lens = [(int(2 ** r.uniform(4, 16.5)), r.choice([1, 1, 1, 2, 3])) for _ in range(r.randint(2, 3))]
        if h_kv == 1:
            lens[0] = (int(2 ** r.uniform(14, 16.9)), 1)
        have = slots_of(workspace(lens, h_q, h_kv, d), min(max(n for _, n in lens) * (h_q // h_kv), 256), d)
        if have and slots in [c for c, _ in pieces(lens, h_q, h_kv, have)][:-1]:
            break
    else:
        pytest.skip("no such list found for this device's slots")
    assert slots in run_and_check(dev, lens, h_q, h_kv, d)
