"""SfaPagedCache beyond one stream's plain steps: streams, refusals, other cache types, and a free
list that runs out."""

import pytest
import torch

from paged_util import UBF, attend_exact, check_close

pytestmark = pytest.mark.gpu

sfa = pytest.importorskip("indexer_selected_sparse_block_gb300")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    return torch.device("cuda:0")


def lens(dev, *n):
    return torch.tensor(n, dtype=torch.int32, device=dev)


def test_release_behind_a_step_on_another_stream(dev):
    """A step and a release on a stream that still has other work: the release sees the step's
    lengths and pages."""
    c = sfa.SfaPagedCache(n_seq=2, n_pages=12, page_size=4, max_pages=6, n_tok_cap=20, h_kv=1, dkq=64, dv=64)
    K, new = torch.ones((20, 1, 64), dtype=torch.bfloat16, device=dev), lens(dev, 9, 5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)          # about 10 ms
    c.step(new, K, stream=side)
    c.release(0, stream=side)
    torch.cuda.synchronize()
    assert c.length.tolist() == [0, 5]
    assert c.page_table.tolist() == [[-1] * 6, [3, 4, -1, -1, -1, -1]]
    assert int(c.free_head) == 2
    assert sorted(c.free_pages[2:].tolist()) == sorted(set(range(12)) - {3, 4})
    assert sfa.sfa_read_device_status(c.status) == 0


def cells_of(c, s, n):
    """Cells of the first n positions of sequence s, -1 where there is none."""
    row = c.page_table[s].tolist()
    return [row[t // c.page_size] * c.page_size + t % c.page_size if row[t // c.page_size] >= 0 else -1
            for t in range(n)]


def check_attend(c, Q, new, scale, p_round=UBF ** 2, product=0.0, K=None, V=None):
    """attend of a step's tokens against the plain form on what the cache holds (or K, V)."""
    O = torch.full((Q.shape[0], Q.shape[1], c.dv), 5.0, device=Q.device)
    total = c.length.tolist()
    c.attend(Q, max(new), max(total), scale, O)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    ref, _, tol, _ = attend_exact(Q, c.K if K is None else K, c.V if V is None else V,
                                  [cells_of(c, s, t) for s, t in enumerate(total)], cu, total, scale, c.dv,
                                  product=product, p_round=p_round)
    check_close(O[:cu[-1]], ref[:cu[-1]], tol[:cu[-1]], f"step {new}")
    assert bool((O[cu[-1]:] == 5.0).all())


def test_free_list_runs_out(dev):
    """Tokens without a page are left out, from then on too; a sequence that is released and fed
    again is whole."""
    c = sfa.SfaPagedCache(n_seq=2, n_pages=4, page_size=4, max_pages=4, n_tok_cap=16, h_kv=2, dkq=64, dv=64,
                          separate_v=True)
    g = torch.Generator(device=dev).manual_seed(1)
    draw = lambda h: torch.randn((16, h, 64), generator=g, device=dev).to(torch.bfloat16)

    def step(*new):
        c.status.zero_()
        c.step(lens(dev, *new), draw(2), draw(2))
        flags = sfa.sfa_read_device_status(c.status)
        check_attend(c, draw(8), list(new), 0.125)
        return flags

    assert step(9, 7) == sfa.SFA_DEV_NO_PAGES
    assert c.page_table.tolist() == [[0, 1, 2, -1], [3, -1, -1, -1]] and c.length.tolist() == [9, 7]
    c.release(0)
    assert step(0, 1) == sfa.SFA_DEV_BAD_CELL              # position 7: a page that was not there
    assert step(0, 2) == 0                                 # positions 8 and 9: a page of their own
    assert cells_of(c, 1, 10)[4:8] == [-1] * 4 and min(cells_of(c, 1, 10)[8:]) >= 0
    c.release(1)
    assert c.length.tolist() == [0, 0] and int(c.free_head) == 0
    assert step(0, 10) == 0
    assert sfa.sfa_read_device_status(c.status) == 0       # after attend too


@pytest.mark.parametrize("kind", ["f32", "q8"])
@pytest.mark.parametrize("dkq,dv,h_q,h_kv,sep", [(576, 512, 16, 1, False), (512, 512, 8, 2, True), (128, 128, 8, 2, True),
                                                 (64, 64, 4, 4, True)])
def test_steps_of_other_caches(dev, kind, dkq, dv, h_q, h_kv, sep):
    """fp32 caches (rows, queries and values of fp32 with all their bits) and q8_0 ones over prefill,
    mixed and decode steps.  Their products are three tf32 ones: hi, an operand rounded to 11 bits, is
    off by 2^-11 at most; lo, what is left cut to 11 bits, leaves out 2^-10 of that, 2^-21; two such
    and lo lo, 2^-22, are below 2^-19."""
    q8 = kind == "q8"
    c = sfa.SfaPagedCache(n_seq=3, n_pages=60, page_size=8, max_pages=16, n_tok_cap=80, h_kv=h_kv, dkq=dkq, dv=dv,
                          separate_v=sep, d_idx=64, q8_0=q8, dtype=torch.bfloat16 if q8 else torch.float32)
    g = torch.Generator(device=dev).manual_seed(dkq)
    dt = torch.bfloat16 if q8 else torch.float32
    draw = lambda *s: torch.randn(s, generator=g, device=dev).to(dt)

    def values(x, d):                          # what q8_0 rows stand for
        if x is None or not q8:
            return x
        return (x[..., :d].contiguous().view(torch.int8).float()
                * x[..., d:d + d // 16].contiguous().view(torch.float16).float().repeat_interleave(32, -1))

    want_x = {}
    for new in ([50, 0, 7], [1, 9, 33], [1, 1, 1], [0, 60, 1]):
        before = c.length.tolist()
        X = draw(80, 64)
        c.step(lens(dev, *new), draw(80, h_kv, dkq), draw(80, h_kv, dv) if sep else None, X)
        at = 0
        for s, n in enumerate(new):
            for j in range(n):
                want_x[s, before[s] + j] = X[at + j]
            at += n
        check_attend(c, draw(80, h_q, dkq), new, dkq ** -0.5, p_round=0.0, product=2.0 ** -19, K=values(c.K, dkq),
                     V=values(c.V, dv))
        assert sfa.sfa_read_device_status(c.status) == 0
    for (s, pos), x in want_x.items():
        assert torch.equal(c.X[c.cell_of[s, pos].long()], x)
