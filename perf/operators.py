"""The paged-serving operators as they are measured: cases, inputs, plain forms and exact values.

Three operators of one step of a paged cache:
  maps    page tables and slot maps from the sequences' lengths        (sfa_build_page_maps)
  write   the new tokens' rows into their cells                        (sfa_write_cells)
  attend  causal attention of each sequence's chunk of new tokens over its pages
                                                                       (sfa_chunk_attend_paged)
"""
import math
import random

import torch

own = False

if torch.cuda.is_available():
    DEV = torch.device("cuda")
else:
    DEV = torch.device("cpu")

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one decode step of a full batch: what every generated token pays
        dict(name="maps decode 32x131072", op="maps", n_seq=32, old=131072, new=1, spread=0.0,
             page=64, pad=0),
        # a mixed batch of many requests, chunks of up to 64 tokens, a padded capacity
        dict(name="maps ragged 256", op="maps", n_seq=256, old=4096, new=64, spread=1.0, page=16,
             pad=100),
        # admission of whole prompts
        dict(name="maps prompts 32x131072", op="maps", n_seq=32, old=0, new=131072, spread=0.0,
             page=64, pad=0),
        # a decode step's rows of a latent cache and its index keys
        dict(name="write decode 32", op="write", rows=32, h_kv=1, dk=576, dv=0, dx=128, src="bf16",
             dst="bf16", page=64, pad=0),
        # a prefill chunk with two KV heads and V apart, projected in fp32, stored as bf16
        dict(name="write chunk 2048 f32", op="write", rows=2048, h_kv=2, dk=512, dv=512, dx=128,
             src="f32", dst="bf16", page=16, pad=37),
        # the rows of whole prompts
        dict(name="write prompt 65536", op="write", rows=65536, h_kv=1, dk=576, dv=0, dx=128,
             src="bf16", dst="bf16", page=64, pad=0),
        # one new token of one sequence: latency
        dict(name="attend decode 1x4096", op="attend", n_seq=1, old=4096, new=1, spread=0.0, page=64,
             h_q=16, h_kv=1, dkq=576, dv=512, sep_v=False, dtype="bf16", out="bf16"),
        # a decode step of a full batch: the cache's bytes
        dict(name="attend decode 32x131072", op="attend", n_seq=32, old=131072, new=1, spread=0.0,
             page=64, h_q=16, h_kv=1, dkq=576, dv=512, sep_v=False, dtype="bf16", out="bf16"),
        # a prefill chunk over a cache of medium depth
        dict(name="attend 512 at 8192", op="attend", n_seq=1, old=8192, new=512, spread=0.0, page=64,
             h_q=16, h_kv=1, dkq=576, dv=512, sep_v=False, dtype="bf16", out="bf16"),
        # a mixed batch of decodes and chunks, grouped heads of 128, small pages
        dict(name="attend ragged 24, 128 wide", op="attend", n_seq=24, old=8192, new=333, spread=1.0,
             page=16, h_q=16, h_kv=4, dkq=128, dv=128, sep_v=True, dtype="bf16", out="bf16"),
        # two KV heads with V apart, fp32 results, pages that end inside every tile
        dict(name="attend 512 at 1000, 512/512", op="attend", n_seq=1, old=1000, new=512, spread=0.0,
             page=24, h_q=16, h_kv=2, dkq=512, dv=512, sep_v=True, dtype="bf16", out="f32"),
        # a long prefill chunk deep in a long context: the tensor cores
        dict(name="attend 2048 at 131072", op="attend", n_seq=1, old=131072, new=2048, spread=0.0,
             page=64, h_q=16, h_kv=1, dkq=576, dv=512, sep_v=False, dtype="bf16", out="bf16"),
    ]


def _log_int(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["maps", "write", "attend", "attend"])
    page = rng.choice([8, 16, 24, 32, 48, 64, 128, 256])
    if op == "maps":
        n_seq = _log_int(rng, 1, 2048)
        old = _log_int(rng, 1, 131072) - 1
        new = _log_int(rng, 1, max(1, min(131072, 4194304 // n_seq)))
        while n_seq * (old + new) > 8388608:
            old //= 2
        return dict(op=op, n_seq=n_seq, old=old, new=new, spread=rng.choice([0.0, 0.5, 1.0]),
                    page=page, pad=rng.choice([0, 1, 77]))
    if op == "write":
        h_kv, dk, dv, dx = rng.choice([(1, 576, 0, 128), (1, 576, 0, 64), (2, 512, 512, 128),
                                       (4, 128, 128, 64), (2, 64, 64, 0)])
        src, dst = rng.choice([("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
        most = 65536 * 704 // (h_kv * (dk + dv) + dx) // (1 if src == "bf16" else 2)
        return dict(op=op, rows=_log_int(rng, 1, min(65536, most)), h_kv=h_kv, dk=dk, dv=dv, dx=dx,
                    src=src, dst=dst, page=page, pad=rng.choice([0, 1, 37]))
    dkq, dv, sep_v, heads = rng.choice([(576, 512, False, [(16, 1), (12, 1), (32, 2)]),
                                        (512, 512, True, [(16, 2), (16, 1)]),
                                        (512, 512, False, [(16, 1)]),
                                        (128, 128, True, [(16, 4), (16, 16), (32, 4), (15, 3)]),
                                        (64, 64, True, [(16, 2), (8, 8)])])
    h_q, h_kv = rng.choice(heads)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    out = "f32" if dtype == "f32" else rng.choice(["bf16", "bf16", "f32"])
    n_seq = _log_int(rng, 1, 48)
    old = _log_int(rng, 1, 131072) - 1
    new = 1 if rng.random() < 0.25 else _log_int(rng, 1, 2048)
    most = 2e12 if dtype == "bf16" else 5e10
    while (2.0 * (dkq + dv) * h_q * n_seq * new * (old + new) > most
           or n_seq * (old + new) * h_kv * (dkq + (dv if sep_v else 0)) > 2.4e9
           or n_seq * h_q * new * (old + new) > 4e9):
        if n_seq > 2:
            n_seq //= 2
        elif old >= new:
            old //= 2
        else:
            new = max(1, new // 2)
    return dict(op=op, n_seq=n_seq, old=old, new=new, spread=rng.choice([0.0, 0.5, 1.0]), page=page,
                h_q=h_q, h_kv=h_kv, dkq=dkq, dv=dv, sep_v=sep_v, dtype=dtype, out=out)


def _lengths(case):
    """(cached, new) lengths of each sequence: part of the case's shape, so that work() knows
    them.  spread 1 draws them over the whole range (the new ones mostly short), 0 makes all
    equal; the first sequence has the largest of both."""
    n, old, new, spread = case["n_seq"], case["old"], case["new"], case["spread"]
    r = random.Random(n * 1000003 + old * 101 + new * 7 + int(spread * 10))
    a = [int(old * (1 - spread * r.random())) for _ in range(n)]
    b = [max(1, int(new * (1 - spread * r.random()) ** (1 + 2 * spread))) for _ in range(n)]
    a[0], b[0] = old, new
    return a, b


def _gen(seed, k):
    return torch.Generator(device=DEV).manual_seed(seed * 100 + k)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _table(pages, order, width):
    """A page table whose row s holds the next pages[s] pages of `order`, the rest -1."""
    n = torch.tensor(pages, device=DEV)
    table = torch.full((len(pages), width), -1, dtype=torch.int32, device=DEV)
    live = torch.arange(width, device=DEV)[None, :] < n[:, None]
    table[live] = order[: sum(pages)]
    return table


def _randn(shape, gen, dtype):
    """Standard normal values, drawn as bf16 would hold them in either type."""
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16).to(dtype)


def prepare(case, seed):
    s = dict(op=case["op"], case=case)
    if case["op"] == "maps":
        a, b = _lengths(case)
        P, n = case["page"], case["n_seq"]
        p_old = [-(-x // P) for x in a]
        width = max(-(-(x + y) // P) for x, y in zip(a, b))
        total = sum(-(-(x + y) // P) for x, y in zip(a, b))
        order = torch.randperm(total + 9, generator=_gen(seed, 1), device=DEV).to(torch.int32)
        cap = sum(b) + case["pad"]
        table = _table(p_old, order, width)
        pos = torch.arange(width * P, device=DEV)
        cells = torch.full((n, width * P), -1, dtype=torch.int32, device=DEV)
        live = pos[None, :] < _i32(a)[:, None]
        cells = torch.where(live, table[:, pos // P] * P + (pos % P).to(torch.int32), cells)
        s.update(page=P, n_pages=total + 9, len_old=_i32(a), len_new=_i32(b), table=table,
                 free=order[sum(p_old):].contiguous(), head=_i32([0]), cells=cells,
                 cu=_i32([0] * (n + 1)), total=_i32([0] * n), q_seq=_i32([0] * cap),
                 q_pos=_i32([0] * cap), slot=_i32([0] * cap), head_out=_i32([0]))
        return s
    if case["op"] == "write":
        rows, P = case["rows"], case["page"]
        cap = rows + case["pad"]
        n_pages = -(-rows // P) + 3
        order = torch.randperm(n_pages, generator=_gen(seed, 1), device=DEV)
        i = torch.arange(cap, device=DEV)
        slot = torch.where(i < rows, order[(i // P).clamp(max=n_pages - 1)] * P + i % P, -1)
        s["slot"] = slot.to(torch.int32)
        s["src"], s["dst"] = [], []
        for k, (h, d) in enumerate([(case["h_kv"], case["dk"]), (case["h_kv"], case["dv"]),
                                    (1, case["dx"])]):
            if d:
                x = torch.randn((cap, h, d), generator=_gen(seed, 2 + k), device=DEV)
                s["src"].append(x.to(TYPES[case["src"]]))
                s["dst"].append(_randn((n_pages * P, h, d), _gen(seed, 6 + k), TYPES[case["dst"]]))
        return s
    a, b = _lengths(case)
    P, h_q, h_kv = case["page"], case["h_q"], case["h_kv"]
    pages = [-(-(x + y) // P) for x, y in zip(a, b)]
    n_pages = sum(pages) + 5
    order = torch.randperm(n_pages, generator=_gen(seed, 1), device=DEV).to(torch.int32)
    dt = TYPES[case["dtype"]]
    cu = [0]
    for y in b:
        cu.append(cu[-1] + y)
    s.update(page=P, table=_table(pages, order, max(pages)), cu=_i32(cu),
             total=_i32([x + y for x, y in zip(a, b)]), new_max=max(b),
             kv_max=max(x + y for x, y in zip(a, b)), scale=1.0 / math.sqrt(case["dkq"]),
             Q=_randn((cu[-1], h_q, case["dkq"]), _gen(seed, 2), dt),
             K=_randn((n_pages * P, h_kv, case["dkq"]), _gen(seed, 3), dt),
             V=_randn((n_pages * P, h_kv, case["dv"]), _gen(seed, 4), dt) if case["sep_v"] else None,
             O=torch.empty((cu[-1], h_q, case["dv"]), dtype=TYPES[case["out"]], device=DEV),
             lse=torch.empty((cu[-1], h_q), device=DEV))
    return s


# ------------------------------------------------------------------------------ plain forms
def _maps_plain(s):
    P, table, cells = s["page"], s["table"], s["cells"]
    a, n = s["len_old"].long(), s["len_new"].long()
    first = torch.cumsum(n, 0) - n
    ends = first + n
    p_old = (a + P - 1) // P
    taken = (a + n + P - 1) // P - p_old
    base = s["head"].long() + torch.cumsum(taken, 0) - taken
    i = torch.arange(s["slot"].numel(), device=DEV)
    live = i < ends[-1]
    i = torch.where(live, i, 0)                     # padding repeats token 0 below
    seq = torch.searchsorted(ends, i, right=True)
    pos = a[seq] + i - first[seq]
    pg = pos // P
    k = pg - p_old[seq]                             # >= 0: a page taken now
    page = torch.where(k >= 0, s["free"][(base[seq] + k).clamp(min=0, max=s["free"].numel() - 1)],
                       table[seq, pg])
    slot = (page * P + pos % P).to(torch.int32)
    table[seq, pg] = page
    cells[seq, pos] = slot
    pad = torch.full_like(slot, -1)
    return dict(cu=torch.cat([torch.zeros_like(ends[:1]), ends]).to(torch.int32),
                total=(a + n).to(torch.int32), table=table, cells=cells,
                q_seq=torch.where(live, seq.to(torch.int32), pad),
                q_pos=torch.where(live, pos.to(torch.int32), pad),
                slot=torch.where(live, slot, pad),
                head=(s["head"].long() + taken.sum()).to(torch.int32))


def _write_plain(s):
    slot = s["slot"].long()
    i = torch.arange(slot.numel(), device=DEV)
    i = torch.where(slot >= 0, i, 0)                # padding repeats row 0
    out = []
    for x, y in zip(s["src"], s["dst"]):
        y[slot[i]] = x[i].to(y.dtype)
        out.append(y)
    return out


def _attend_plain(s):
    P, h_q = s["page"], s["Q"].shape[1]
    K, h_kv = s["K"], s["K"].shape[1]
    G, dv = h_q // h_kv, s["O"].shape[2]
    cu, total = s["cu"].long(), s["total"].long()
    n_seq, M, T = total.numel(), s["new_max"], s["kv_max"]
    t = torch.arange(T, device=DEV)
    page = s["table"].long()[:, t // P]
    cell = (page * P + t % P).clamp(min=0)          # positions past a sequence's end: masked
    Kf = K[cell].float().movedim(2, 1)              # [n_seq][h_kv][T][dkq]
    Vf = Kf[..., :dv] if s["V"] is None else s["V"][cell].float().movedim(2, 1)
    j = torch.arange(M, device=DEV)
    n_new = cu[1:] - cu[:-1]
    row = (cu[:-1, None] + j).clamp(max=s["Q"].shape[0] - 1)
    q = s["Q"][row].float().view(n_seq, M, h_kv, G, -1).movedim(1, 3).reshape(n_seq, h_kv, G * M, -1)
    x = torch.matmul(q, Kf.transpose(2, 3)).mul_(s["scale"]).view(n_seq, h_kv, G, M, T)
    pos = (total - n_new)[:, None] + j
    x.masked_fill_((t > pos[:, :, None])[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(n_seq, h_kv, G * M, T), Vf).view(n_seq, h_kv, G, M, dv) / l
    lse = (m + torch.log(l)).squeeze(-1)
    i = torch.arange(s["Q"].shape[0], device=DEV)
    seq = torch.searchsorted(cu[1:].contiguous(), i, right=True)
    at = i - cu[seq]
    o = o.movedim(3, 1)[seq, at].reshape(-1, h_q, dv)
    return dict(O=o.to(s["O"].dtype), lse=lse.movedim(3, 1)[seq, at].reshape(-1, h_q))


def run(s):
    if own:
        import indexer_selected_sparse_block_gb300 as sfa
        if s["op"] == "maps":
            sfa.sfa_build_page_maps(s["len_old"], s["len_new"], s["page"], s["free"], s["head"],
                                    s["n_pages"], s["table"], s["cu"], s["total"], s["q_seq"],
                                    s["q_pos"], s["slot"], s["head_out"], cell_of=s["cells"])
            return dict(cu=s["cu"], total=s["total"], table=s["table"], cells=s["cells"],
                        q_seq=s["q_seq"], q_pos=s["q_pos"], slot=s["slot"], head=s["head_out"])
        if s["op"] == "write":
            sfa.sfa_write_cells(list(zip(s["src"], s["dst"])), s["slot"])
            return s["dst"]
        sfa.sfa_chunk_attend_paged(s["Q"], s["K"], s["V"], s["table"], s["page"], s["cu"],
                                   s["total"], s["new_max"], s["kv_max"], s["scale"], s["O"],
                                   lse=s["lse"])
        return dict(O=s["O"], lse=s["lse"])
    return {"maps": _maps_plain, "write": _write_plain, "attend": _attend_plain}[s["op"]](s)


# ------------------------------------------------------------------------------- what it costs
def work(case):
    if case["op"] == "maps":
        a, b = _lengths(case)
        P, n = case["page"], case["n_seq"]
        taken = sum(-(-(x + y) // P) + (-x // P) for x, y in zip(a, b))
        # lengths in; offsets and totals out; per token q_seq, q_pos, slot and the cell map's
        # entry; per page one free entry in and one table entry out
        return dict(bytes=8 * n + 8 * n + 4 + 16 * sum(b) + 12 * case["pad"] + 8 * taken, flops=0)
    if case["op"] == "write":
        per = case["h_kv"] * (case["dk"] + case["dv"]) + case["dx"]
        size = {"bf16": 2, "f32": 4}
        return dict(bytes=case["rows"] * (per * (size[case["src"]] + size[case["dst"]]) + 4), flops=0)
    a, b = _lengths(case)
    size = 2 if case["dtype"] == "bf16" else 4
    kv = sum(x + y for x, y in zip(a, b))
    pairs = sum(y * x + y * (y + 1) // 2 for x, y in zip(a, b))
    row = case["h_kv"] * (case["dkq"] + (case["dv"] if case["sep_v"] else 0)) * size
    n_q = sum(b)
    io = n_q * case["h_q"] * (case["dkq"] * size + case["dv"] * (2 if case["out"] == "bf16" else 4) + 4)
    return dict(bytes=kv * row + io + 4 * (kv // case["page"]),
                flops=2.0 * pairs * case["h_q"] * (case["dkq"] + case["dv"]))


# --------------------------------------------------------------------------------- exact values
def exact(case, seed):
    if case["op"] == "maps":
        return None                                  # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "write":
        # the values before any rounding, in the rows that a slot names
        out = []
        rows = case["rows"]
        for x, y in zip(s["src"], s["dst"]):
            z = y.double()
            z.index_copy_(0, s["slot"][:rows].long(), x[:rows].double())
            out.append(z)
        return out
    if work(case)["flops"] > 5e12:
        return None
    a, b = _lengths(case)
    dv, h_q, h_kv, P = case["dv"], case["h_q"], case["h_kv"], case["page"]
    O = torch.zeros((sum(b), h_q, dv), dtype=torch.float64, device=DEV)
    L = torch.zeros((sum(b), h_q), dtype=torch.float64, device=DEV)
    at = 0
    for k, (x, y) in enumerate(zip(a, b)):
        t = torch.arange(x + y, device=DEV)
        cell = s["table"][k][t // P].long() * P + t % P
        for h in range(h_q):
            g = h // (h_q // h_kv)
            key = s["K"][cell, g].double()
            val = key[:, :dv] if s["V"] is None else s["V"][cell, g].double()
            for r in range(0, y, 512):
                q = s["Q"][at + r: at + min(y, r + 512), h].double()
                z = q @ key.t() / math.sqrt(case["dkq"])
                seen = t[None, :] <= x + r + torch.arange(q.shape[0], device=DEV)[:, None]
                z = torch.where(seen, z, torch.full_like(z, -math.inf))
                top = z.max(1).values
                e = torch.exp(z - top[:, None])
                den = e.sum(1)
                O[at + r: at + r + q.shape[0], h] = (e @ val) / den[:, None]
                L[at + r: at + r + q.shape[0], h] = top + torch.log(den)
        at += y
    return dict(O=O, lse=L)
