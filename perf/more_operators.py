"""The operators of a step that verifies drafted trees over a paged cache, as they are measured:
cases, inputs, plain forms and exact values.

  rope     rotary positions of the new rows, the keys' straight into their cells  (sfa_rotate_rows)
  maps     the trees' ancestor masks and the nodes' positions                (sfa_build_tree_maps)
  attend   attention of every drafted token over the cached tokens and its ancestors, or over the
           drafted ones alone (beside the sparse attention of the cache)    (sfa_tree_attend_paged)
  commit   the accepted path of each tree, its rows to the front of the new cells, the pages behind
           it back to the free list                          (sfa_tree_accept, sfa_tree_commit)
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
        # one decode step of a full batch of a latent cache: 64 rotated dims behind 512, adjacent pairs
        dict(name="rope decode 32", op="rope", rows=32, pad=0, far=131072, h_q=16, h_kv=1, d=576,
             rot=64, split=True, pairs=True, factor=1.0, orig=0, src="bf16", dst="bf16", page=64),
        # a prefill chunk deep in a context four times as long as the trained one
        dict(name="rope chunk 2048 scaled", op="rope", rows=2048, pad=37, far=131072, h_q=16, h_kv=1,
             d=576, rot=64, split=False, pairs=False, factor=4.0, orig=32768, src="f32", dst="bf16",
             page=64),
        # whole prompts of grouped heads of 128, all dims rotated: the memory
        dict(name="rope prompt 65536", op="rope", rows=65536, pad=0, far=65536, h_q=16, h_kv=4, d=128,
             rot=128, split=False, pairs=False, factor=1.0, orig=0, src="bf16", dst="bf16", page=16),
        # a small tree for one sequence: latency
        dict(name="maps 1 x 16", op="maps", n_seq=1, old=4096, new=16, spread=0.0, pad=0),
        # trees of many sequences, some short, a padded capacity
        dict(name="maps ragged 256 x 64", op="maps", n_seq=256, old=4096, new=64, spread=1.0, pad=100),
        # one sequence's small tree: latency
        dict(name="attend 1x4096 16 nodes", op="attend", n_seq=1, old=4096, new=16, spread=0.0, page=64,
             h_q=16, h_kv=1, dkq=576, dv=512, sep_v=False, dtype="bf16", out="bf16", part="all"),
        # a full batch's trees over a latent cache
        dict(name="attend 32x32768 16 nodes", op="attend", n_seq=32, old=32768, new=16, spread=0.0,
             page=64, h_q=16, h_kv=1, dkq=576, dv=512, sep_v=False, dtype="bf16", out="bf16", part="all"),
        # large trees deep in long contexts: the tensor cores
        dict(name="attend 8x131072 63 nodes", op="attend", n_seq=8, old=131072, new=63, spread=0.0,
             page=64, h_q=16, h_kv=1, dkq=576, dv=512, sep_v=False, dtype="bf16", out="bf16", part="all"),
        # a mixed batch with grouped heads of 128, small pages
        dict(name="attend ragged 24 128 wide", op="attend", n_seq=24, old=8192, new=61, spread=1.0,
             page=16, h_q=16, h_kv=4, dkq=128, dv=128, sep_v=True, dtype="bf16", out="bf16", part="all"),
        # the drafted tokens alone, fp32 results to be merged with the sparse attention's of the cache
        dict(name="attend drafted 32 x 64", op="attend", n_seq=32, old=16411, new=64, spread=0.0,
             page=64, h_q=16, h_kv=1, dkq=576, dv=512, sep_v=False, dtype="bf16", out="f32",
             part="drafted"),
        # one sequence's tree: latency
        dict(name="commit 1 x 16", op="commit", n_seq=1, old=4096, new=16, spread=0.0, page=64, h_kv=1,
             dk=576, dv=0, dx=128, dtype="bf16"),
        # many sequences with grouped heads, V apart
        dict(name="commit ragged 256 x 64", op="commit", n_seq=256, old=1024, new=64, spread=1.0, page=16,
             h_kv=4, dk=128, dv=128, dx=128, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "maps", "attend", "attend", "attend", "commit"])
    page = rng.choice([8, 16, 24, 32, 48, 64, 128, 256])
    if op == "rope":
        d, rot, h_q, h_kv, split = rng.choice([(576, 64, 16, 1, True), (576, 64, 16, 1, False),
                                               (576, 64, 12, 1, True), (512, 64, 16, 2, False),
                                               (128, 128, 16, 4, False), (128, 64, 15, 3, False),
                                               (128, 32, 16, 16, False), (64, 64, 16, 2, False),
                                               (64, 32, 8, 8, False)])
        src, dst = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
        most = 65536 * 20 * 128 // ((h_q + h_kv) * d) // (1 if src == "bf16" else 2)
        factor, orig = rng.choice([(1.0, 0), (8.0, 0), (4.0, 32768), (32.0, 8192)])
        return dict(op=op, rows=_log_int(rng, 1, most), pad=rng.choice([0, 1, 37]),
                    far=_log_int(rng, 64, 1048576), h_q=h_q, h_kv=h_kv, d=d, rot=rot, split=split,
                    pairs=rng.random() < 0.5, factor=factor, orig=orig, src=src, dst=dst, page=page)
    new = _log_int(rng, 1, 200)
    if op == "maps":
        return dict(op=op, n_seq=_log_int(rng, 1, max(1, 16384 // new)), old=_log_int(rng, 1, 131072) - 1,
                    new=new, spread=rng.choice([0.0, 0.5, 1.0]), pad=rng.choice([0, 1, 77]))
    if op == "commit":
        h_kv, dk, dv, dx = rng.choice([(1, 576, 0, 128), (1, 576, 0, 64), (2, 512, 512, 128),
                                       (4, 128, 128, 64), (2, 64, 64, 0)])
        return dict(op=op, n_seq=_log_int(rng, 1, max(1, min(256, 16384 // new))),
                    old=_log_int(rng, 1, 1024) - 1, new=new, spread=rng.choice([0.0, 0.5, 1.0]), page=page,
                    h_kv=h_kv, dk=dk, dv=dv, dx=dx, dtype=rng.choice(["bf16", "bf16", "f32"]))
    dkq, dv, sep_v, heads = rng.choice([(576, 512, False, [(16, 1), (12, 1), (32, 2)]),
                                        (512, 512, True, [(16, 2), (16, 1)]),
                                        (512, 512, False, [(16, 1)]),
                                        (128, 128, True, [(16, 4), (16, 16), (32, 4), (15, 3)]),
                                        (64, 64, True, [(16, 2), (8, 8)])])
    h_q, h_kv = rng.choice(heads)
    dtype = rng.choice(["bf16", "bf16", "bf16", "bf16", "f32", "q8_0"])
    out = "f32" if dtype == "f32" else rng.choice(["bf16", "bf16", "f32"])
    part = rng.choice(["all", "all", "all", "drafted"])
    n_seq = _log_int(rng, 1, 48)
    old = _log_int(rng, 1, 131072) - 1
    most = 2e12 if dtype == "bf16" else 5e10
    while (2.0 * (dkq + dv) * h_q * n_seq * new * (old + new) > most
           or n_seq * (old + new) * h_kv * (dkq + (dv if sep_v else 0)) > 1.2e9
           or n_seq * h_q * new * (old + new) > 2e9):
        if n_seq > 2:
            n_seq //= 2
        elif old >= new:
            old //= 2
        else:
            new = max(1, new // 2)
    return dict(op=op, n_seq=n_seq, old=old, new=new, spread=rng.choice([0.0, 0.5, 1.0]), page=page,
                h_q=h_q, h_kv=h_kv, dkq=dkq, dv=dv, sep_v=sep_v, dtype=dtype, out=out, part=part)


def _lengths(case):
    """(cached, drafted) lengths of each sequence: part of the case's shape, so that work() knows
    them.  spread 1 draws them over the whole range, 0 makes all equal; the first sequence has the
    largest of both."""
    n, old, new, spread = case["n_seq"], case["old"], case["new"], case["spread"]
    r = random.Random(n * 1000003 + old * 101 + new * 7 + int(spread * 10))
    a = [int(old * (1 - spread * r.random())) for _ in range(n)]
    b = [max(1, int(round(new * (1 - spread * r.random())))) for _ in range(n)]
    a[0], b[0] = old, new
    return a, b


def _shape(n):
    """(levels below the root, nodes of a level) of a tree of n nodes: some more wide than deep."""
    depth = max(1, math.isqrt(n) - 1)
    w = max(1, -(-(n - 1) // depth))
    return -(-(n - 1) // w), w


def _accepted(case):
    """How many nodes of each tree will be accepted, its root and down to any level: part of the
    shape, too."""
    r = random.Random(case["n_seq"] * 31 + case["new"])
    return [1 + r.randint(0, _shape(n)[0]) for n in _lengths(case)[1]]


def _tree(n, m, r):
    """Parents of a tree of n nodes, a root and then levels of equal width, each node under any one of
    the level above, and a path of m of them.  Of the first level the path takes the node that is in
    place or one behind the path's length, so that a second pass finds the rows where they were."""
    depth, w = _shape(n)
    last = n - 1 - (depth - 1) * w                 # nodes of the last level
    lane = r.choice([0] + list(range(m - 1, last))) if m > 1 else 0
    parent, path = [-1], [0]
    for j in range(1, n):
        k, q = (j - 1) // w, (j - 1) % w
        above = 1 + (k - 1) * w
        parent.append(0 if k == 0 else above + (lane if q == lane else r.randrange(w)))
        if q == lane and len(path) < m:
            path.append(j)
    return parent, path


def _gen(seed, k):
    return torch.Generator(device=DEV).manual_seed(seed * 100 + k)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _offsets(b):
    cu = [0]
    for y in b:
        cu.append(cu[-1] + y)
    return cu


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


def _cache(n_cells, h, d, gen, dtype):
    """Rows of a cache; of a q8_0 one: d codes, d / 32 binary16 scales, zeros up to 16 bytes."""
    if dtype != "q8_0":
        return _randn((n_cells, h, d), gen, TYPES[dtype])
    codes = torch.randint(-127, 128, (n_cells, h, d), generator=gen, device=DEV, dtype=torch.int8)
    scales = (0.01 + 0.01 * torch.rand((n_cells, h, d // 32), generator=gen, device=DEV)).half()
    row = torch.zeros((n_cells, h, (d + d // 16 + 15) // 16 * 16), dtype=torch.uint8, device=DEV)
    row[..., :d] = codes.view(torch.uint8)
    row[..., d:d + d // 16] = scales.view(torch.uint8)
    return row


def _values(rows, d):
    """What the first d elements of cache rows stand for, in 32 bits."""
    if rows.dtype != torch.uint8:
        return rows[..., :d].float()
    full = {624: 576, 544: 512, 144: 128, 80: 64}[rows.shape[-1]]
    codes = rows[..., :full].contiguous().view(torch.int8).float()
    scales = rows[..., full:full + full // 16].contiguous().view(torch.float16).float()
    return (codes * scales.repeat_interleave(32, -1))[..., :d]


def _frequencies(case):
    """Radians a position of each pair, in 64 bits: base ** (-2 j / rot), all of them divided by the
    factor, or, for a trained length, those that turn less than once over it; those that turn more
    than 32 times kept, and a mean in between that goes from the one to the other with the turns."""
    rot, factor, orig = case["rot"], case["factor"], case["orig"]
    out = []
    for j in range(rot // 2):
        f = 10000.0 ** (-2.0 * j / rot)
        keep = 0.0 if orig == 0 else min(1.0, max(0.0, (orig * f / (2 * math.pi) - 1.0) / (32.0 - 1.0)))
        out.append(f * keep + f / factor * (1.0 - keep))
    return out


def _magnitude(case):
    return 1.0 if case["orig"] == 0 else 0.1 * math.log(case["factor"]) + 1.0


def _prepare_rope(case, seed, s):
    rows, d, rot, P = case["rows"], case["d"], case["rot"], case["page"]
    cap = rows + case["pad"]
    n_pages = -(-rows // P) + 3
    order = torch.randperm(n_pages, generator=_gen(seed, 1), device=DEV)
    i = torch.arange(cap, device=DEV)
    first = torch.randint(0, max(1, case["far"]), (1,), generator=_gen(seed, 2), device=DEV)
    s["pos"] = torch.where(i < rows, (first + i) % max(1, case["far"]), -1).to(torch.int32)
    slot = torch.where(i < rows, order[(i // P).clamp(max=n_pages - 1)] * P + i % P, -1)
    s["slot"] = slot.to(torch.int32)
    dst = TYPES[case["dst"]]
    s["Q"] = torch.randn((cap, case["h_q"], rot if case["split"] else d), generator=_gen(seed, 3),
                         device=DEV).to(TYPES[case["src"]])
    s["K"] = torch.randn((cap, case["h_kv"], d), generator=_gen(seed, 4), device=DEV).to(TYPES[case["src"]])
    # the queries' other dims, where the rotated ones come apart, are there already
    s["Q_out"] = _randn((cap, case["h_q"], d), _gen(seed, 5), dst)
    s["cells"] = _randn((n_pages * P, case["h_kv"], d), _gen(seed, 6), dst)
    if own:
        import indexer_selected_sparse_block_gb300 as sfa
        s["rope"] = sfa.SfaRope(rot, base=10000.0, pairs=case["pairs"], factor=case["factor"],
                                original_len=case["orig"], magnitude=_magnitude(case))
    else:
        s["freq"] = torch.tensor(_frequencies(case), dtype=torch.float64, device=DEV)
        s["mag"] = _magnitude(case)
    return s


def prepare(case, seed):
    s = dict(op=case["op"], case=case)
    if case["op"] == "rope":
        return _prepare_rope(case, seed, s)
    a, b = _lengths(case)
    cu = _offsets(b)
    r = random.Random(seed * 7919 + 11)
    parent, paths = [], []
    for n, m in zip(b, _accepted(case)):
        t, path = _tree(n, m, r)
        parent += t
        paths.append(path)
    words = (max(b) + 31) // 32
    s.update(cu=_i32(cu), total=_i32([x + y for x, y in zip(a, b)]), new_max=max(b),
             depth=1 + max(_shape(n)[0] for n in b))
    if case["op"] == "maps":
        cap = cu[-1] + case["pad"]
        s.update(parent=_i32(parent + [-1] * case["pad"]), mask=_i32([[0] * words] * cap),
                 q_pos=_i32([0] * cap), cached=_i32([0] * cap))
        return s
    P = case["page"]
    pages = [-(-(x + y) // P) for x, y in zip(a, b)]
    n_pages = sum(pages) + 5
    order = torch.randperm(n_pages, generator=_gen(seed, 1), device=DEV).to(torch.int32)
    s.update(page=P, table=_table(pages, order, max(pages)))
    if case["op"] == "commit":
        # tokens, and the model's own next ones: the path's, or none that was drafted
        token, target = [], []
        for n, path in zip(b, paths):
            tok = [r.randrange(100000) for _ in range(n)]
            tgt = [100000 + r.randrange(100000) for _ in range(n)]
            for x, y in zip(path, path[1:]):
                tgt[x] = tok[y]
            token += tok
            target += tgt
        pos = [(k, x + j) for k, (x, y) in enumerate(zip(a, b)) for j in range(y)]
        seq, at = (torch.tensor(v, device=DEV) for v in zip(*pos))
        s.update(parent=_i32(parent), token=_i32(token), target=_i32(target), free=order.clone(),
                 slot=(s["table"][seq, at // P] * P + at % P).to(torch.int32),
                 # every page is taken: the entries before the head are free for what comes back
                 head=_i32([sum(pages)]), path=_i32([[-1] * s["depth"]] * len(b)), n_acc=_i32([0] * len(b)),
                 next=_i32([0] * len(b)), len_out=_i32([0] * len(b)), head_out=_i32([0]), caches=[])
        for k, (h, d) in enumerate([(case["h_kv"], case["dk"]), (case["h_kv"], case["dv"]), (1, case["dx"])]):
            if d:
                s["caches"].append(_randn((n_pages * P, h, d), _gen(seed, 2 + k), TYPES[case["dtype"]]))
        return s
    h_q, h_kv = case["h_q"], case["h_kv"]
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    s.update(kv_max=max(x + y for x, y in zip(a, b)), scale=1.0 / math.sqrt(case["dkq"]),
             parent=_i32(parent), Q=_randn((cu[-1], h_q, case["dkq"]), _gen(seed, 2), dt),
             K=_cache(n_pages * P, h_kv, case["dkq"], _gen(seed, 3), case["dtype"]),
             V=_cache(n_pages * P, h_kv, case["dv"], _gen(seed, 4), case["dtype"]) if case["sep_v"] else None,
             O=torch.empty((cu[-1], h_q, case["dv"]), dtype=TYPES[case["out"]], device=DEV),
             lse=torch.empty((cu[-1], h_q), device=DEV))
    s["mask"] = _masks(s["parent"], s["cu"], words, s["depth"])
    return s


# ------------------------------------------------------------------------------ plain forms
def _sequence_of(cu, n_rows):
    """Sequence and place in its tree of each row; of padding those of row 0; whether it is one."""
    cu = cu.long()
    i = torch.arange(n_rows, device=DEV)
    live = i < cu[-1]
    i = torch.where(live, i, 0)
    seq = torch.searchsorted(cu[1:].contiguous(), i, right=True)
    return seq, i - cu[seq], live


def _masks(parent, cu, words, depth):
    """Bit x of row i: node x of its tree is row i's own or an ancestor's."""
    n = parent.numel()
    seq, at, live = _sequence_of(cu, n)
    first = cu.long()[seq]
    bits = torch.zeros((n, 32 * words + 1), dtype=torch.int64, device=DEV)   # the last column: no node
    cur = at
    for _ in range(depth + 1):
        bits.scatter_(1, torch.where(cur >= 0, cur, 32 * words)[:, None], 1)
        cur = torch.where(cur >= 0, parent.long()[(first + cur).clamp(min=0)], cur)
    w = (bits[:, :-1].view(n, words, 32) << torch.arange(32, device=DEV)).sum(-1)
    w = torch.where(w >= 2 ** 31, w - 2 ** 32, w)
    return torch.where(live[:, None], w, 0).to(torch.int32)


def _maps_plain(s):
    n = s["parent"].numel()
    seq, at, live = _sequence_of(s["cu"], n)
    cu = s["cu"].long()
    cached = (s["total"].long() - (cu[1:] - cu[:-1]))[seq]
    mask = _masks(s["parent"], s["cu"], s["mask"].shape[1], s["depth"])
    one = torch.arange(32, device=DEV)
    depth = ((mask.long()[:, :, None] >> one) & 1).sum((1, 2)) - 1
    return dict(mask=mask, q_pos=torch.where(live, cached + depth, -1).to(torch.int32),
                cached=torch.where(live, cached - 1, -1).to(torch.int32))


def _rotated(x, pos, freq, mag, begin, pairs, dtype):
    rot = 2 * freq.numel()
    angle = pos.double()[:, None] * freq
    c, sn = ((f(angle) * mag).float()[:, None, :] for f in (torch.cos, torch.sin))
    y = x.float()
    z = y[..., begin:begin + rot]
    if pairs:
        u, v = z[..., 0::2], z[..., 1::2]
        z = torch.stack([u * c - v * sn, u * sn + v * c], -1).flatten(-2)
    else:
        u, v = z[..., : rot // 2], z[..., rot // 2:]
        z = torch.cat([u * c - v * sn, u * sn + v * c], -1)
    return torch.cat([y[..., :begin], z, y[..., begin + rot:]], -1).to(dtype)


def _rope_plain(s):
    case = s["case"]
    d, rot = case["d"], case["rot"]
    i = torch.arange(s["pos"].numel(), device=DEV)
    i = torch.where(s["pos"] >= 0, i, 0)                   # padding repeats row 0
    at = 0 if case["split"] else d - rot
    q = _rotated(s["Q"], s["pos"], s["freq"], s["mag"], at, case["pairs"], s["Q_out"].dtype)
    k = _rotated(s["K"], s["pos"], s["freq"], s["mag"], d - rot, case["pairs"], s["cells"].dtype)
    out = s["Q_out"][..., d - rot:] if case["split"] else s["Q_out"]
    out[i] = q[i]
    s["cells"][s["slot"].long()[i]] = k[i]
    return dict(Q=s["Q_out"], K=s["cells"])


def _attend_plain(s):
    P, h_q, part = s["page"], s["Q"].shape[1], s["case"]["part"]
    K, h_kv, dkq = s["K"], s["K"].shape[1], s["Q"].shape[2]
    G, dv = h_q // h_kv, s["O"].shape[2]
    cu, total = s["cu"].long(), s["total"].long()
    n_seq, M = total.numel(), s["new_max"]
    n_new = cu[1:] - cu[:-1]
    cached = total - n_new
    T = M if part == "drafted" else s["kv_max"]
    t = torch.arange(T, device=DEV)[None, :].expand(n_seq, T)
    if part == "drafted":
        t = t + cached[:, None]
    page = torch.gather(s["table"].long(), 1, (t // P).clamp(max=s["table"].shape[1] - 1))
    cell = (page * P + t % P).clamp(min=0)                 # positions past a sequence's end: masked
    Kf = _values(K[cell], dkq).movedim(2, 1)               # [n_seq][h_kv][T][dkq]
    Vf = Kf[..., :dv] if s["V"] is None else _values(s["V"][cell], dv).movedim(2, 1)
    j = torch.arange(M, device=DEV)
    row = (cu[:-1, None] + j).clamp(max=s["Q"].shape[0] - 1)
    q = s["Q"][row].float().view(n_seq, M, h_kv, G, -1).movedim(1, 3).reshape(n_seq, h_kv, G * M, -1)
    x = torch.matmul(q, Kf.transpose(2, 3)).mul_(s["scale"]).view(n_seq, h_kv, G, M, T)
    # a key is seen that is cached, or whose bit of the row's mask is set
    node = (t - cached[:, None])[:, None, :].expand(n_seq, M, T)
    word = torch.gather(s["mask"][row].long(), 2, (node >> 5).clamp(0, s["mask"].shape[1] - 1))
    seen = ((word >> (node & 31)) & 1).bool() & (node >= 0) & (node < n_new[:, None, None])
    if part == "all":
        seen = seen | (node < 0)
    x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(n_seq, h_kv, G * M, T), Vf).view(n_seq, h_kv, G, M, dv) / l
    lse = (m + torch.log(l)).squeeze(-1)
    seq, at, _ = _sequence_of(s["cu"], s["Q"].shape[0])
    o = o.movedim(3, 1)[seq, at].reshape(-1, h_q, dv)
    return dict(O=o.to(s["O"].dtype), lse=lse.movedim(3, 1)[seq, at].reshape(-1, h_q))


def _commit_plain(s):
    cu, total, P = s["cu"].long(), s["total"].long(), s["page"]
    n_seq, M, D = total.numel(), s["new_max"], s["path"].shape[1]
    n_new = cu[1:] - cu[:-1]
    j = torch.arange(M, device=DEV)
    at = (cu[:-1, None] + j).clamp(max=s["parent"].numel() - 1)
    live = j < n_new[:, None]
    parent = torch.where(live, s["parent"].long()[at], -2)
    token, target = s["token"].long()[at], s["target"].long()[at]
    far = M + 1
    cur = torch.where(live & (parent == -1), j, far).amin(1)         # the first root
    path, count, last = [], torch.zeros_like(cur), torch.zeros_like(cur)
    for _ in range(D):
        on = cur < far
        path.append(torch.where(on, cur, -1))
        count = count + on
        last = torch.where(on, cur, last)
        want = torch.gather(target, 1, last[:, None])
        hit = (parent == last[:, None]) & (token == want) & on[:, None]
        cur = torch.where(hit, j, far).amin(1)
    path = torch.stack(path, 1)
    nxt = torch.gather(target, 1, last[:, None])[:, 0]
    k = torch.arange(D, device=DEV)
    on = path >= 0
    slot = s["slot"].long()
    src = slot[cu[:-1, None] + path.clamp(min=0)]
    dst = slot[cu[:-1, None] + torch.where(on, k, 0)]
    src = torch.where(on, src, src[:, :1])                           # padding repeats the root
    for c in s["caches"]:
        c[dst] = c[src]
    cached = total - n_new
    keep, had = (cached + count + P - 1) // P, (total + P - 1) // P
    back = had - keep
    head = s["head"].long() - back.sum()
    first = head + torch.cumsum(back, 0) - back
    x = torch.arange(M // P + 2, device=DEV)
    out = torch.cat([s["free"], s["free"][:1]])                      # the last entry: none
    to = torch.where(x < back[:, None], first[:, None] + x, s["free"].numel())
    out[to] = torch.gather(s["table"], 1, (keep[:, None] + x).clamp(max=s["table"].shape[1] - 1))
    s["free"].copy_(out[:-1])
    return dict(path=path.to(torch.int32), n_acc=count.to(torch.int32), next=nxt.to(torch.int32),
                length=(cached + count).to(torch.int32), head=head.to(torch.int32), free=s["free"],
                caches=s["caches"])


def run(s):
    if own:
        import indexer_selected_sparse_block_gb300 as sfa
        case = s["case"]
        if s["op"] == "rope":
            d, rot = case["d"], case["rot"]
            if case["split"]:
                q = (s["Q"], s["Q_out"][..., d - rot:], 0)
            else:
                q = (s["Q"], s["Q_out"], d - rot)
            sfa.sfa_rotate_rows([q], s["pos"], s["rope"], cells=[(s["K"], s["cells"], d - rot)],
                                slot=s["slot"])
            return dict(Q=s["Q_out"], K=s["cells"])
        if s["op"] == "maps":
            sfa.sfa_build_tree_maps(s["parent"], s["cu"], s["total"], s["mask"], s["q_pos"],
                                    cached_pos=s["cached"])
            return dict(mask=s["mask"], q_pos=s["q_pos"], cached=s["cached"])
        if s["op"] == "commit":
            sfa.sfa_tree_accept(s["parent"], s["token"], s["target"], s["cu"], s["path"], s["n_acc"],
                                s["next"])
            sfa.sfa_tree_commit(s["caches"], s["slot"], s["cu"], s["path"], s["n_acc"], s["total"],
                                s["page"], s["table"], s["free"], s["head"], s["len_out"], s["head_out"])
            return dict(path=s["path"], n_acc=s["n_acc"], next=s["next"], length=s["len_out"],
                        head=s["head_out"], free=s["free"], caches=s["caches"])
        sfa.sfa_tree_attend_paged(s["Q"], s["K"], s["V"], s["table"], s["page"], s["cu"], s["total"],
                                  s["mask"], s["new_max"], s["kv_max"], s["scale"], s["O"], lse=s["lse"],
                                  part=sfa.SFA_PART_DRAFTED if case["part"] == "drafted" else sfa.SFA_PART_ALL)
        return dict(O=s["O"], lse=s["lse"])
    return {"rope": _rope_plain, "maps": _maps_plain, "attend": _attend_plain,
            "commit": _commit_plain}[s["op"]](s)


# ------------------------------------------------------------------------------- what it costs
_SIZE = {"bf16": 2, "f32": 4}


def work(case):
    if case["op"] == "rope":
        rows, d, rot = case["rows"], case["d"], case["rot"]
        per = case["h_q"] * (rot if case["split"] else d) + case["h_kv"] * d
        return dict(bytes=rows * per * (_SIZE[case["src"]] + _SIZE[case["dst"]]) + 8 * (rows + case["pad"]),
                    flops=3.0 * rows * (case["h_q"] + case["h_kv"]) * rot)
    a, b = _lengths(case)
    n = len(b)
    if case["op"] == "maps":
        words = (max(b) + 31) // 32
        return dict(bytes=4 * sum(b) + 8 * n + 4 + (sum(b) + case["pad"]) * (8 + 4 * words), flops=0)
    if case["op"] == "commit":
        per = (case["h_kv"] * (case["dk"] + case["dv"]) + case["dx"]) * _SIZE[case["dtype"]]
        acc = _accepted(case)
        # a moved row is read and written; the root's place is its own
        return dict(bytes=12 * sum(b) + 24 * n + 2 * per * sum(m - 1 for m in acc) + 8 * sum(acc), flops=0)
    size = {"bf16": 2.0, "f32": 4.0, "q8_0": 1.0625}[case["dtype"]]
    q_size = 4 if case["dtype"] == "f32" else 2
    drafted = case["part"] == "drafted"
    kv = sum(y if drafted else x + y for x, y in zip(a, b))
    # a node attends its ancestors, some few; what a tile of keys computes beside them is not counted
    pairs = sum(y * (0 if drafted else x) + y * (1 + _shape(y)[0] / 2) for x, y in zip(a, b))
    row = case["h_kv"] * (case["dkq"] + (case["dv"] if case["sep_v"] else 0)) * size
    io = sum(b) * (case["h_q"] * (case["dkq"] * q_size + case["dv"] * _SIZE[case["out"]] + 4)
                   + 4 * ((max(b) + 31) // 32))
    return dict(bytes=int(kv * row + io + 4 * (kv // case["page"])),
                flops=2.0 * pairs * case["h_q"] * (case["dkq"] + case["dv"]))


# --------------------------------------------------------------------------------- exact values
def _exact_rope(case, s):
    """The rotation as a product of complex numbers."""
    d, rot = case["d"], case["rot"]
    pos = s["pos"][: case["rows"]].double()
    turn = torch.polar(torch.full_like(pos, _magnitude(case))[:, None].expand(-1, rot // 2).contiguous(),
                       torch.outer(pos, torch.tensor(_frequencies(case), dtype=torch.float64, device=DEV)))
    j = torch.arange(rot // 2, device=DEV)
    re, im = (2 * j, 2 * j + 1) if case["pairs"] else (j, j + rot // 2)

    def one(x, out, begin, to):
        for i in range(0, case["rows"], 8192):
            y = x[i: min(i + 8192, case["rows"])].double()
            z = torch.complex(y[..., begin + re], y[..., begin + im]) * turn[i: i + y.shape[0], None, :]
            y[..., begin + re], y[..., begin + im] = z.real, z.imag
            out[to[i: i + y.shape[0]]] = y

    Q, K = s["Q_out"].double(), s["cells"].double()
    rows = torch.arange(case["rows"], device=DEV)
    if case["split"]:
        one(s["Q"], Q[..., d - rot:], 0, rows)
    else:
        one(s["Q"], Q, d - rot, rows)
    one(s["K"], K, d - rot, s["slot"].long())
    return dict(Q=Q, K=K)


def exact(case, seed):
    if case["op"] == "maps":
        return None                                  # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, s)
    a, b = _lengths(case)
    cu = _offsets(b)
    if case["op"] == "commit":
        parent, token, target = s["parent"].tolist(), s["token"].tolist(), s["target"].tolist()
        src, dst = [], []
        for c0, n in zip(cu, b):
            path = [0]
            while True:
                go = [c for c in range(path[-1] + 1, n)
                      if parent[c0 + c] == path[-1] and token[c0 + c] == target[c0 + path[-1]]]
                if not go:
                    break
                path.append(go[0])
            src += [c0 + x for x in path]
            dst += [c0 + k for k in range(len(path))]
        slot = s["slot"].long()
        out = []
        for c in s["caches"]:
            z = c.double()
            z[slot[dst]] = z[slot[src]]
            out.append(z)
        return dict(path=None, n_acc=None, next=None, length=None, head=None, free=None, caches=out)
    if work(case)["flops"] > 3e12:
        return None
    dkq, dv, h_q, h_kv, P = case["dkq"], case["dv"], case["h_q"], case["h_kv"], case["page"]
    O = torch.zeros((cu[-1], h_q, dv), dtype=torch.float64, device=DEV)
    L = torch.zeros((cu[-1], h_q), dtype=torch.float64, device=DEV)
    parent = s["parent"].tolist()
    for k, (x, y) in enumerate(zip(a, b)):
        begin = x if case["part"] == "drafted" else 0
        t = torch.arange(begin, x + y, device=DEV)
        cell = s["table"][k][t // P].long() * P + t % P
        seen = torch.zeros((y, x + y - begin), dtype=torch.bool, device=DEV)
        seen[:, : x - begin] = True
        sees = [[False] * y for _ in range(y)]
        for j in range(y):
            up = parent[cu[k] + j]
            if up >= 0:
                sees[j][: j] = sees[up][: j]
            sees[j][j] = True
        seen[:, x - begin:] = torch.tensor(sees, device=DEV)
        for g in range(h_kv):
            key = _values(s["K"][cell, g], dkq).double()
            val = key[:, :dv] if s["V"] is None else _values(s["V"][cell, g], dv).double()
            for h in range(g * (h_q // h_kv), (g + 1) * (h_q // h_kv)):
                z = s["Q"][cu[k]: cu[k + 1], h].double() @ key.t() / math.sqrt(dkq)
                z = torch.where(seen, z, torch.full_like(z, -math.inf))
                top = z.max(1).values
                e = torch.exp(z - top[:, None])
                den = e.sum(1)
                O[cu[k]: cu[k + 1], h] = (e @ val) / den[:, None]
                L[cu[k]: cu[k + 1], h] = top + torch.log(den)
    return dict(O=O, lse=L)
