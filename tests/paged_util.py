"""Plain 64-bit implementations of the paged-serving operators, and error bounds derived from
their arithmetic.  Shared by the tests of page maps, cell writes and chunk attention."""
import math

import torch

U32, UBF = 2.0 ** -24, 2.0 ** -8     # half a step of fp32 and of bf16, relative


def maps_reference(len_old, len_new, page, free, head, n_pages, table, cap):
    """Python loops; table (a list of lists) is updated.  Returns cu, total, q_seq, q_pos, slot,
    head_out."""
    cu, q_seq, q_pos, slot = [0], [], [], []
    total = []
    width = len(table[0]) if table else 0
    head = max(head, 0)
    for s, (a, n) in enumerate(zip(len_old, len_new)):
        a, n = max(a, 0), max(n, 0)
        n = min(n, cap - cu[-1])
        for pg in range(-(-a // page), min(-(-(a + n) // page), width)):
            f = free[head] if head < len(free) else -1
            head = min(head + 1, len(free))
            table[s][pg] = f if 0 <= f < n_pages else -1
        for pos in range(a, a + n):
            pg = pos // page
            e = table[s][pg] if pg < width else -1
            q_seq.append(s)
            q_pos.append(pos)
            slot.append(e * page + pos % page if 0 <= e < n_pages else -1)
        cu.append(cu[-1] + n)
        total.append(a + n)
    pad = [-1] * (cap - cu[-1])
    return cu, total, q_seq + pad, q_pos + pad, slot + pad, min(head, len(free))


def attend_reference(Q, K, V, table, page, cu, total, scale, dv, kv_max=None, p_round=0.0,
                     o_round=0.0):
    """Double-precision chunk attention over the page table (lists of ints; entries outside the
    cache are left out) and, per element, a bound on a kernel's error.

    Bound.  Scores are fp32 sums of dkq exact products (bf16 inputs: a product has 16 significant
    bits), so an error of g(dkq) * sum_d |q_d k_d|, with g(n) = 6 sqrt(n) 2^-23 (the rounding
    errors of n sums of either sign, each at most a step: six standard deviations); scaling them
    to base 2, the subtraction of the maximum and the exponential add 2^-20 (1 + max |s|).  A
    relative error d of every weight moves the result by at most 2 d A, A_d = sum_t p_t |v_td|;
    rounding the weights by p_round moves it by 2 p_round A; summing n keys by g(n) A; the
    result's own rounding by o_round |O|."""
    Q, K = Q.double().cpu(), K.double().cpu()
    V = K[..., :dv] if V is None else V.double().cpu()
    n_q, h_q, dkq = Q.shape
    h_kv = K.shape[1]
    G = h_q // h_kv
    n_pages = K.shape[0] // page
    O = torch.zeros((n_q, h_q, dv), dtype=torch.float64)
    L = torch.full((n_q, h_q), -math.inf, dtype=torch.float64)
    tol_o, tol_l = torch.zeros_like(O), torch.zeros((n_q, h_q), dtype=torch.float64)

    def g(n):
        return 6 * math.sqrt(max(n, 1)) * 2 * U32

    for s in range(len(total)):
        n = cu[s + 1] - cu[s]
        limit = min(total[s], len(table[s]) * page, kv_max if kv_max is not None else total[s])
        pos = [t for t in range(max(limit, 0)) if 0 <= table[s][t // page] < n_pages]
        cell = torch.tensor([table[s][t // page] * page + t % page for t in pos], dtype=torch.long)
        post = torch.tensor(pos, dtype=torch.long)
        for j in range(n):
            keep = post <= total[s] - n + j
            if not bool(keep.any()):
                continue
            k, v = K[cell[keep]], V[cell[keep]]
            for h in range(h_q):
                q = Q[cu[s] + j, h]
                x = (k[:, h // G] @ q) * scale
                m = x.max()
                e = torch.exp(x - m)
                l = e.sum()
                p = e / l
                vv = v[:, h // G]
                O[cu[s] + j, h] = p @ vv
                L[cu[s] + j, h] = m + torch.log(l)
                d = (float((k[:, h // G].abs() @ q.abs()).max()) * abs(scale) * g(dkq)
                     + 2.0 ** -20 * (1 + float(x.abs().max())))
                A = p @ vv.abs()
                cnt = int(keep.sum())
                tol_o[cu[s] + j, h] = (2 * d + 2 * p_round + g(cnt)) * A + o_round * O[cu[s] + j, h].abs() + 1e-30
                tol_l[cu[s] + j, h] = d + g(cnt) + 4 * U32 * abs(float(L[cu[s] + j, h]))
    return O, L, tol_o, tol_l


def check_close(got, ref, tol, what):
    """|got - ref| <= tol everywhere; infinities in the same places."""
    got = got.double().cpu()
    inf = torch.isinf(ref)
    assert torch.equal(torch.where(inf, got, torch.zeros_like(got)),
                       torch.where(inf, ref, torch.zeros_like(ref))), f"{what}: infinities differ"
    err = torch.where(inf, torch.zeros_like(got), (got - ref).abs())
    ratio = err / torch.where(inf, torch.ones_like(tol), tol).clamp(min=1e-30)
    bad = ~(ratio <= 1)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound, worst "
                                 f"{float(ratio[~torch.isnan(ratio)].max()) if (~torch.isnan(ratio)).any() else math.nan:.3g} x, "
                                 f"first at {torch.nonzero(bad)[0].tolist()}, {int(torch.isnan(got).sum())} NaN")


def g_sum(n):
    """The bound of attend_reference on a sum of n terms in fp32, relative to its terms' sizes."""
    return 6 * math.sqrt(max(n, 1)) * 2 * U32


def attend_exact(Q, K, V, cells, cu, total, scale, dv, product=0.0, p_round=0.0, o_round=0.0):
    """What attend_reference gives, for long lists: on the tensors' device, a KV head at a time, from
    each sequence's cells of its positions (a list or tensor; below 0: left out).  product: how far
    one product of a score or a value may be off, relative, at worst and all one way; it moves a
    score by product sum_d |q_d k_d|, and so a result by twice that A and by product A itself."""
    dev, h_q, h_kv = Q.device, Q.shape[1], K.shape[1]
    G = h_q // h_kv
    O = torch.zeros((Q.shape[0], h_q, dv), dtype=torch.float64, device=dev)
    L = torch.full((Q.shape[0], h_q), -math.inf, dtype=torch.float64, device=dev)
    tol_o, tol_l = torch.zeros_like(O), torch.zeros((Q.shape[0], h_q), dtype=torch.float64, device=dev)
    for s in range(len(total)):
        n = cu[s + 1] - cu[s]
        cell = torch.as_tensor(cells[s], dtype=torch.long, device=dev)
        pos = torch.nonzero(cell >= 0)[:, 0]
        cell = cell[pos]
        if n == 0 or pos.numel() == 0:
            continue
        seen = pos[None, :] <= total[s] - n + torch.arange(n, device=dev)[:, None]
        any_, cnt = seen.any(1)[:, None, None], seen.sum(1)
        g_keys = torch.tensor([g_sum(int(c)) for c in cnt], dtype=torch.float64, device=dev)[:, None]
        for i in range(h_kv):
            rows, heads = slice(cu[s], cu[s + 1]), slice(i * G, (i + 1) * G)
            k = K[cell, i].double()
            v = k[:, :dv] if V is None else V[cell, i].double()
            q = Q[rows, heads].double()
            x = (torch.einsum("ngd,td->ngt", q, k) * scale).masked_fill(~seen[:, None], -math.inf)
            p = torch.where(any_, torch.softmax(x, -1), torch.zeros_like(x))
            O[rows, heads], L[rows, heads] = p @ v, torch.logsumexp(x, -1)
            size = torch.einsum("ngd,td->ngt", q.abs(), k.abs()).masked_fill(~seen[:, None], 0.0).amax(-1) * abs(scale)
            d = size * (g_sum(q.shape[-1]) + product) + 2.0 ** -20 * (1 + size)
            tol_o[rows, heads] = ((2 * d + 2 * p_round + product + g_keys)[..., None] * (p @ v.abs())
                                  + o_round * O[rows, heads].abs() + 1e-30)
            tol_l[rows, heads] = d + g_keys + 4 * U32 * torch.where(any_[..., 0], L[rows, heads], 0.0).abs()
    return O.cpu(), L.cpu(), tol_o.cpu(), tol_l.cpu()
