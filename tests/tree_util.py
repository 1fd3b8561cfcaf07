"""Plain implementations of the drafted-tree operators, and their inputs."""
import math

import torch

from paged_util import g_sum


def random_tree(n, r, roots=1, chain=0.3):
    """Parents of n nodes: some roots, the others under any earlier node, often the last one."""
    return [-1 if j < roots else j - 1 if r.random() < chain else r.randrange(j) for j in range(n)]


def ancestors(parent):
    """seen[j][x]: node x is j or above it (a parent that is none: a root)."""
    n = len(parent)
    seen = [[False] * n for _ in range(n)]
    depth = [0] * n
    for j, up in enumerate(parent):
        if 0 <= up < j:
            seen[j][:j] = seen[up][:j]
            depth[j] = depth[up] + 1
        seen[j][j] = True
    return seen, depth


def pack(seen, words):
    """Rows of truth values as int32 words."""
    out = []
    for row in seen:
        w = [0] * words
        for x, on in enumerate(row):
            if on:
                w[x // 32] |= 1 << (x % 32)
        out.append([v - (1 << 32) if v >> 31 else v for v in w])
    return out


def accept_reference(parent, token, target, root, most):
    """path, its length, the next token."""
    path, cur, want = [], -1, root
    while len(path) < most:
        hit = [c for c in range(cur + 1, len(parent)) if parent[c] == cur and (cur < 0 and root is None or token[c] == want)]
        if not hit:
            break
        cur = hit[0]
        path.append(cur)
        want = target[cur]
    return path, len(path), want if path else (-1 if root is None else root)


def tree_attend_exact(Q, K, V, cells, cu, total, seen, scale, dv, drafted=False, product=0.0, p_round=0.0, o_round=0.0):
    """Double-precision attention of drafted nodes (seen[s][j][x]: node j of sequence s attends node x)
    and a bound on each element's error, that of paged_util.attend_exact: scores off by
    size (g(dkq) + product) + 2^-20 (1 + size), results by (2 of that + 2 p_round + product + g(keys)) A and
    their own rounding.  cells[s]: the cell of each position, below 0: none."""
    dev, h_q, h_kv = Q.device, Q.shape[1], K.shape[1]
    G = h_q // h_kv
    O = torch.zeros((Q.shape[0], h_q, dv), dtype=torch.float64, device=dev)
    L = torch.full((Q.shape[0], h_q), -math.inf, dtype=torch.float64, device=dev)
    tol_o, tol_l = torch.zeros_like(O), torch.zeros((Q.shape[0], h_q), dtype=torch.float64, device=dev)
    for s in range(len(total)):
        n = cu[s + 1] - cu[s]
        if n == 0:
            continue
        a = total[s] - n
        cell = torch.as_tensor(cells[s], dtype=torch.long, device=dev)[:total[s]]
        on = torch.zeros((n, total[s]), dtype=torch.bool, device=dev)
        on[:, :a] = not drafted
        on[:, a:] = torch.tensor(seen[s], device=dev)[:n, :n]
        on &= cell >= 0
        cell = cell.clamp(min=0)
        any_, cnt = on.any(1)[:, None, None], on.sum(1)
        g_keys = torch.tensor([g_sum(int(c)) for c in cnt], dtype=torch.float64, device=dev)[:, None]
        for i in range(h_kv):
            rows, heads = slice(cu[s], cu[s + 1]), slice(i * G, (i + 1) * G)
            used = on.any(0)
            k = torch.where(used[:, None], K[cell, i].double(), 0.0)
            v = k[:, :dv] if V is None else torch.where(used[:, None], V[cell, i].double(), 0.0)
            q = Q[rows, heads].double()
            x = (torch.einsum("ngd,td->ngt", q, k) * scale).masked_fill(~on[:, None], -math.inf)
            p = torch.where(any_, torch.softmax(x, -1), torch.zeros_like(x))
            O[rows, heads], L[rows, heads] = p @ v, torch.logsumexp(x, -1)
            size = torch.einsum("ngd,td->ngt", q.abs(), k.abs()).masked_fill(~on[:, None], 0.0).amax(-1) * abs(scale)
            d = size * (g_sum(q.shape[-1]) + product) + 2.0 ** -20 * (1 + size)
            tol_o[rows, heads] = ((2 * d + 2 * p_round + product + g_keys)[..., None] * (p @ v.abs())
                                  + o_round * O[rows, heads].abs() + 1e-30)
            tol_l[rows, heads] = d + g_keys + 2.0 ** -22 * torch.where(any_[..., 0], L[rows, heads], 0.0).abs()
    return O.cpu(), L.cpu(), tol_o.cpu(), tol_l.cpu()
