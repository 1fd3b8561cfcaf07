"""The dealt-out work of the chunk attention (128- and 64-wide heads, bf16), in whole numbers on the
host: which slots have keys of each list, for tests that need lists of a given number of pieces."""

PIECE_KEYS = 448      # what a piece's start and end weigh, in keys


def slots_of(need, part_rows, dv):
    """Slots of a workspace of `need` bytes for dealt-out work (two row tiles of partial results and
    notes a slot), or None where the work is not dealt out."""
    return next((s for s in range(1, 161) if need == 2 * s * part_rows * (dv + 2) * 4 + 32 * s), None)


def pieces(lens, h_q, h_kv, slots):
    """For each list in the line (sequence by sequence, KV head by KV head, row tile by row tile):
    (slots from its first to its last, those of them that have keys of it).
    lens: (cached before, new) of each sequence."""
    item_q = 2 * (128 // (h_q // h_kv))
    units = []
    for a, n in lens:
        tiles = -(-n // item_q)
        for _ in range(h_kv):
            for j in range(tiles):
                keys = a + min((j + 1) * item_q, n)
                units.append((keys, keys + PIECE_KEYS))
    W = sum(w for _, w in units)
    per, rem = divmod(W, slots)

    def border(c):
        return per * c + min(c, rem)

    out, u0 = [], 0
    for keys, w in units:
        first = next(c for c in range(slots) if border(c + 1) > u0)
        last = next(c for c in range(first, slots) if border(c + 1) >= u0 + w)
        live = 0
        for c in range(first, last + 1):
            a, b = border(c) - u0, border(c + 1) - u0
            k0 = 0 if a <= 0 else min((a + 64) & ~127, keys)
            k1 = keys if b >= w else min((b + 64) & ~127, keys)
            live += k0 < k1
        out.append((last - first + 1, live))
        u0 += w
    return out
