// chunk_common.cuh -- what the chunk attention kernels share (chunk.cu: the kernel of fp32
// and q8_0 caches, the merge of split lists, the launch plan and the C entry points).
//
// A chunk is the new tokens of one sequence: rows cu[s] .. cu[s + 1] of the packed Q, at the
// last positions of the sequence's total[s] cached tokens.  The rows of one KV head are (query,
// head of the group) pairs, flattened query-major; a work item is a tile of such rows of one
// sequence and KV head, and a piece of its keys 0 .. p_last.
#pragma once

#include "sfa_common.cuh"

namespace sfa {
namespace chunk {

constexpr float kLog2e = 1.4426950408889634f;

struct Params {
    const void *Q, *K, *V;
    const int32_t *table, *cu, *total;
    void *O;
    float *lse, *part_o, *part_ml;
    int4 *slot_info;     // [slots][2], see Share
    int32_t *status;
    int64_t table_stride;
    FastDiv page_div;
    int page, n_pages, n_seq, n_q, h_q, h_kv, G;
    int o_bf16;          // O is bf16 (else fp32)
    int items;           // row tiles of all sequences, at most
    int item_rows;       // rows of a tile
    int part_rows;       // of those, the ones a tile of partial results has room for (no chunk has more)
    int item_q;          // queries of a tile, 0: tiles cut the flattened rows anywhere
    int one_tile;        // no chunk has more than one row tile
    int slots;           // > 0: the work is dealt out evenly to this many CTAs, see Share;
                         // 0: a CTA (pair) for each item, KV head and piece of n_split
    int n_split;         // pieces a list is cut into, at most
    int split_keys;      // keys of a piece
    int n_new_max;       // the caller's bound on a chunk's length
    int64_t n_kv_max;    // the caller's bound on total[s]
    float scale_log2;
};

// Sequence s: its first row in Q, its chunk's length, its cached tokens.  Offsets that are not
// ascending within [0, n_q] give an empty chunk, a chunk longer than n_new_max its first
// n_new_max queries, both flagged (flag: one caller per sequence).
struct Seq {
    int c0, n, total;
};
__device__ __forceinline__ Seq make_seq(const Params &p, int c0, int c1, int total, bool flag) {
    Seq q;
    q.c0 = c0;
    q.total = max(total, 0);   // negative: positions below 0 all the same, and no overflow
    bool bad = q.c0 < 0 || c1 < q.c0 || c1 > p.n_q;
    q.n = bad ? 0 : c1 - q.c0;
    // the positions follow from the true length: a clipped chunk keeps its first queries
    if (q.n > p.n_new_max || total < q.n || q.total > p.n_kv_max ||
        (int64_t)q.total > p.table_stride * p.page)
        bad = true;
    if (bad && flag) set_status(p.status, SFA_DEV_BAD_QUERY);
    return q;
}
__device__ __forceinline__ Seq load_seq(const Params &p, int s, bool flag) {
    return make_seq(p, p.cu[s], p.cu[s + 1], p.total[s], flag);
}

// Row tiles of a chunk of n queries.
__device__ __forceinline__ int n_items(const Params &p, int n) {
    n = min(n, p.n_new_max);
    return p.item_q > 0 ? (n + p.item_q - 1) / p.item_q
                        : (int)(((int64_t)n * p.G + p.item_rows - 1) / p.item_rows);
}

// A work item: tile `tile` of sequence `seq`; seq < 0: past the last tile.
struct Item {
    int seq, tile;
    Seq q;
};
// By one whole warp: the row tiles of the sequences are counted 32 sequences at a time.  Where no
// chunk has more than one tile, item s is sequence s (2048 decode steps, 576 wide, lists of up to
// 500 keys: 837 us with the count, 388 so).
// lead: one caller per item, which flags lengths and offsets that cannot be.
__device__ __forceinline__ Item find_item(const Params &p, int item, bool lead) {
    const int lane = threadIdx.x & 31;
    Item it;
    it.seq = -1;
    it.tile = 0;
    it.q = Seq{0, 0, 0};
    if (p.one_tile) {
        if (item < p.n_seq) it.q = load_seq(p, item, lead && lane == 0);
        if (it.q.n > 0) it.seq = item;
        return it;
    }
    const bool flag = lead && item == 0;
    int base = 0;
    for (int s0 = 0; s0 < p.n_seq; s0 += 32) {
        const int s = s0 + lane;
        Seq q{0, 0, 0};
        if (s < p.n_seq) q = load_seq(p, s, flag);
        const int cnt = n_items(p, q.n);
        int x = cnt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x += y;
        }
        const unsigned in = __ballot_sync(0xFFFFFFFFu, item < base + x);
        if (in && !flag) {
            const int l = __ffs(in) - 1;
            it.seq = s0 + l;
            it.tile = item - base - __shfl_sync(0xFFFFFFFFu, x - cnt, l);
            it.q.c0 = __shfl_sync(0xFFFFFFFFu, q.c0, l);
            it.q.n = __shfl_sync(0xFFFFFFFFu, q.n, l);
            it.q.total = __shfl_sync(0xFFFFFFFFu, q.total, l);
            return it;
        }
        if (in && it.seq < 0) {   // the flagging caller looks at every sequence
            const int l = __ffs(in) - 1;
            it.seq = s0 + l;
            it.tile = item - base - __shfl_sync(0xFFFFFFFFu, x - cnt, l);
            it.q.c0 = __shfl_sync(0xFFFFFFFFu, q.c0, l);
            it.q.n = __shfl_sync(0xFFFFFFFFu, q.n, l);
            it.q.total = __shfl_sync(0xFFFFFFFFu, q.total, l);
        }
        base += __shfl_sync(0xFFFFFFFFu, x, 31);
    }
    return it;
}

// Keys the sequence can attend: its cached tokens within the caller's bound and its page table.
__device__ __forceinline__ int key_limit(const Params &p, const Seq &q) {
    int64_t t = q.total;
    if (t > p.n_kv_max) t = p.n_kv_max;
    if (t > p.table_stride * p.page) t = p.table_stride * p.page;
    if (t > 0x7FFFFFFF - 1023) t = 0x7FFFFFFF - 1023;   // a tile's end is an int
    return (int)(t > 0 ? t : 0);
}

// Cell of position t of sequence s, or -1 (flagged) when the page table's entry is no page.
__device__ __forceinline__ int64_t cell_of(const Params &p, int s, int t) {
    const int pg = p.page_div.div(t);
    const int e = __ldg(p.table + (int64_t)s * p.table_stride + pg);
    if (e < 0 || e >= p.n_pages) {
        set_status(p.status, SFA_DEV_BAD_CELL);
        return -1;
    }
    return (int64_t)e * p.page + (t - pg * p.page);
}

// A piece of work of the narrow heads' kernel: keys k0 .. k1 - 1 of the list of one row tile (nq
// queries from q0 on, the first at position pos0) and KV head.  n_tiles 0 with whole: a list of no key.
struct Piece {
    int seq, c0, q0, nq, pos0, g, len, k0, k1;
    int r0;      // queries of the row tile before q0: 0, but for a piece that is done again
    int part;    // where its partial results go, in row tiles; -1: the piece is the whole list
    int state;   // kRun, kSkip (nothing to do), kEnd (no further piece)
    int head, ends;   // of a slot's share: the list began in an earlier slot; it ends in this one
};
enum { kRun, kSkip, kEnd };

__device__ __forceinline__ void piece_rows(const Params &p, const Seq &q, int tile, Piece &w) {
    w.c0 = q.c0;
    w.r0 = 0;
    w.q0 = tile * p.item_q;
    w.nq = min(p.item_q, min(q.n, p.n_new_max) - w.q0);
    w.pos0 = q.total - q.n + w.q0;
    w.len = max(0, min(key_limit(p, q), w.pos0 + w.nq));
}
// One piece a CTA: `split` of item and KV head g; by a whole warp.
__device__ __forceinline__ Piece piece_of(const Params &p, int item, int g, int split) {
    Piece w;
    w.state = kEnd;
    const Item it = find_item(p, item, g == 0 && split == 0);
    if (it.seq < 0) return w;
    w.seq = it.seq;
    w.g = g;
    piece_rows(p, it.q, it.tile, w);
    w.k0 = (int)min((int64_t)w.len, (int64_t)split * p.split_keys);
    w.k1 = (int)min((int64_t)w.len, (int64_t)w.k0 + p.split_keys);
    w.part = w.len <= p.split_keys ? -1 : ((item * p.h_kv + g) * p.n_split + split);
    w.state = split > 0 && w.k0 >= w.k1 ? kEnd : kRun;
    return w;
}

// The work dealt out evenly.  Every row tile and KV head weighs as many keys as its list has, and
// kPieceKeys more for the start and end of a piece (about 6 us; without them slots with ten short
// lists took 156 us where the others took 100); in a line, sequence by sequence, KV head by KV head,
// row tile by row tile, the weights sum up to W, and slot c takes the keys from c W / slots to
// (c + 1) W / slots: whole lists, and at each end perhaps a part of one, cut on tile borders (a
// border among the added keys leaves the list whole before it).  A slot then has at most two partial
// results, one that starts inside a list (2 c) and one that ends inside one (2 c + 1), however long
// the lists are.
// For the merge a slot says in slot_info of its partial results, [c][0] = (written, the list ends
// here) for the one that starts inside a list, [c][1] = (written, first query, queries, KV head) for
// the one that is a list's start: the pieces of that list are it and the following slots' [0], up to
// the one where the list ends.
// The weights of a sequence's row tiles grow by item_q from one to the next, so their sums have a
// closed form and a place in the line is found without a pass over the tiles.
constexpr int kPieceKeys = 448;
struct Unit {
    int seq, tile, g;
    int64_t w, u0;        // its weight, its place in the line
    Seq q;
};
// One sequence's part of the line, a lane's of a group of 32.
struct SeqWork {
    Seq q;
    int n, tiles;
    int64_t a, head, upto;   // head: the weights of one KV head; upto: all of the group's, to this lane
};
struct Share {
    int64_t per, rem;        // W / slots and what is left over
    int64_t at, end;         // of this slot: what is left of its part of the line
    int64_t before;          // the weights of the sequences before s0, the group that `at` is in
    int s0;
    SeqWork group;           // of s0
};
// Where slot c begins: the first rem slots have a key more than the others.
__device__ __forceinline__ int64_t share_border(const Share &h, int c) {
    return h.per * c + min((int64_t)c, h.rem);
}
// Sum of the weights of the first j row tiles of a sequence with n new tokens behind a cached ones
// (j at most their number; the last one may be short).
__device__ __forceinline__ int64_t tile_weights(const Params &p, int64_t a, int n, int tiles, int64_t j) {
    const int64_t full = j < tiles ? j : tiles - 1;
    return full * a + p.item_q * (full * (full + 1) / 2) + (j < tiles ? 0 : a + n) + j * kPieceKeys;
}
// By one whole warp, as all of the following.
__device__ __forceinline__ SeqWork seq_work(const Params &p, int s0, bool flag) {
    const int lane = threadIdx.x & 31, s = s0 + lane;
    SeqWork v;
    v.q = Seq{0, 0, 0};
    if (s < p.n_seq) v.q = load_seq(p, s, flag);
    v.n = min(v.q.n, p.n_new_max);
    v.tiles = n_items(p, v.q.n);
    v.a = max(v.q.total - v.q.n, 0);
    v.head = v.n > 0 ? tile_weights(p, v.a, v.n, v.tiles, v.tiles) : 0;
    v.upto = v.head * p.h_kv;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xFFFFFFFFu, v.upto, o);
        if (lane >= o) v.upto += y;
    }
    return v;
}
__device__ __forceinline__ Share share_of(const Params &p, int c, bool flag) {
    const int lane = threadIdx.x & 31;
    Share h;
    h.group = seq_work(p, 0, flag);
    int64_t W = lane == 31 ? h.group.upto : 0;
    for (int s0 = 32; s0 < p.n_seq; s0 += 128) {   // four sequences a lane: their loads at once
        int c0[4], c1[4], total[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int s = s0 + 32 * k + lane;
            c0[k] = c1[k] = total[k] = 0;
            if (s < p.n_seq) {
                c0[k] = p.cu[s];
                c1[k] = p.cu[s + 1];
                total[k] = p.total[s];
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const Seq q = make_seq(p, c0[k], c1[k], total[k], flag);
            const int n = min(q.n, p.n_new_max), tiles = n_items(p, n);
            if (n > 0) W += tile_weights(p, max(q.total - q.n, 0), n, tiles, tiles) * p.h_kv;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) W += __shfl_xor_sync(0xFFFFFFFFu, W, o);
    h.per = W / p.slots;
    h.rem = W - h.per * p.slots;
    h.at = share_border(h, c);
    h.end = share_border(h, c + 1);
    h.before = 0;
    h.s0 = 0;
    return h;
}
// The unit at place x < W of the line, no place before an earlier call's.
__device__ __forceinline__ Unit share_unit(const Params &p, Share &h, int64_t x) {
    unsigned in = __ballot_sync(0xFFFFFFFFu, x < h.before + h.group.upto);
    while (!in && h.s0 + 32 < p.n_seq) {
        h.before += __shfl_sync(0xFFFFFFFFu, h.group.upto, 31);
        h.s0 += 32;
        h.group = seq_work(p, h.s0, false);
        in = __ballot_sync(0xFFFFFFFFu, x < h.before + h.group.upto);
    }
    const SeqWork &v = h.group;
    const int l = in ? __ffs(in) - 1 : 31;
    Unit u;
    u.seq = h.s0 + l;
    u.q.c0 = __shfl_sync(0xFFFFFFFFu, v.q.c0, l);
    u.q.n = __shfl_sync(0xFFFFFFFFu, v.q.n, l);
    u.q.total = __shfl_sync(0xFFFFFFFFu, v.q.total, l);
    const int64_t head = __shfl_sync(0xFFFFFFFFu, v.head, l), a = __shfl_sync(0xFFFFFFFFu, v.a, l);
    const int n = __shfl_sync(0xFFFFFFFFu, v.n, l), tiles = __shfl_sync(0xFFFFFFFFu, v.tiles, l);
    int64_t r = x - h.before - __shfl_sync(0xFFFFFFFFu, v.upto - v.head * p.h_kv, l);
    u.g = 0;
    if (p.h_kv > 1) {
        u.g = (int)(r / head);
        r -= u.g * head;
    }
    int lo = 0, hi = tiles - 1;   // the last tile whose weights begin at or before r
    while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (tile_weights(p, a, n, tiles, m) <= r) lo = m;
        else hi = m - 1;
    }
    u.tile = lo;
    u.w = a + min((int64_t)(lo + 1) * p.item_q, (int64_t)n) + kPieceKeys;
    u.u0 = x - r + tile_weights(p, a, n, tiles, lo);
    return u;
}
// Keys [k0, k1) of a unit with a list of len that slot c has; by its borders alone, so that
// neighbours and the merge agree.
__device__ __forceinline__ void share_keys(const Share &h, int c, const Unit &u, int len, int &k0, int &k1) {
    const int64_t a = share_border(h, c) - u.u0, b = share_border(h, c + 1) - u.u0;
    k0 = a <= 0 ? 0 : (int)min((a + 64) & ~(int64_t)127, (int64_t)len);
    k1 = b >= u.w ? len : (int)min((b + 64) & ~(int64_t)127, (int64_t)len);
}
// Slot c's next piece.
__device__ __forceinline__ Piece share_next(const Params &p, int c, Share &h) {
    Piece w;
    w.state = kEnd;
    if (h.at >= h.end) return w;
    const Unit u = share_unit(p, h, h.at);
    w.seq = u.seq;
    w.g = u.g;
    piece_rows(p, u.q, u.tile, w);
    share_keys(h, c, u, w.len, w.k0, w.k1);
    const bool first = u.u0 >= share_border(h, c);   // the list's start is this slot's
    const bool all = w.k0 == 0 && w.k1 == w.len;
    w.part = all ? -1 : 2 * c + (w.k0 > 0 ? 0 : 1);
    w.state = w.k0 < w.k1 || (all && first) ? kRun : kSkip;
    w.head = !first;
    w.ends = u.u0 + u.w <= share_border(h, c + 1);
    // lengths that change while the call runs can put the list's end behind this place: the slot then ends
    h.at = u.u0 + u.w > h.at ? min(h.end, u.u0 + u.w) : h.end;
    return w;
}
// Slot c's next piece (first: its first one).  Not inlined: the kernel's other warps keep their registers.
static __device__ __noinline__ Piece share_piece(const Params &p, int c, Share &h, bool first) {
    const bool lead = (threadIdx.x & 31) == 0;
    if (first) {
        h = share_of(p, c, c == 0);
        if (lead) {
            p.slot_info[2 * c] = make_int4(0, 1, 0, 0);
            p.slot_info[2 * c + 1] = make_int4(0, 0, 0, 0);
        }
    }
    const Piece w = share_next(p, c, h);
    if (w.state != kEnd && lead) {
        if (w.head) p.slot_info[2 * c] = make_int4(w.state == kRun && w.part == 2 * c, w.ends, 0, 0);
        if (w.state == kRun && w.part == 2 * c + 1)
            p.slot_info[2 * c + 1] = make_int4(1, w.c0 + w.q0, w.nq, w.g);
    }
    return w;
}

// Values that are not finite.  A product gives a key that a query does not attend a weight of zero, and
// zero times such a value is NaN: a NaN in a chunk's token would reach the queries before it that share
// its row tile.  The kernels on tcgen05 look at their results: where one is NaN, they look for such
// values among the keys that some query of the tile does not attend, and do the queries up to the
// first of them (a group; then those up to the next one) again, over the keys before it.
//
// The first key in [a, b) of sequence seq whose values of KV head g are not all finite, b if there is
// none; by one whole warp.  Positions without a cell read as zeros.
template <int DV>
__device__ __forceinline__ int first_odd(const Params &p, const void *rows, int stride, int seq, int g, int a, int b) {
    for (int t0 = a; t0 < b; t0 += 32) {
        const int t = t0 + (threadIdx.x & 31);
        bool odd = false;
        if (t < b) {
            const int64_t cell = cell_of(p, seq, t);
            if (cell >= 0) {
                const uint4 *v = reinterpret_cast<const uint4 *>(reinterpret_cast<const __nv_bfloat16 *>(rows) +
                                                                 (cell * p.h_kv + g) * stride);
                auto bad = [](uint32_t x) { return (x & 0x7F80u) == 0x7F80u || (x & 0x7F800000u) == 0x7F800000u; };
                for (int i = 0; i < DV / 8; ++i) {
                    const uint4 x = v[i];
                    odd = odd || bad(x.x) || bad(x.y) || bad(x.z) || bad(x.w);
                }
            }
        }
        const unsigned any = __ballot_sync(0xFFFFFFFFu, odd);
        if (any) return t0 + __ffs(any) - 1;
    }
    return b;
}
// The next group of piece w, whose queries before `from` are done: kEnd if its results are right.
template <int DV>
__device__ __forceinline__ Piece odd_group(const Params &p, const Piece &w, int from, int stride) {
    Piece f = w;
    const int a = max(max(w.k0, 0), w.pos0 + from + 1), t = first_odd<DV>(p, p.V ? p.V : p.K, stride, w.seq, w.g, a, w.k1);
    f.r0 = from;
    f.q0 += from;
    f.pos0 += from;
    f.nq = t - f.pos0;
    f.k1 = t;
    f.state = t >= w.k1 ? kEnd : w.part < 0 || f.k0 < f.k1 ? kRun : kSkip;   // a part without a key: nothing is read of it
    return f;
}

// The kernel for 512 value dims on tcgen05 CTA pairs (chunk_wide.cu): queries of one CTA's 64
// rows, and the launch (p.item_q = twice that, p.item_rows = 128).
inline int wide_qpc(int G) { return 64 / G; }
int launch_wide(const Params &p, int dkq, int64_t n_cells, cudaStream_t st);
// The kernel for 128- and 64-wide heads on tcgen05 (chunk_narrow.cu): queries of one 128-row tile,
// and the launch (p.item_q = twice that, p.item_rows = 256).
inline int narrow_qpt(int G) { return 128 / G; }
int launch_narrow(const Params &p, int d, int64_t n_cells, cudaStream_t st);

}  // namespace chunk
}  // namespace sfa
