// chunk_common.cuh -- what the chunk attention kernels share (chunk.cu: the SIMT kernel, the
// merge of split lists, the launch plan and the C entry points).
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
    int32_t *status;
    int64_t table_stride;
    FastDiv page_div;
    int page, n_pages, n_seq, n_q, h_q, h_kv, G;
    int o_bf16;          // O is bf16 (else fp32)
    int items;           // row tiles of all sequences, at most
    int item_rows;       // rows of a tile
    int item_q;          // queries of a tile, 0: tiles cut the flattened rows anywhere
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
__device__ __forceinline__ Seq load_seq(const Params &p, int s, bool flag) {
    Seq q;
    q.c0 = p.cu[s];
    const int c1 = p.cu[s + 1];
    q.total = p.total[s];
    bool bad = q.c0 < 0 || c1 < q.c0 || c1 > p.n_q;
    q.n = bad ? 0 : c1 - q.c0;
    // the positions follow from the true length: a clipped chunk keeps its first queries
    if (q.n > p.n_new_max || q.total < q.n || q.total > p.n_kv_max ||
        (int64_t)q.total > p.table_stride * p.page)
        bad = true;
    if (bad && flag) set_status(p.status, SFA_DEV_BAD_QUERY);
    return q;
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
// By one whole warp: the row tiles of the sequences are counted 32 sequences at a time.
__device__ __forceinline__ Item find_item(const Params &p, int item, bool flag) {
    const int lane = threadIdx.x & 31;
    Item it;
    it.seq = -1;
    it.tile = 0;
    it.q = Seq{0, 0, 0};
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
