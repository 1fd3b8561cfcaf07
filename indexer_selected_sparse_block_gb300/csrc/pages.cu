// pages.cu -- a paged cache's bookkeeping on the device: page tables and slot maps from the
// sequences' lengths (sfa_build_page_maps), and the new tokens' rows written into their cells
// (sfa_write_cells).
#include "sfa_common.cuh"

namespace sfa {
namespace {

// ------------------------------------------------------------------------ page tables, slots
constexpr int kMapThreads = 256;
constexpr int64_t kMapFourFrom = 1 << 18;
constexpr int kMapMaxSeq = 16384;   // offsets and page bases of every sequence fit shared memory

struct MapParams {
    const int32_t *len_old, *len_new, *free_pages, *free_head;
    int32_t *table, *cu, *total, *q_seq, *q_pos, *slot, *cell_of, *head_out, *status;
    int64_t n_free, table_stride, n_tok_cap, n_pos_cap;
    int64_t table_pos;   // positions a table's row holds, below 2^31
    FastDiv page_div;
    int n_seq, page, n_pages;
    int vec;             // 16-byte stores of slot, q_seq and q_pos
};

// The lengths a sequence counts with: negative ones as 0.
__device__ __forceinline__ void map_lengths(const MapParams &p, int s, int64_t &a, int64_t &n,
                                            bool &bad) {
    a = p.len_old[s];
    n = p.len_new[s];
    bad = a < 0 || n < 0;
    a = a < 0 ? 0 : a;
    n = n < 0 ? 0 : n;
}

// Pages of the first t positions (t < 2^31).
__device__ __forceinline__ int map_pages(const MapParams &p, int64_t t) {
    return t > 0 ? p.page_div.div((int)t - 1) + 1 : 0;
}
// Pages sequence s takes for n new tokens behind a cached ones: those of its table's row only.
__device__ __forceinline__ int64_t map_taken(const MapParams &p, int64_t a, int64_t n) {
    if (a >= p.table_pos) return 0;
    const int64_t e = a + n < p.table_pos ? a + n : p.table_pos;
    return map_pages(p, e) - map_pages(p, a);
}

// cu[s] = sum of the new lengths before s and base[s] = pages taken before s: exclusive prefix
// sums over the sequences, which every CTA makes for itself in shared memory (8 bytes read per
// sequence, from L2; no CTA waits for another).  Then a thread for four tokens: their sequence
// by bisection in cu, their page from the table (the partly filled last page) or from the free
// list, their cells; the first token of a page that is taken also writes the table's entry.
// Integer sums in a fixed order: the maps are the same on every run.
// A decode step is one CTA and latency (2.8 us); whole prompts are 16 bytes of stores per token:
// 4.2 M tokens in 44 us with one token a thread and 64-bit divisions, 18 us (3.8 TB/s of stores) with
// four a thread, 16-byte stores and one 32-bit division (a product) for the four.  (Eight a thread:
// 25 us, a warp's stores no longer whole lines; CTAs of 512 threads and stores that stay in L2: 19.3.)
template <int N>
__global__ void __launch_bounds__(kMapThreads, 6) page_maps_kernel(const MapParams p) {
    extern __shared__ int32_t s_map[];
    int32_t *s_cu = s_map;                    // [n_seq + 1], clipped to n_tok_cap
    int32_t *s_base = s_map + p.n_seq + 1;    // [n_seq]
    __shared__ int64_t s_warp[2][kMapThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    const int per = (p.n_seq + kMapThreads - 1) / kMapThreads;
    const int s0 = min(tid * per, p.n_seq), s1 = min(s0 + per, p.n_seq);
    int64_t tok = 0;
    int32_t flags = 0;
    for (int s = s0; s < s1; ++s) {
        int64_t a, n;
        bool bad;
        map_lengths(p, s, a, n, bad);
        if (bad || a + n > p.table_pos) flags |= SFA_DEV_BAD_LENGTH;
        tok += n;
    }
    // block-wide exclusive sum of v
    auto scan = [&](int64_t v, int which) -> int64_t {
        int64_t x = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) s_warp[which][warp] = x;
        __syncthreads();
        int64_t before = 0;
        for (int w = 0; w < warp; ++w) before += s_warp[which][w];
        return before + x - v;
    };
    int64_t cu = scan(tok, 0);
    int64_t pages = 0;
    {   // tokens past the rows given are dropped; pages are counted for the kept ones
        int64_t c = cu;
        for (int s = s0; s < s1; ++s) {
            int64_t a, n;
            bool bad;
            map_lengths(p, s, a, n, bad);
            const int64_t e = c + n;
            if (e > p.n_tok_cap) flags |= SFA_DEV_BAD_LENGTH;
            const int64_t c0 = c < p.n_tok_cap ? c : p.n_tok_cap, c1 = e < p.n_tok_cap ? e : p.n_tok_cap;
            pages += map_taken(p, a, c1 - c0);
            c = e;
        }
    }
    int64_t base = scan(pages, 1);
    const int64_t head0 = *p.free_head, head = head0 < 0 ? 0 : head0;
    const bool lead = blockIdx.x == 0;
    for (int s = s0; s < s1; ++s) {
        int64_t a, n;
        bool bad;
        map_lengths(p, s, a, n, bad);
        const int64_t c0 = cu < p.n_tok_cap ? cu : p.n_tok_cap;
        const int64_t c1 = cu + n < p.n_tok_cap ? cu + n : p.n_tok_cap;
        s_cu[s] = (int32_t)c0;
        // past the free list's end every base is as good as its end
        s_base[s] = (int32_t)(base + head < p.n_free ? base + head : p.n_free);
        base += map_taken(p, a, c1 - c0);
        if (s == p.n_seq - 1) {
            s_cu[p.n_seq] = (int32_t)c1;
            if (lead) {
                p.cu[p.n_seq] = (int32_t)c1;
                *p.head_out = (int32_t)(base + head < p.n_free ? base + head : p.n_free);
                if (base + head > p.n_free) flags |= SFA_DEV_NO_PAGES;
            }
        }
        if (lead) {
            p.cu[s] = (int32_t)c0;
            const int64_t t = a + (c1 - c0);
            p.total[s] = (int32_t)(t < 0x7FFFFFFF ? t : 0x7FFFFFFF);
        }
        cu += n;
    }
    if (p.n_seq == 0 && lead && tid == 0) {
        p.cu[0] = 0;
        *p.head_out = (int32_t)(head < p.n_free ? head : p.n_free);
    }
    if (p.n_seq == 0 && tid == 0) s_cu[0] = 0;
    if (lead && flags) set_status(p.status, flags);
    __syncthreads();
    const int64_t live = s_cu[p.n_seq];
    flags = 0;
    int s = -1, pg = -1;                // the sequence and page of the token before
    int64_t a = 0, s_end = 0;           // the sequence's cached tokens, the end of its rows
    int32_t page = -1;
    int old_pages = 0;
    const int64_t groups = (p.n_tok_cap + N - 1) / N;
    for (int64_t q = (int64_t)blockIdx.x * kMapThreads + tid; q < groups;
         q += (int64_t)gridDim.x * kMapThreads) {
        int cells[N], seqs[N], poss[N];
        int off = 0;
        s_end = 0;                      // found anew for the group's first token
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int64_t i = N * q + k;
            if (i >= live) {
                cells[k] = seqs[k] = poss[k] = -1;
                continue;
            }
            int64_t pos;
            bool fresh_page;
            if (i >= s_end) {           // another sequence: the last s with cu[s] <= i
                int lo = 0, hi = p.n_seq - 1;
                while (lo < hi) {
                    const int m = (lo + hi + 1) >> 1;
                    if (s_cu[m] <= i) lo = m;
                    else hi = m - 1;
                }
                s = lo;
                s_end = s_cu[s + 1];
                a = max(p.len_old[s], 0);
                old_pages = a < p.table_pos ? map_pages(p, a) : 0;
                pos = a + (i - s_cu[s]);
                if (pos < p.table_pos) {
                    pg = p.page_div.div((int)pos);
                    off = (int)pos - pg * p.page;
                }
                fresh_page = true;
            } else {
                pos = a + (i - s_cu[s]);
                fresh_page = ++off == p.page;
                if (fresh_page) {
                    off = 0;
                    ++pg;
                }
            }
            int32_t cell = -1;
            if (pos < p.table_pos) {
                if (fresh_page) {
                    int32_t *entry = p.table + (int64_t)s * p.table_stride + pg;
                    const bool taken = pg >= old_pages;
                    if (taken) {
                        const int64_t f = (int64_t)s_base[s] + (pg - old_pages);
                        page = f < p.n_free ? p.free_pages[f] : -1;
                    } else {
                        page = *entry;
                    }
                    if (page < 0 || page >= p.n_pages) {
                        flags |= taken && page < 0 ? SFA_DEV_NO_PAGES : SFA_DEV_BAD_CELL;
                        page = -1;
                    }
                    if (taken && off == 0) *entry = page;
                }
                if (page >= 0) cell = page * p.page + off;
            }
            cells[k] = cell;
            seqs[k] = s;
            poss[k] = (int32_t)(pos < 0x7FFFFFFF ? pos : 0x7FFFFFFF);
        }
        auto vec = [](const int *v) { return make_int4(v[0], v[1 % N], v[2 % N], v[3 % N]); };
        if (N == 4 && p.vec && 4 * q + 4 <= p.n_tok_cap) {   // slot is read next: it may stay in L2
            reinterpret_cast<int4 *>(p.slot)[q] = vec(cells);
            __stcs(reinterpret_cast<int4 *>(p.q_seq) + q, vec(seqs));
            __stcs(reinterpret_cast<int4 *>(p.q_pos) + q, vec(poss));
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k)
                if (N * q + k < p.n_tok_cap) {
                    p.slot[N * q + k] = cells[k];
                    p.q_seq[N * q + k] = seqs[k];
                    p.q_pos[N * q + k] = poss[k];
                }
        }
        if (p.cell_of) {
            int32_t *row = p.cell_of + (int64_t)seqs[0] * p.n_pos_cap + poss[0];
            if (N == 4 && seqs[0] >= 0 && seqs[N - 1] == seqs[0] && (int64_t)poss[0] + 4 <= p.n_pos_cap &&
                (reinterpret_cast<uintptr_t>(row) & 15u) == 0) {
                __stcs(reinterpret_cast<int4 *>(row), vec(cells));
            } else {
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    if (seqs[k] < 0) continue;
                    if (poss[k] < p.n_pos_cap) p.cell_of[(int64_t)seqs[k] * p.n_pos_cap + poss[k]] = cells[k];
                    else flags |= SFA_DEV_BAD_LENGTH;
                }
            }
        }
    }
    if (flags) set_status(p.status, flags);
}

// ------------------------------------------------------------------------------ cell writes
enum WriteKind { kCopy16, kCopy2, kRound16, kRound1, kQ8 };
struct CellWrites {
    sfa_cell_write w[SFA_MAX_CELL_WRITES];
    int kind[SFA_MAX_CELL_WRITES];
    int units[SFA_MAX_CELL_WRITES];      // pieces of a row: 16 bytes stored, one element, a q8_0 block
    FastDiv div[SFA_MAX_CELL_WRITES];    // by units
};

// The rows' pieces in one line, four a thread in flight: their slots, their loads, their stores.
// A row's neighbours in the line are its neighbours in memory on both sides.  With a warp to a row
// a row of 72 pieces left a third of the lanes idle (65536 rows of 1408 bytes: 39 us; 29 so,
// 6.3 TB/s).
template <int KIND>
__device__ __forceinline__ void write_pieces(const sfa_cell_write &w, int units, const FastDiv &div,
                                             const int32_t *__restrict__ slot, int64_t n_rows,
                                             int64_t n_cells, int32_t *status) {
    constexpr int U = 4, B = 256 * U;
    const int elems = w.n_inner * w.d;
    const int64_t total = n_rows * units;
    const int es = w.src_dtype == SFA_F32 ? 4 : 2;   // copies: of both sides
    for (int64_t b = (int64_t)blockIdx.x * B; b < total; b += (int64_t)gridDim.x * B) {
        const int64_t r0 = b / units;
        const int u0 = (int)(b - r0 * units) + threadIdx.x;
        const int n = (int)min((int64_t)B, total - b);
        int64_t row[U], cell[U];
        int piece[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int r = div.div(u0 + 256 * k);
            piece[k] = u0 + 256 * k - r * units;
            row[k] = r0 + r;
            cell[k] = (int)threadIdx.x + 256 * k < n ? slot[row[k]] : -1;
            if (cell[k] >= n_cells) {
                set_status(status, SFA_DEV_BAD_CELL);
                cell[k] = -1;
            }
        }
        if constexpr (KIND == kCopy16) {
            uint4 v[U];
#pragma unroll
            for (int k = 0; k < U; ++k)
                if (cell[k] >= 0)
                    v[k] = __ldcs(reinterpret_cast<const uint4 *>(
                        reinterpret_cast<const uint8_t *>(w.src) + row[k] * w.src_stride * es + 16 * piece[k]));
#pragma unroll
            for (int k = 0; k < U; ++k)
                if (cell[k] >= 0)
                    *reinterpret_cast<uint4 *>(reinterpret_cast<uint8_t *>(w.dst) + cell[k] * elems * es + 16 * piece[k]) = v[k];
        } else if constexpr (KIND == kRound16) {
            float4 v[U][2];
#pragma unroll
            for (int k = 0; k < U; ++k)
                if (cell[k] >= 0) {
                    const float4 *x = reinterpret_cast<const float4 *>(
                        reinterpret_cast<const float *>(w.src) + row[k] * w.src_stride + 8 * piece[k]);
                    v[k][0] = __ldcs(x);
                    v[k][1] = __ldcs(x + 1);
                }
#pragma unroll
            for (int k = 0; k < U; ++k)
                if (cell[k] >= 0)
                    *reinterpret_cast<uint4 *>(reinterpret_cast<__nv_bfloat16 *>(w.dst) + cell[k] * elems + 8 * piece[k]) =
                        make_uint4(pack_bf16(v[k][0].x, v[k][0].y), pack_bf16(v[k][0].z, v[k][0].w),
                                   pack_bf16(v[k][1].x, v[k][1].y), pack_bf16(v[k][1].z, v[k][1].w));
        } else {
#pragma unroll
            for (int k = 0; k < U; ++k) {
                if (cell[k] < 0) continue;
                if constexpr (KIND == kCopy2)
                    reinterpret_cast<uint16_t *>(w.dst)[cell[k] * units + piece[k]] =
                        reinterpret_cast<const uint16_t *>(w.src)[row[k] * w.src_stride * (es / 2) + piece[k]];
                else
                    reinterpret_cast<__nv_bfloat16 *>(w.dst)[cell[k] * elems + piece[k]] =
                        __float2bfloat16_rn(reinterpret_cast<const float *>(w.src)[row[k] * w.src_stride + piece[k]]);
            }
        }
    }
}

// fp32 rows for a bf16 cache are rounded to nearest, as every bf16 cache value here is; q8_0 rows
// follow the rule of sfa_quantize_kv_q8_0 (one warp per block of 32: binary32 scale and codes,
// the scale then rounded to binary16).
__global__ void __launch_bounds__(256)
    write_cells_kernel(const CellWrites cw, const int32_t *__restrict__ slot, int64_t n_rows,
                       int64_t n_cells, int32_t *status) {
    pdl_wait();
    const sfa_cell_write &w = cw.w[blockIdx.y];
    const int kind = cw.kind[blockIdx.y], units = cw.units[blockIdx.y];
    const FastDiv &div = cw.div[blockIdx.y];
    if (kind == kCopy16) return write_pieces<kCopy16>(w, units, div, slot, n_rows, n_cells, status);
    if (kind == kRound16) return write_pieces<kRound16>(w, units, div, slot, n_rows, n_cells, status);
    if (kind == kCopy2) return write_pieces<kCopy2>(w, units, div, slot, n_rows, n_cells, status);
    if (kind == kRound1) return write_pieces<kRound1>(w, units, div, slot, n_rows, n_cells, status);
    const int lane = threadIdx.x & 31, nb = w.d / 32, rb = q8_row_bytes(w.d);
    const int64_t total = n_rows * units, stride = (int64_t)gridDim.x * 8;
    for (int64_t u = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); u < total; u += stride) {
        const int64_t i = u / units;
        const int b = (int)(u - i * units);
        const int64_t c = slot[i];
        if (c < 0) continue;
        if (c >= n_cells) {
            if (lane == 0) set_status(status, SFA_DEV_BAD_CELL);
            continue;
        }
        const int h = b / nb, k = b - h * nb;
        const int64_t e = i * w.src_stride + (int64_t)b * 32 + lane;
        const float x = w.src_dtype == SFA_F32
                            ? reinterpret_cast<const float *>(w.src)[e]
                            : __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(w.src)[e]);
        uint8_t *y = reinterpret_cast<uint8_t *>(w.dst) + (c * w.n_inner + h) * rb;
        float amax = fabsf(x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
        const float delta = __fdiv_rn(amax, 127.f);
        const int q = delta == 0.f ? 0 : (int)roundf(__fdiv_rn(x, delta));
        y[k * 32 + lane] = (uint8_t)(int8_t)q;
        if (lane == 0) {
            const __half sc = __float2half_rn(delta);
            *reinterpret_cast<__half *>(y + w.d + 2 * k) = sc;
            if (__hisinf(sc)) set_status(status, SFA_DEV_FP16_RANGE);
        }
        const int used = w.d + w.d / 16;
        if (k == nb - 1 && lane < rb - used) y[used + lane] = 0;
    }
}

int write_elem_bytes(int dtype) { return dtype == SFA_F32 ? 4 : 2; }

}  // namespace
}  // namespace sfa

extern "C" int sfa_build_page_maps(const int32_t *len_old, const int32_t *len_new, int n_seq,
                                   int page_size, const int32_t *free_pages, int64_t n_free,
                                   const int32_t *free_head, int n_pages, int32_t *page_table,
                                   int64_t table_stride, int32_t *cu_new, int32_t *len_total,
                                   int32_t *q_seq, int32_t *q_pos, int32_t *slot,
                                   int64_t n_tok_cap, int32_t *cell_of, int64_t n_pos_cap,
                                   int32_t *free_head_out, int32_t *dev_status,
                                   sfa_stream_t stream) {
    using namespace sfa;
    if (n_seq < 0 || page_size < 1 || n_pages < 0 || n_free < 0 || n_free > 0x7FFFFFFF ||
        table_stride < 0 || n_tok_cap < 0 || n_tok_cap > 0x7FFFFFFF || n_pos_cap < 0)
        return SFA_ERR_INVALID_ARG;
    if (!cu_new || !free_head || !free_head_out || free_head == free_head_out)
        return SFA_ERR_INVALID_ARG;
    if (n_seq > 0 && (!len_old || !len_new || !len_total || len_total == len_old ||
                      len_total == len_new || !page_table))
        return SFA_ERR_INVALID_ARG;
    if (n_free > 0 && !free_pages) return SFA_ERR_INVALID_ARG;
    if (n_tok_cap > 0 && (!q_seq || !q_pos || !slot)) return SFA_ERR_INVALID_ARG;
    if ((int64_t)n_pages * page_size > 0x7FFFFFFF) return SFA_ERR_INVALID_ARG;
    // positions are 32-bit (both factors are below 2^31: no overflow of the product)
    if (table_stride > 0x7FFFFFFF || table_stride * page_size > 0x7FFFFFFF)
        return SFA_ERR_INVALID_ARG;
    if (n_seq > kMapMaxSeq) return SFA_ERR_UNSUPPORTED;
    MapParams p{};
    p.len_old = len_old;
    p.len_new = len_new;
    p.free_pages = free_pages;
    p.free_head = free_head;
    p.table = page_table;
    p.cu = cu_new;
    p.total = len_total;
    p.q_seq = q_seq;
    p.q_pos = q_pos;
    p.slot = slot;
    p.cell_of = cell_of;
    p.head_out = free_head_out;
    p.status = dev_status;
    p.n_free = n_free;
    p.table_stride = table_stride;
    p.n_tok_cap = n_tok_cap;
    p.n_pos_cap = n_pos_cap;
    p.table_pos = table_stride * page_size;
    p.page_div.set(page_size);
    p.n_seq = n_seq;
    p.page = page_size;
    p.n_pages = n_pages;
    p.vec = aligned16(slot) && aligned16(q_seq) && aligned16(q_pos);
    const size_t smem = (2 * (size_t)n_seq + 1) * sizeof(int32_t);
    // four tokens a thread once every thread of the device has one
    const bool four = n_tok_cap > (int64_t)kMapFourFrom;
    const int per_block = (four ? 4 : 1) * kMapThreads;
    int64_t blocks = (n_tok_cap + per_block - 1) / per_block;
    const int64_t most = 6 * (int64_t)device_sm_count();   // resident at once
    blocks = blocks < 1 ? 1 : blocks > most ? most : blocks;
    auto kernel = four ? page_maps_kernel<4> : page_maps_kernel<1>;
    if (smem > 48 * 1024 && !ensure_max_dynamic_smem(kernel)) return SFA_ERR_CUDA;
    if (launch_pdl(kernel, dim3((unsigned)blocks), dim3(kMapThreads), smem, (cudaStream_t)stream, p) !=
        cudaSuccess) {
        cudaGetLastError();
        return SFA_ERR_CUDA;
    }
    return SFA_OK;
}

extern "C" int sfa_write_cells(int n, const sfa_cell_write *writes, const int32_t *slot,
                               int64_t n_rows, int64_t n_cells, int32_t *dev_status,
                               sfa_stream_t stream) {
    using namespace sfa;
    if (n < 0 || n > SFA_MAX_CELL_WRITES || (n > 0 && !writes) || n_rows < 0 || n_cells < 0 ||
        n_cells > 0x7FFFFFFF)
        return SFA_ERR_INVALID_ARG;
    CellWrites cw{};
    int64_t blocks = 0;
    for (int k = 0; k < n; ++k) {
        const sfa_cell_write &w = writes[k];
        const bool q8 = w.dst_dtype == SFA_Q8_0;
        if ((w.src_dtype != SFA_BF16 && w.src_dtype != SFA_F32) ||
            (w.dst_dtype != SFA_BF16 && w.dst_dtype != SFA_F32 && !q8))
            return SFA_ERR_INVALID_ARG;
        if (w.n_inner < 1 || w.d < 1 || (int64_t)w.n_inner * w.d > (1 << 24))
            return SFA_ERR_INVALID_ARG;
        if (w.src_dtype == SFA_BF16 && w.dst_dtype == SFA_F32) return SFA_ERR_UNSUPPORTED;
        if (q8 && w.d != 64 && w.d != 128 && w.d != 512 && w.d != 576) return SFA_ERR_UNSUPPORTED;
        const int64_t elems = (int64_t)w.n_inner * w.d;
        const int ss = write_elem_bytes(w.src_dtype), ds = write_elem_bytes(w.dst_dtype);
        if (n_rows > 1 && w.src_stride < elems) return SFA_ERR_INVALID_ARG;
        if (n_rows > 0) {
            if (!w.src || !w.dst || !aligned16(w.dst) ||
                reinterpret_cast<uintptr_t>(w.src) % ss != 0)
                return SFA_ERR_INVALID_ARG;
        }
        cw.w[k] = w;
        // 16 bytes a store where every row of both sides starts on such a boundary
        const bool vec = aligned16(w.src) && (w.src_stride * ss) % 16 == 0 && (elems * ds) % 16 == 0;
        const bool copy = w.src_dtype == w.dst_dtype;
        cw.kind[k] = q8 ? kQ8 : copy ? (vec ? kCopy16 : kCopy2) : (vec ? kRound16 : kRound1);
        cw.units[k] = (int)(q8 ? elems / 32 : vec ? elems * ds / 16 : copy ? elems * ds / 2 : elems);
        cw.div[k].set(cw.units[k]);
        const int64_t work = (n_rows * cw.units[k] + (q8 ? 7 : 1023)) / (q8 ? 8 : 1024);
        if (work > blocks) blocks = work;
    }
    if (n == 0 || n_rows == 0) return SFA_OK;
    if (!slot) return SFA_ERR_INVALID_ARG;
    const int64_t most = 8 * (int64_t)device_sm_count();
    if (blocks > most) blocks = most;
    if (launch_pdl(write_cells_kernel, dim3((unsigned)blocks, (unsigned)n), dim3(256), 0,
                   (cudaStream_t)stream, cw, slot, n_rows, n_cells, dev_status) != cudaSuccess) {
        cudaGetLastError();
        return SFA_ERR_CUDA;
    }
    return SFA_OK;
}
