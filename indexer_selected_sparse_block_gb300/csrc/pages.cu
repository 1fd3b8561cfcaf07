// pages.cu -- a paged cache's bookkeeping on the device: page tables and slot maps from the
// sequences' lengths (sfa_build_page_maps), and the new tokens' rows written into their cells
// (sfa_write_cells).
#include "sfa_common.cuh"

namespace sfa {
namespace {

// ------------------------------------------------------------------------ page tables, slots
constexpr int kMapThreads = 512;
constexpr int kMapMaxSeq = 16384;   // offsets and page bases of every sequence fit shared memory

struct MapParams {
    const int32_t *len_old, *len_new, *free_pages, *free_head;
    int32_t *table, *cu, *total, *q_seq, *q_pos, *slot, *cell_of, *head_out, *status;
    int64_t n_free, table_stride, n_tok_cap, n_pos_cap;
    int n_seq, page, n_pages;
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

// Pages sequence s takes for n new tokens behind a cached ones: those of its table's row only.
__device__ __forceinline__ int64_t map_taken(const MapParams &p, int64_t a, int64_t n) {
    const int64_t p0 = (a + p.page - 1) / p.page;
    int64_t p1 = (a + n + p.page - 1) / p.page;
    p1 = p1 < p.table_stride ? p1 : p.table_stride;
    return p1 > p0 ? p1 - p0 : 0;
}

// cu[s] = sum of the new lengths before s and base[s] = pages taken before s: exclusive prefix
// sums over the sequences, which every CTA makes for itself in shared memory (8 bytes read per
// sequence, from L2; no CTA waits for another).  Then a thread per token: its sequence by
// bisection in cu, its page from the table (the partly filled last page) or from the free list,
// its cell; the first token of a page that is taken also writes the table's entry.  Integer
// sums in a fixed order: the maps are the same on every run.
// A decode step is one CTA and latency; a whole prompt is 16 bytes of stores per token.
__global__ void __launch_bounds__(kMapThreads) page_maps_kernel(const MapParams p) {
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
        if (bad || a + n > p.table_stride * p.page) flags |= SFA_DEV_BAD_LENGTH;
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
    for (int64_t i = (int64_t)blockIdx.x * kMapThreads + tid; i < p.n_tok_cap;
         i += (int64_t)gridDim.x * kMapThreads) {
        if (i >= live) {
            p.slot[i] = p.q_seq[i] = p.q_pos[i] = -1;
            continue;
        }
        int lo = 0, hi = p.n_seq - 1;   // the last s with cu[s] <= i
        while (lo < hi) {
            const int m = (lo + hi + 1) >> 1;
            if (s_cu[m] <= i) lo = m;
            else hi = m - 1;
        }
        const int s = lo;
        const int64_t a = max(p.len_old[s], 0);
        const int64_t pos = a + (i - s_cu[s]);
        const int64_t pg = pos / p.page, off = pos - pg * p.page;
        int32_t cell = -1;
        if (pg < p.table_stride) {
            const int64_t p0 = (a + p.page - 1) / p.page;
            int32_t *entry = p.table + (int64_t)s * p.table_stride + pg;
            int32_t page;
            if (pg >= p0) {
                const int64_t f = s_base[s] + (pg - p0);
                page = f < p.n_free ? p.free_pages[f] : -1;
                if (page < 0 || page >= p.n_pages) {
                    flags |= page < 0 ? SFA_DEV_NO_PAGES : SFA_DEV_BAD_CELL;
                    page = -1;
                }
                if (off == 0) *entry = page;
            } else {
                page = *entry;
                if (page < 0 || page >= p.n_pages) {
                    flags |= SFA_DEV_BAD_CELL;
                    page = -1;
                }
            }
            if (page >= 0) cell = (int32_t)((int64_t)page * p.page + off);
        }
        p.q_seq[i] = s;
        p.q_pos[i] = (int32_t)(pos < 0x7FFFFFFF ? pos : 0x7FFFFFFF);
        p.slot[i] = cell;
        if (p.cell_of) {
            if (pos < p.n_pos_cap) p.cell_of[(int64_t)s * p.n_pos_cap + pos] = cell;
            else flags |= SFA_DEV_BAD_LENGTH;
        }
    }
    if (flags) set_status(p.status, flags);
}

// ------------------------------------------------------------------------------ cell writes
struct CellWrites {
    sfa_cell_write w[SFA_MAX_CELL_WRITES];
    int vec[SFA_MAX_CELL_WRITES];   // 16-byte accesses on both sides
};

// One warp per (row, cache): the row's slot once, then the row.  Copies move 16 bytes a lane;
// fp32 rows for a bf16 cache are rounded to nearest, as every bf16 cache value here is; q8_0
// rows follow the rule of sfa_quantize_kv_q8_0 (one warp per block of 32: binary32 scale and
// codes, the scale then rounded to binary16).
__global__ void __launch_bounds__(256)
    write_cells_kernel(const CellWrites cw, const int32_t *__restrict__ slot, int64_t n_rows,
                       int64_t n_cells, int32_t *status) {
    pdl_wait();
    const sfa_cell_write &w = cw.w[blockIdx.y];
    const int vec = cw.vec[blockIdx.y];
    const int lane = threadIdx.x & 31;
    const int64_t stride = (int64_t)gridDim.x * 8;
    const int elems = w.n_inner * w.d;
    for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < n_rows; i += stride) {
        const int64_t c = slot[i];
        if (c < 0) continue;
        if (c >= n_cells) {
            if (lane == 0) set_status(status, SFA_DEV_BAD_CELL);
            continue;
        }
        if (w.dst_dtype == SFA_Q8_0) {
            const int nb = w.d / 32, rb = q8_row_bytes(w.d);
            for (int b = 0; b < w.n_inner * nb; ++b) {
                const int h = b / nb, k = b - h * nb;
                const int64_t e = i * w.src_stride + (int64_t)b * 32 + lane;
                const float x = w.src_dtype == SFA_F32
                                    ? reinterpret_cast<const float *>(w.src)[e]
                                    : __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(w.src)[e]);
                uint8_t *y = reinterpret_cast<uint8_t *>(w.dst) + (c * w.n_inner + h) * rb;
                float amax = fabsf(x);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
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
        } else if (w.src_dtype == w.dst_dtype) {
            const int es = w.src_dtype == SFA_F32 ? 4 : 2;
            const uint8_t *x = reinterpret_cast<const uint8_t *>(w.src) + i * w.src_stride * es;
            uint8_t *y = reinterpret_cast<uint8_t *>(w.dst) + c * elems * es;
            if (vec) {
                for (int e = lane; e < elems * es / 16; e += 32)
                    reinterpret_cast<uint4 *>(y)[e] = reinterpret_cast<const uint4 *>(x)[e];
            } else {
                for (int e = lane; e < elems * es / 2; e += 32)
                    reinterpret_cast<uint16_t *>(y)[e] = reinterpret_cast<const uint16_t *>(x)[e];
            }
        } else {   // fp32 -> bf16
            const float *x = reinterpret_cast<const float *>(w.src) + i * w.src_stride;
            __nv_bfloat16 *y = reinterpret_cast<__nv_bfloat16 *>(w.dst) + c * elems;
            if (vec) {
                for (int e = lane; e < elems / 4; e += 32) {
                    const float4 v = reinterpret_cast<const float4 *>(x)[e];
                    reinterpret_cast<uint2 *>(y)[e] =
                        make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
                }
            } else {
                for (int e = lane; e < elems; e += 32) y[e] = __float2bfloat16_rn(x[e]);
            }
        }
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
    MapParams p{len_old, len_new, free_pages, free_head, page_table, cu_new, len_total, q_seq,
                q_pos, slot, cell_of, free_head_out, dev_status, n_free, table_stride, n_tok_cap,
                n_pos_cap, n_seq, page_size, n_pages};
    const size_t smem = (2 * (size_t)n_seq + 1) * sizeof(int32_t);
    if (smem > 48 * 1024 && !ensure_max_dynamic_smem(page_maps_kernel)) return SFA_ERR_CUDA;
    int64_t blocks = (n_tok_cap + kMapThreads - 1) / kMapThreads;
    const int64_t most = 2 * (int64_t)device_sm_count();
    blocks = blocks < 1 ? 1 : blocks > most ? most : blocks;
    if (launch_pdl(page_maps_kernel, dim3((unsigned)blocks), dim3(kMapThreads), smem,
                   (cudaStream_t)stream, p) != cudaSuccess) {
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
        // 16 bytes a lane where every row of both sides starts on such a boundary
        // (the fp32 -> bf16 case stores 8 bytes a lane)
        cw.vec[k] = !q8 && aligned16(w.src) && (w.src_stride * ss) % 16 == 0 &&
                    (elems * ss) % 16 == 0 && (ss != ds ? (elems * ds) % 8 == 0 : (elems * ds) % 16 == 0);
    }
    if (n == 0 || n_rows == 0) return SFA_OK;
    if (!slot) return SFA_ERR_INVALID_ARG;
    int64_t blocks = (n_rows + 7) / 8;
    const int64_t most = 8 * (int64_t)device_sm_count();
    if (blocks > most) blocks = most;
    if (launch_pdl(write_cells_kernel, dim3((unsigned)blocks, (unsigned)n), dim3(256), 0,
                   (cudaStream_t)stream, cw, slot, n_rows, n_cells, dev_status) != cudaSuccess) {
        cudaGetLastError();
        return SFA_ERR_CUDA;
    }
    return SFA_OK;
}
