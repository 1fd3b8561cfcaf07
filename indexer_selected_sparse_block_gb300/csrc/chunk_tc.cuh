// chunk_tc.cuh -- what the chunk attention kernels on tcgen05 share: bounded waits, tensor memory
// access, and the loads of a tile's keys through the page table.
#pragma once

#include "chunk_common.cuh"

namespace sfa {
namespace chunk {

constexpr float kLazy = 8.f;   // base-2 growth of the maximum that O is not rescaled for

struct KeyMaps {
    CUtensorMap k[3], v[3];    // boxes of 1 << bxs, min(1 << bxs, 8) and 1 rows
};

// Waits for the phase of `parity`; the limit counts from the wait's own start.
__device__ __forceinline__ bool wait2(uint32_t bar, uint32_t parity) {
    uint64_t t0 = 0;
    for (uint32_t it = 0;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 63u) == 63u) {
            const uint64_t now = global_timer_ns();
            if (t0 == 0) t0 = now;
            else if (now - t0 > kWaitLimitNs) return false;
        }
    }
}
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity) {   // does not block
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
        "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Tiled loads into this CTA's shared memory, their bytes counted on a barrier of this CTA
// (tma_load) or, in a pair, of its first CTA (tma2_load).
__device__ __forceinline__ void tma2_load(uint32_t dst, const CUtensorMap *map, int x, int y, int z,
                                          uint32_t leader_bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(leader_bar)
        : "memory");
}
__device__ __forceinline__ void tma1_load(uint32_t dst, const CUtensorMap *map, int x, int y, int z,
                                          uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// ------------------------------------------------------------------------------- key rows
// The next kernel's CTAs (the merge) may take what SMs are free and wait there for this grid's end:
// asked for by each CTA when its last results are on their way out (1 us of a single token's 13; in
// the narrow heads' kernel, whose slots end at different times, it did not pay).
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A warp's 32 rows (its tensor memory lanes) x C value dims of O from column tcol, times each
// row's inv, to the output (whole) or the partial results: rows of DV values at `row`, dims d0 ...
// By way of shared memory (C * 128 bytes at `stage`): a row's values leave as one line.  (Each lane
// storing its own row's 16 bytes took 5.8 us for 64 rows of 512 fp32 values and 32 sectors a
// store.)  16-byte pieces are exchanged by the row's number, so neither side meets bank conflicts.
// Returns look and whether the lane's row has a NaN here (the maximum of three with NaN: two values an
// instruction, which costs nothing that can be measured).
template <int C, int DV>
__device__ __forceinline__ bool store_tile(const Params &p, uint32_t stage, uint32_t tcol, float inv,
                                           bool live, int64_t row, bool whole, int d0, bool look) {
    constexpr int PIECES = C / 4;   // of a row
    float most = -INFINITY;         // NaN once a value is
    const int lane = threadIdx.x & 31;
    const uint32_t mine = stage + lane * (C * 4);
#pragma unroll 1
    for (int x = 0; x < C / 32; ++x) {
        uint32_t r[32];
        tmem_ld32(tcol + 32 * x, r);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = __uint_as_float(r[4 * j + k]) * inv;
            asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(most) : "f"(v[0]), "f"(v[1]));
            asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(most) : "f"(v[2]), "f"(v[3]));
            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                             mine + (((x * 8 + j) ^ (lane & (PIECES - 1))) << 4)),
                         "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3])
                         : "memory");
        }
    }
    __syncwarp();
    constexpr int ROWS = 32 / PIECES;   // rows of one step: 1 for C = 128, 2 for C = 64
    const int sub = lane / PIECES, piece = lane & (PIECES - 1);
#pragma unroll 4
    for (int i = 0; i < 32; i += ROWS) {
        const int rr = i + sub;
        const bool on = __shfl_sync(0xFFFFFFFFu, (int)live, rr) != 0;
        const int64_t to = __shfl_sync(0xFFFFFFFFu, row, rr) * DV + d0 + 4 * piece;
        float4 v;
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                     : "r"(stage + rr * (C * 4) + ((piece ^ (rr & (PIECES - 1))) << 4)));
        if (!on) continue;
        if (!whole) *reinterpret_cast<float4 *>(p.part_o + to) = v;
        else if (p.o_bf16)
            *reinterpret_cast<uint2 *>(reinterpret_cast<__nv_bfloat16 *>(p.O) + to) =
                make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
        else
            *reinterpret_cast<float4 *>(reinterpret_cast<float *>(p.O) + to) = v;
    }
    return look && most != most;
}

// fp32 results: tensor memory sums kDrain tiles only, then the sums move on.  The tensor cores cut
// what they add to an accumulator towards zero: 16 additions a tile (hi and lo) leave the result
// 2.2e-7 short for each tile of its list (measured: 5.1e-5 at 30000 keys, and 7e-6 so, however long
// the list).  The sums wait where the result will be (O, or the partial results, fp32 both), in no
// order of their own: a full warp's lanes write whole lines, another warp's live lanes their own
// rows.  It costs about 8% of a long list: with 16 tiles 12%; leaving the addition to L2 (red) made
// wide heads 2% faster, narrow ones 1% slower.  bf16 results are rounded by 2^-8: not for them.
constexpr int kDrain = 24;

// A warp's 32 rows x C value dims of tensor memory from column tcol: added to keep times the sums at
// base (first: there are none), or (back) the sums times keep added to tensor memory.
template <int C, int DV>
__device__ __forceinline__ void drain_tile(float *base, uint32_t tcol, int64_t row, bool live, int d0,
                                           float keep, bool first, bool back) {
    constexpr int PIECES = C / 4, ROWS = 32 / PIECES;   // 16-byte pieces of a row, rows of a step
    const int lane = threadIdx.x & 31;
    const bool all = __all_sync(0xFFFFFFFFu, live);
#pragma unroll 1
    for (int x = 0; x < C / 32; ++x) {
        float4 *at[8], v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = 8 * x + j;
            const int64_t line = __shfl_sync(0xFFFFFFFFu, row, i * ROWS + lane / PIECES);
            at[j] = reinterpret_cast<float4 *>(base + d0 + (all ? line * DV + 4 * (lane % PIECES) : row * DV + 4 * i));
            v[j] = live && !first ? *at[j] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        uint32_t r[32];
        tmem_ld32(tcol + 32 * x, r);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j].x = fmaf(v[j].x, keep, __uint_as_float(r[4 * j]));
            v[j].y = fmaf(v[j].y, keep, __uint_as_float(r[4 * j + 1]));
            v[j].z = fmaf(v[j].z, keep, __uint_as_float(r[4 * j + 2]));
            v[j].w = fmaf(v[j].w, keep, __uint_as_float(r[4 * j + 3]));
        }
        if (back) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                r[4 * j] = __float_as_uint(v[j].x);
                r[4 * j + 1] = __float_as_uint(v[j].y);
                r[4 * j + 2] = __float_as_uint(v[j].z);
                r[4 * j + 3] = __float_as_uint(v[j].w);
            }
            tmem_st32(tcol + 32 * x, r);
        } else if (live) {
#pragma unroll
            for (int j = 0; j < 8; ++j) *at[j] = v[j];
        }
    }
    if (back) tmem_st_wait();
}
// The factor from sums scaled to 2^-m_sum to ones scaled to 2^-m (m_sum -inf: sums of nothing).
__device__ __forceinline__ float drain_keep(float m_sum, float m) {
    return m_sum == -INFINITY ? 1.f : ex2(m_sum - m);
}

template <int N>
struct Const {
    static constexpr int value = N;
};

// How the 64 keys of a half tile are loaded, a lane's share: 64 >> bs boxes of 1 << bs rows, this
// lane's being lane and lane + 32; where the list ends inside one (`edge`) that one row by row.
// The page table is read a tile ahead (`entry`: the raw entries), the cells follow from it.
struct HalfRows {
    int pos0, bs, edge;
    int entry[2], single;
    int row[2], srow;
};
// Keys pos0 .. pos0 + 63; the list ends before `end`.
__device__ __forceinline__ void read_entries(HalfRows &h, const Params &p, const int32_t *table, int pos0,
                                             int end, int bxs) {
    const int lane = threadIdx.x & 31;
    auto entry = [&](int pos) -> int { return pos < end ? __ldg(table + p.page_div.div(pos)) : -1; };
    h.pos0 = pos0;
    const bool whole = pos0 + 64 <= end;
    h.bs = whole ? bxs : min(bxs, 3);
    h.edge = -1;
    h.single = -1;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int box = lane + 32 * i;
        h.entry[i] = box < (64 >> h.bs) ? entry(pos0 + (box << h.bs)) : -1;
    }
    const int in = end - pos0;
    if (!whole && in > 0 && (in & ((1 << h.bs) - 1)) != 0) {
        h.edge = in >> h.bs;
        if (lane < (1 << h.bs)) h.single = entry(pos0 + (h.edge << h.bs) + lane);
    }
}
// Entries -> cells.  Keys past the list's end and those of pages that are none get n_cells: outside
// the tensor, read as zeros.
__device__ __forceinline__ void find_rows(HalfRows &h, const Params &p, int n_cells) {
    const int lane = threadIdx.x & 31;
    auto cell = [&](int e, int pos) -> int {
        return e < 0 || e >= p.n_pages ? n_cells : e * p.page + (pos - p.page_div.div(pos) * p.page);
    };
#pragma unroll
    for (int i = 0; i < 2; ++i) h.row[i] = cell(h.entry[i], h.pos0 + ((lane + 32 * i) << h.bs));
    h.srow = cell(h.single, h.pos0 + (h.edge << h.bs) + lane);
}
// SLABS slabs [64 keys][64 dims from x, x + 64, ..] of KV head g, STRIDE bytes apart; by a whole
// warp, one lane of which issues (elect.sync and coordinates that are the same in all lanes: a
// copy or product issued under a lane test costs the warp four times as long).  PAIR: the bytes
// are counted in the pair's first CTA.
template <int SLABS, int STRIDE, bool PAIR>
__device__ __forceinline__ void load_slabs(const HalfRows &h, uint32_t dst, const CUtensorMap *maps,
                                           int x, int g, int bxs, uint32_t bar) {
    auto copy = [&](const CUtensorMap *map, uint32_t at, int row) {
#pragma unroll
        for (int s = 0; s < SLABS; ++s) {
            if (PAIR) tma2_load(dst + s * STRIDE + at, map, x + 64 * s, g, row, bar);
            else tma1_load(dst + s * STRIDE + at, map, x + 64 * s, g, row, bar);
        }
    };
    // the whole half in N boxes: the rows to all lanes, then every copy at once
    auto whole = [&](auto n_boxes) {
        constexpr int N = decltype(n_boxes)::value;
        int r[N];
#pragma unroll
        for (int b = 0; b < N; ++b) r[b] = __shfl_sync(0xFFFFFFFFu, h.row[0], b);
        if (elect_one()) {
#pragma unroll
            for (int b = 0; b < N; ++b) copy(maps, (uint32_t)b * (64 / N) * 128, r[b]);
        }
    };
    if (h.bs == bxs && h.edge < 0) {
        if (bxs == 6) return whole(Const<1>{});
        if (bxs == 5) return whole(Const<2>{});
        if (bxs == 4) return whole(Const<4>{});
        if (bxs == 3) return whole(Const<8>{});
    }
    // the list's end, or pages whose size has no factor of 8
    const CUtensorMap *map = maps + (h.bs == bxs ? 0 : 1);
    const int n = 64 >> h.bs;
    for (int b = 0; b < n; ++b) {
        const int row = __shfl_sync(0xFFFFFFFFu, b < 32 ? h.row[0] : h.row[1], b & 31);
        if (b != h.edge && elect_one()) copy(map, (uint32_t)(b << h.bs) << 7, row);
    }
    if (h.edge >= 0)
        for (int i = 0; i < (1 << h.bs); ++i) {
            const int row = __shfl_sync(0xFFFFFFFFu, h.srow, i);
            if (elect_one()) copy(maps + 2, (uint32_t)((h.edge << h.bs) + i) << 7, row);
        }
}

// The same for a half tile within one page (pages of a multiple of 64 rows), by one thread: rows
// row0 .. row0 + v - 1 and zeros behind them.
template <int SLABS, int STRIDE, bool PAIR>
__device__ __forceinline__ void load_slabs_one(int row0, int v, uint32_t dst, const CUtensorMap *maps,
                                               int x, int g, int n_cells, uint32_t bar) {
    auto copy = [&](const CUtensorMap *map, uint32_t at, int row) {
#pragma unroll
        for (int s = 0; s < SLABS; ++s) {
            if (PAIR) tma2_load(dst + s * STRIDE + at, map, x + 64 * s, g, row, bar);
            else tma1_load(dst + s * STRIDE + at, map, x + 64 * s, g, row, bar);
        }
    };
    if (v == 64 || v == 0) {
        copy(maps, 0, v ? row0 : n_cells);
        return;
    }
#pragma unroll 1
    for (int b = 0; b < 8; ++b) {
        const int in = v - 8 * b;   // rows of this box in the list
        if (in >= 8 || in <= 0) {
            copy(maps + 1, b * 1024, in > 0 ? row0 + 8 * b : n_cells);
        } else {
#pragma unroll 1
            for (int i = 0; i < 8; ++i) copy(maps + 2, b * 1024 + i * 128, i < in ? row0 + 8 * b + i : n_cells);
        }
    }
}

// Tensor map of rows [n][heads][d] bf16 with boxes of `rows` x `heads_box` x 64 elements.
inline bool encode_rows(CUtensorMap *map, const void *base, int d, int heads, int64_t n, int heads_box, int rows) {
    EncodeTiledFn enc = encode_tiled();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)n};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)heads * d * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)heads_box, (cuuint32_t)rows}, es[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The boxes' rows (1 << *bxs = gcd(page, 64)) and the maps of K (and V, unless null).
inline bool encode_keys(KeyMaps *m, int *bxs, const Params &p, int dkq, int dv, int64_t n_cells) {
    int s = 0;
    while (s < 6 && p.page % (2 << s) == 0) ++s;
    *bxs = s;
    const int rows[3] = {1 << s, s < 3 ? 1 << s : 8, 1};
    for (int i = 0; i < 3; ++i) {
        if (!encode_rows(&m->k[i], p.K, dkq, p.h_kv, n_cells, 1, rows[i])) return false;
        if (p.V && !encode_rows(&m->v[i], p.V, dv, p.h_kv, n_cells, 1, rows[i])) return false;
    }
    return true;
}

}  // namespace chunk
}  // namespace sfa
