// chunk_narrow.cuh -- chunk attention with 128- and 64-wide heads (bf16) on tcgen05; TREE: of drafted
// trees.
//
// One CTA owns two row tiles of 128 rows (query, head) of one KV head and streams tiles of 128
// keys that both share.  Per row tile:
//   S[128 x 128] = Q K^T (operands in shared memory), the softmax, half a row a thread,
//   O[128 x D]  += P V, P in tensor memory where S was (the weights never pass through shared
//                  memory, whose bandwidth the products already use up), V from shared memory.
// While one row tile's softmax runs, the other's products do: P V (t) and S(t + 1) of a row tile
// are issued together, so a row tile's chain is S, softmax, P V and the two chains interleave.
// Tensor memory: two S / P tiles of 128 columns, two O tiles of D.
//
// For fp32 results the weights are two bf16 halves (hi + lo, 2^-16 relative) and P V runs twice; for
// bf16 results a weight is one bf16 value, off by 2^-8 of itself at most (see chunk_wide.cuh).  The running
// maximum moves only when a tile raises it by more than 2^8, and O in tensor memory is rescaled only then.
//
// The chains are what bounds it: in a ragged batch (24 sequences, 128 wide) the tensor pipe is busy
// 41% of the time, the schedulers 44%, the exponentials' unit 20%.  With one row a thread (four warps a
// row tile) the softmax took most of 3800 cycles a pair of tiles, the products 1024.  Measured: that
// batch 129 us with the merge (650 TFLOP/s), 1000 tokens behind 30000 (16 heads on 4, 128 wide, bf16
// results) 202 us (1240 TFLOP/s), 64 wide 168 us (740 TFLOP/s: twice the softmax a product); a pair of
// CTAs with one row tile each was slower (2300 cycles for 128 rows against 1700).
//
// Warps 0-7 and 8-15: softmax, correction and result of the two row tiles, the first four of each
// for keys 0-63 of a tile and the lower half of the value dims; warp 16: Q and K; warp 17: V;
// warp 18: products (one lane); warp 19: the next piece of work.  A CTA has one piece, or its even
// share of all (Share in chunk_common.cuh), piece after piece.  Pages as in chunk_wide.cuh.
#pragma once

#include "chunk_tc.cuh"

namespace sfa {
namespace chunk {
namespace {

constexpr int kT = 128;
constexpr int kThreads = 640;

template <int D, bool VK>
struct Narrow {
    static constexpr int kSlabs = D / 64;
    static constexpr int kTileBytes = kSlabs * 128 * 128;      // 128 rows x D bf16
    static constexpr int kKS = VK ? 5 : D == 128 ? 3 : 5;      // stages of K and of V
    static constexpr int kVS = VK ? 0 : D == 128 ? 2 : 5;
    static constexpr int kOffQ = 0;                            // two row tiles
    static constexpr int kOffK = 2 * kTileBytes;
    static constexpr int kOffV = kOffK + kKS * kTileBytes;
    static constexpr int kOffMax = kOffV + kVS * kTileBytes;   // float [2][256]
    static constexpr int kOffPiece = kOffMax + 2 * 256 * 4;    // Piece [3], 64 bytes each
    static constexpr int kOffBar = kOffPiece + 192;
    static constexpr int kBars = 2 + 2 * kKS + 2 * kVS + 2 + 2 + 2 + 1;
    static constexpr int kBytes = kOffBar + kBars * 8 + 32;
    static_assert(kBytes <= 227 * 1024, "one CTA per SM");
    static_assert(sizeof(Piece) <= 64, "fits its place");
    static_assert((kKS + kVS) * kTileBytes >= 8 * D * 128, "the result's way through shared memory");
};

struct NarrowMaps {
    CUtensorMap q;
    KeyMaps kv;
};

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// D[tmem] (+)= A[tmem: lane = row, two bf16 of K a column] * B[smem desc].
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// The words behind the barriers: tensor memory's address; a wait ran out; a result is not finite.
enum { kWordTmem, kWordAbort, kWordOdd };

// The barriers' phases: tiles so far, those of the second row tile, and the pieces of both; whether no
// wait ran out.
struct Phases {
    uint32_t u0, u1, np, np2;
    bool ok;
};

// One piece of work, by all warps but the last.
template <int D, bool VK, bool HL, bool TREE>
__device__ __forceinline__ void narrow_piece(const NarrowMaps &maps, const Params &p, int bxs, int qpt, int n_cells,
                                             uint8_t *smem, uint32_t tmem, const Piece &pc, Phases &ph) {
    using L = Narrow<D, VK>;
    constexpr int KS = L::kKS, VS = L::kVS;
    float *sMax = reinterpret_cast<float *>(smem + L::kOffMax);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kOffBar);
    volatile int *words = reinterpret_cast<volatile int *>(bars + L::kBars);
    const uint32_t bar0 = smem_u32(bars);
    const uint32_t b_q = bar0, b_kFull = b_q + 16, b_kEmpty = b_kFull + 8 * KS, b_vFull = b_kEmpty + 8 * KS,
                   b_vEmpty = b_vFull + 8 * VS, b_s = b_vEmpty + 8 * VS, b_p = b_s + 16, b_o = b_p + 16,
                   b_drain = b_o + 16;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sQ = smem_u32(smem + L::kOffQ), sK = smem_u32(smem + L::kOffK), sV = smem_u32(smem + L::kOffV);
    const int G = p.G;
    // a softmax thread's row: query ql of row tile w, head h; kg: its half of the keys and dims
    const int w = warp >> 3, kg = (warp >> 2) & 1, row = (warp & 3) * 32 + lane;
    const int ql = row / G, h = row - ql * G;
    uint32_t &u0 = ph.u0, &u1 = ph.u1, &np = ph.np, &np2 = ph.np2;
    bool &ok = ph.ok;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (ok && !wait2(bar, parity)) {
            ok = false;
            words[kWordAbort] = 1;
            set_status(p.status, SFA_DEV_TIMEOUT);
        }
    };
    const int g = pc.g, k0 = pc.k0, k1 = pc.k1, pos0 = pc.pos0, nq = pc.nq;
    const bool whole = pc.part < 0;
    const int n_tiles = pc.state == kSkip ? 0 : (k1 - k0 + kT - 1) / kT;
    const bool two = nq > qpt;                                // the second row tile has rows
    const bool live = pc.state == kRun && warp < 16 && ql < qpt && w * qpt + ql < nq;
    const int64_t orow = (int64_t)(pc.c0 + pc.q0 + w * qpt + ql) * p.h_q + g * G + h;
    const int32_t *table = p.table + (int64_t)pc.seq * p.table_stride;

    if (n_tiles == 0) {
        if (live) {   // nothing to attend: zeros
            for (int d = kg * (D / 2); d < (kg + 1) * (D / 2); d += 4) {
                if (p.o_bf16)
                    *reinterpret_cast<uint2 *>(reinterpret_cast<__nv_bfloat16 *>(p.O) + orow * D + d) = make_uint2(0, 0);
                else
                    *reinterpret_cast<float4 *>(reinterpret_cast<float *>(p.O) + orow * D + d) = make_float4(0.f, 0.f, 0.f, 0.f);
            }
            if (kg == 0 && p.lse) p.lse[orow] = -INFINITY;
        }
    } else if (warp == 16 || (warp == 17 && !VK)) {
        // --------------------------------------------------------------------------------- loads
        const bool is_k = warp == 16;
        if (is_k && elect_one()) {
            for (int i = 0; i < (two ? 2 : 1); ++i) {
                mbar_arrive_expect_tx(bars + i, (uint32_t)(L::kSlabs * 128 * qpt * G));
                for (int d = 0; d < L::kSlabs; ++d)
                    tma1_load(sQ + i * L::kTileBytes + d * 16384, &maps.q, d * 64, g * G,
                              pc.c0 + pc.q0 + i * qpt, b_q + 8 * i);
            }
        }
        __syncwarp();
        const int S = is_k ? KS : VS;
        const uint32_t full0 = is_k ? b_kFull : b_vFull, empty0 = is_k ? b_kEmpty : b_vEmpty, at0 = is_k ? sK : sV;
        const CUtensorMap *m = is_k ? maps.kv.k : maps.kv.v;
        HalfRows r[2];   // table entries read a tile ahead
#pragma unroll
        for (int i = 0; i < 2; ++i) read_entries(r[i], p, table, k0 + i * 64, k1, bxs);
        int s = u0 % S;
        uint32_t par = ((u0 / S) & 1) ^ 1;
        for (int t = 0; t < n_tiles; ++t) {
#pragma unroll
            for (int i = 0; i < 2; ++i) find_rows(r[i], p, n_cells);
            wait(empty0 + 8 * s, par);
            ok = __all_sync(0xFFFFFFFFu, ok);   // the warp's lanes agree
            if (!ok) break;
            if (elect_one()) mbar_arrive_expect_tx(bars + (full0 - bar0) / 8 + s, (uint32_t)L::kTileBytes);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 2; ++i)
                load_slabs<L::kSlabs, 16384, false>(r[i], at0 + s * L::kTileBytes + i * 8192, m, 0, g, bxs, full0 + 8 * s);
#pragma unroll
            for (int i = 0; i < 2; ++i) read_entries(r[i], p, table, k0 + (t + 1) * kT + i * 64, k1, bxs);
            if (++s == S) {
                s = 0;
                par ^= 1;
            }
        }
    } else if (warp == 18) {
        // ------------------------------------------------------------------------------ products
        if (elect_one()) {
            const uint32_t idS = idesc_bf16_f32(128, 128);
            const uint32_t idPV = idesc_bf16_f32(128, D) | (1u << 16);   // V: N-major
            const uint64_t dQ = sw128_desc(sQ, 16, 1024), dK = sw128_desc(sK, 16, 1024),
                           dV = sw128_desc(VK ? sK : sV, 16384, 1024);
            auto s_op = [&](int i, int s) {   // S of row tile i from K stage s
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t o = (kk >> 2) * 16384 + (kk & 3) * 32;
                    tc_mma_bf16(tmem + i * 128, dQ + (uint64_t)((i * L::kTileBytes + o) >> 4),
                                dK + (uint64_t)((s * L::kTileBytes + o) >> 4), idS, kk > 0 ? 1u : 0u);
                }
                tc_commit(reinterpret_cast<uint64_t *>(bars) + (b_s - bar0) / 8 + i);
            };
            auto pv_op = [&](int i, int s, bool first) {
#pragma unroll
                for (int x = 0; x < (HL ? 2 : 1); ++x)
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        mma_ts(tmem + 256 + i * D, tmem + i * 128 + (kk >> 2) * 64 + x * 32 + (kk & 3) * 8,
                               dV + (uint64_t)((s * L::kTileBytes + kk * 2048) >> 4), idPV,
                               (!first || x > 0 || kk > 0) ? 1u : 0u);
            };
            auto free_stage = [&](uint32_t empty, int s) { tc_commit(bars + (empty - bar0) / 8 + s); };
            int ks = u0 % KS, vs = u0 % (VK ? KS : VS);   // stages of K (t + 1) and V (t); VK: of K (t + 1) and K (t)
            uint32_t kp = (u0 / KS) & 1, vp = (u0 / (VK ? KS : VS)) & 1;
            auto next_k = [&]() {
                if (++ks == KS) {
                    ks = 0;
                    kp ^= 1;
                }
            };
            wait(b_q, np & 1);
            wait(b_kFull + 8 * ks, kp);
            if (ok) {
                tc_fence_after();
                s_op(0, ks);
                if (two) {
                    wait(b_q + 8, np2 & 1);
                    tc_fence_after();
                    if (ok) s_op(1, ks);
                }
                if (!VK) free_stage(b_kEmpty, ks);
            }
            next_k();
            for (int t = 0; t < n_tiles && ok; ++t) {
                const bool more = t + 1 < n_tiles;
                if (!VK) wait(b_vFull + 8 * vs, vp);
                for (int i = 0; i < (two ? 2 : 1) && ok; ++i) {
                    wait(b_p + 8 * i, ((i ? u1 : u0) + t) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    pv_op(i, vs, HL ? t % kDrain == 0 : t == 0);
                    if (more) {
                        if (i == 0) wait(b_kFull + 8 * ks, kp);
                        if (!ok) break;
                        tc_fence_after();
                        s_op(i, ks);
                    }
                }
                if (!ok) break;
                if (!more)   // both row tiles' results go out through the stages of K and V
                    for (int i = 0; i < 2; ++i) tc_commit(bars + (b_o - bar0) / 8 + i);
                free_stage(VK ? b_kEmpty : b_vEmpty, vs);
                if (more && !VK) free_stage(b_kEmpty, ks);
                next_k();
                if (++vs == (VK ? KS : VS)) {
                    vs = 0;
                    vp ^= 1;
                }
            }
            if (!ok) {   // what was issued has to end before tensor memory is given back
                tc_commit(bars + (b_drain - bar0) / 8);
                wait2(b_drain, 0);
            }
        }
        __syncwarp();
    } else if (warp < 16 && (w == 0 || two)) {
        // -------------------------------------------------------------------------------- softmax
        const int pos = TREE ? k1 : pos0 + w * qpt + ql;      // the row's last key
        const int cached = pos0 - pc.q0;                      // of a tree
        const uint32_t *mask = TREE && live ? p.mask + (int64_t)(pc.c0 + pc.q0 + w * qpt + ql) * p.mask_words : nullptr;
        const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
        // the thread's 64 columns of S; its weights take their place: 32 columns, and 32 for lo
        const uint32_t tS = tmem + w * 128 + kg * 64 + lane_addr, tO = tmem + 256 + w * D + kg * (D / 2) + lane_addr;
        const bool neg = p.scale_log2 < 0.f;
        const float sc = fmaxf(fabsf(p.scale_log2), 1e-30f);  // a zero scale: weights of 1 to 1e-28
        const float sgn = neg ? -sc : sc;
        float m = -INFINITY, l = 0.f;                         // base 2; l of this thread's keys only
        float m_sum = -INFINITY;                              // m of the sums that have moved on
        auto part_row = [&]() { return (int64_t)pc.part * p.part_rows + (pc.r0 + w * qpt + ql) * G + h; };
        auto drain = [&](bool first, bool back) {
            drain_tile<D / 2, D>(whole ? reinterpret_cast<float *>(p.O) : p.part_o, tO, whole ? orow : part_row(), live,
                                 kg * (D / 2), drain_keep(m_sum, m), first, back);
        };
        float *mine = sMax + tid, *other = sMax + (tid ^ 128);
        const int kq = k0 + kg * 64;                          // the thread's first key
        auto read_entry = [&](int key) { return key < k1 ? __ldg(table + p.page_div.div(key)) : 0; };
        int entry[2] = {read_entry(kq + lane), read_entry(kq + 32 + lane)};
        for (int t = 0; t < n_tiles; ++t) {
            const int kb = kq + t * kT;
            uint32_t cells[2];   // bit j of word x: key kb + 32 x + j has a cell
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const bool cell = kb + 32 * x + lane >= k1 || (entry[x] >= 0 && entry[x] < p.n_pages);
                if (!cell) set_status(p.status, SFA_DEV_BAD_CELL);
                cells[x] = __ballot_sync(0xFFFFFFFFu, cell);
                if constexpr (TREE) cells[x] &= tree_bits(p, mask, cached, kb + 32 * x);
                entry[x] = read_entry(kb + kT + 32 * x + lane);
            }
            const int last = min(pos, k1 - 1) - kb;           // the last key attended, from kb
            const bool masked = last < 63 || (cells[0] & cells[1]) != 0xFFFFFFFFu;
            wait(b_s + 8 * w, ((w ? u1 : u0) + t) & 1);
            tc_fence_after();
            if (HL && t > 0 && t % kDrain == 0) {   // behind P V (t - 1); few registers are in use here
                drain(t == kDrain, false);
                m_sum = m;
            }
            uint32_t r[2][32];
            tmem_ld32(tS, r[0]);
            tmem_ld32(tS + 32, r[1]);
            tmem_ld_wait();
            if (masked) {
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (32 * x + j > last || !((cells[x] >> j) & 1)) r[x][j] = neg ? 0x7F800000u : 0xFF800000u;
            }
            float mx[4];
            {   // of the scores times the scale's sign
                float hi[4], lo[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) hi[j] = lo[j] = __uint_as_float(r[0][j]);
                if (neg) {
#pragma unroll
                    for (int j = 4; j < 64; ++j) lo[j & 3] = fminf(lo[j & 3], __uint_as_float(r[j >> 5][j & 31]));
#pragma unroll
                    for (int j = 0; j < 4; ++j) mx[j] = -lo[j];
                } else {
#pragma unroll
                    for (int j = 4; j < 64; ++j) hi[j & 3] = fmaxf(hi[j & 3], __uint_as_float(r[j >> 5][j & 31]));
#pragma unroll
                    for (int j = 0; j < 4; ++j) mx[j] = hi[j];
                }
            }
            mx[0] = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            // S(t + 1) waits for every thread's weights of t: no maximum is overwritten unread
            *mine = mx[0];
            named_barrier(1 + w, 256);
            mx[0] = fmaxf(mx[0], *other) * sc;
            float alpha = 1.f;
            if (mx[0] > m + kLazy || (m == -INFINITY && mx[0] > m)) {
                alpha = ex2(m - mx[0]);
                m = mx[0];
            }
            const float mm = m == -INFINITY ? 0.f : m;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                uint32_t hi[16], lo[HL ? 16 : 1];
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    const float e0 = ex2(fmaf(__uint_as_float(r[x][j]), sgn, -mm)),
                                e1 = ex2(fmaf(__uint_as_float(r[x][j + 1]), sgn, -mm));
                    sum[j & 2] += e0;
                    sum[(j & 2) + 1] += e1;
                    hi[j / 2] = pack_bf16(e0, e1);
                    if constexpr (HL)
                        lo[j / 2] = pack_bf16(e0 - __uint_as_float(hi[j / 2] << 16),
                                              e1 - __uint_as_float(hi[j / 2] & 0xFFFF0000u));
                }
                tmem_st16(tS + 16 * x, hi);
                if constexpr (HL) tmem_st16(tS + 32 + 16 * x, lo);
            }
            // S(t) is committed behind P V (t - 1): O can be rescaled
            if (t > 0 && __any_sync(0xFFFFFFFFu, alpha != 1.f)) {
#pragma unroll 1
                for (int x = 0; x < D / 64; ++x) {
                    uint32_t o[32];
                    tmem_ld32(tO + 32 * x, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
                    tmem_st32(tO + 32 * x, o);
                }
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars + (b_p - bar0) / 8 + w);
            l = l * alpha + ((sum[0] + sum[1]) + (sum[2] + sum[3]));
        }
        // --------------------------------------------------------------------------------- result
        wait(b_o + 8 * w, np & 1);
        *mine = l;   // every maximum was read: the last weights are used up
        named_barrier(1 + w, 256);
        l += *other;
        ok = __all_sync(0xFFFFFFFFu, ok);
        tc_fence_after();
        if (ok) {
            const bool any = l > 0.f || l != l;
            const float inv = whole ? (any ? 1.f / l : 0.f) : 1.f;
            if (HL && n_tiles > kDrain) drain(false, true);
            const int64_t part = part_row();
            // NaN counts where there are keys that some query does not attend
            if (store_tile<D / 2, D>(p, sK + warp * (D * 64), tO, inv, live, whole ? orow : part, whole, kg * (D / 2),
                                     live && (TREE ? k1 > cached || p.tree == kDrafted : k1 > pos0 + 1)))
                words[kWordOdd] = 1;
            if (TREE && kg == 0)   // for add_nodes, where Q was
                reinterpret_cast<float *>(smem + L::kOffQ)[w * 128 + row] = any ? m + log2f(l) : -INFINITY;
            if (live && kg == 0) {
                if (!whole) {
                    p.part_ml[part * 2] = m;
                    p.part_ml[part * 2 + 1] = l;
                } else if (p.lse) {
                    p.lse[orow] = any ? (m + log2f(l)) / kLog2e : -INFINITY;
                }
            }
        }
        fence_proxy_async_smem();   // the next piece's loads land where the results passed
    }
    if (n_tiles > 0) {
        u0 += n_tiles;
        ++np;
        if (two) {
            u1 += n_tiles;
            ++np2;
        }
    }
}
// Between two pieces.
__device__ __forceinline__ void narrow_turn() {
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
}

// The groups of queries of piece w that are done again (odd_group), until there is none.  With its own
// code of a piece, so that the kernel's keeps its registers (24 ragged chunks take 130 us as without
// groups, 132 with one loop over pieces and groups).
template <int D, bool VK, bool HL>
__device__ __noinline__ Phases narrow_again(const NarrowMaps &maps, const Params &p, int bxs, int qpt, int n_cells,
                                            uint32_t tmem, const Piece &w, Phases ph) {
    using L = Narrow<D, VK>;
    extern __shared__ __align__(1024) uint8_t smem[];
    volatile int *words = reinterpret_cast<volatile int *>(smem + L::kOffBar + 8 * L::kBars);
    Piece *group = reinterpret_cast<Piece *>(smem + L::kOffPiece + 128);
    const int warp = threadIdx.x >> 5;
    for (int done = 0;;) {
        __syncthreads();
        if (warp == 19) {
            const Piece f = odd_group<D>(p, w, done, D);
            if ((threadIdx.x & 31) == 0) {
                *group = f;
                words[kWordOdd] = 0;
            }
        }
        narrow_turn();
        const Piece pc = *group;
        if (pc.state == kEnd || words[kWordAbort]) return ph;
        done = pc.r0 + pc.nq;
        if (warp < 19) narrow_piece<D, VK, HL, false>(maps, p, bxs, qpt, n_cells, smem, tmem, pc, ph);
        narrow_turn();
    }
}

// A tree's rows done again (odd_nodes), where there is a reason: over the cached tokens, then node by node.
template <int D, bool VK, bool HL>
__device__ __noinline__ Phases narrow_again_tree(const NarrowMaps &maps, const Params &p, int bxs, int qpt, int n_cells,
                                                 uint32_t tmem, const Piece &w, Phases ph) {
    using L = Narrow<D, VK>;
    extern __shared__ __align__(1024) uint8_t smem[];
    volatile int *words = reinterpret_cast<volatile int *>(smem + L::kOffBar + 8 * L::kBars);
    Piece *again = reinterpret_cast<Piece *>(smem + L::kOffPiece + 128);
    const int warp = threadIdx.x >> 5;
    const Nodes v = piece_nodes(p, w.pos0 - w.q0, w.k0, w.k1);
    __syncthreads();
    if (warp == 19) {
        const bool odd = odd_nodes<D>(p, v, D, w.seq, w.g, w.k0);
        Piece f = w;
        f.k1 = v.k1;
        f.state = !odd ? kEnd : f.k0 < f.k1 ? kRun : kSkip;   // kSkip: nothing of it but nodes
        if ((threadIdx.x & 31) == 0) {
            *again = f;
            words[kWordOdd] = 0;
        }
    }
    narrow_turn();
    const Piece pc = *again;
    if (pc.state == kEnd || words[kWordAbort]) return ph;
    if (warp < 19) narrow_piece<D, VK, HL, true>(maps, p, bxs, qpt, n_cells, smem, tmem, pc, ph);
    narrow_turn();
    const bool fresh = pc.state == kSkip;
    if (!words[kWordAbort]) {
        const float *lse2 = reinterpret_cast<const float *>(smem + L::kOffQ);
        for (int r = warp; r < 2 * qpt * p.G; r += kThreads / 32) {
            const int q = r / p.G, h = r - q * p.G, ql = q % qpt;
            if (q >= pc.nq) break;
            add_nodes<D, D, VK>(p, v, pc.seq, pc.g, pc.c0 + pc.q0 + q, pc.g * p.G + h,
                                pc.part < 0 ? -1 : (int64_t)pc.part * p.part_rows + (int64_t)q * p.G + h,
                                lse2[(q / qpt) * 128 + ql * p.G + h], fresh);
        }
    }
    if (threadIdx.x == 0) words[kWordOdd] = 0;   // what the pass itself saw: a cached token's
    fence_proxy_async_smem();                    // the next piece's Q lands where the sums were
    narrow_turn();
    return ph;
}

template <int D, bool VK, bool HL, bool TREE>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_narrow_kernel(const __grid_constant__ NarrowMaps maps, const __grid_constant__ Params p, int bxs, int qpt,
                        int n_cells) {
    using L = Narrow<D, VK>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *sPiece = smem + L::kOffPiece;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kOffBar);
    volatile int *words = reinterpret_cast<volatile int *>(bars + L::kBars);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // the barriers and tensor memory need nothing from global memory: they overlap the search for
    // the first piece
    if (tid == 0) {
        constexpr int ip = 2 + 2 * L::kKS + 2 * L::kVS + 2;   // b_p
        for (int i = 0; i < L::kBars; ++i) mbar_init(bars + i, i == ip || i == ip + 1 ? 8 : 1);   // P: eight warps
        words[kWordAbort] = words[kWordOdd] = 0;
        fence_mbar_init();
    }
    if (warp == 18) {
        tmem_alloc(reinterpret_cast<uint32_t *>(bars + L::kBars), 512);
        tmem_relinquish();
    }
    pdl_wait();
    Share share;   // warp 19's place in the line of all work
    if (warp == 19) {
        Piece f;
        if (p.slots > 0) {
            f = share_piece<TREE>(p, blockIdx.x, share, true);
        } else {
            f = piece_of<TREE>(p, blockIdx.x, blockIdx.y, blockIdx.z);
        }
        if (lane == 0) *reinterpret_cast<Piece *>(sPiece) = f;
    }
    narrow_turn();
    const uint32_t tmem = (uint32_t)words[kWordTmem];   // S / P: 2 x 128 columns, O: 2 x D
    Phases ph{0, 0, 0, 0, true};
    for (int i_piece = 0;; ++i_piece) {
        const Piece pc = *reinterpret_cast<const Piece *>(sPiece + (i_piece & 1) * 64);
        if (pc.state == kEnd || words[kWordAbort]) break;
        if (warp == 19) {
            Piece f;
            f.state = kEnd;
            if (p.slots > 0) f = share_piece<TREE>(p, blockIdx.x, share, false);
            if (lane == 0) *reinterpret_cast<Piece *>(sPiece + ((i_piece + 1) & 1) * 64) = f;
        } else {
            narrow_piece<D, VK, HL, TREE>(maps, p, bxs, qpt, n_cells, smem, tmem, pc, ph);
        }
        narrow_turn();
        if (words[kWordOdd]) {
            const Piece &done = *reinterpret_cast<const Piece *>(sPiece + (i_piece & 1) * 64);
            if constexpr (TREE) ph = narrow_again_tree<D, VK, HL>(maps, p, bxs, qpt, n_cells, tmem, done, ph);
            else ph = narrow_again<D, VK, HL>(maps, p, bxs, qpt, n_cells, tmem, done, ph);
        }
    }

    // ---------------------------------------------------------------------------------- teardown
    if (words[kWordAbort]) {   // copies in flight land in shared memory that is still ours
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 2000000ull) {
        }
    }
    tc_fence_after();
    __syncwarp();
    if (warp == 18) tmem_dealloc(tmem, 512);
}

template <int D, bool VK, bool HL, bool TREE>
int launch_narrow_t(const Params &p, const NarrowMaps &maps, int bxs, int qpt, int64_t n_cells, cudaStream_t st) {
    if (!ensure_max_dynamic_smem(chunk_narrow_kernel<D, VK, HL, TREE>)) return SFA_ERR_CUDA;
    if (launch_pdl(chunk_narrow_kernel<D, VK, HL, TREE>,
                   p.slots > 0 ? dim3(p.slots) : dim3(p.items, p.h_kv, p.n_split), dim3(kThreads),
                   (size_t)Narrow<D, VK>::kBytes, st, maps, p, bxs, qpt, (int)n_cells) != cudaSuccess) {
        cudaGetLastError();
        return SFA_ERR_CUDA;
    }
    return SFA_OK;
}

template <int D, bool TREE>
int launch_narrow_d(const Params &p, const NarrowMaps &maps, int bxs, int qpt, int64_t n_cells, cudaStream_t st) {
    const bool hl = !p.o_bf16;
    if (p.V)
        return hl ? launch_narrow_t<D, false, true, TREE>(p, maps, bxs, qpt, n_cells, st)
                  : launch_narrow_t<D, false, false, TREE>(p, maps, bxs, qpt, n_cells, st);
    return hl ? launch_narrow_t<D, true, true, TREE>(p, maps, bxs, qpt, n_cells, st)
              : launch_narrow_t<D, true, false, TREE>(p, maps, bxs, qpt, n_cells, st);
}

template <bool TREE>
int launch_narrow_any(const Params &p, int d, int64_t n_cells, cudaStream_t st) {
    const int qpt = narrow_qpt(p.G);
    int bxs;
    NarrowMaps maps;
    if (!encode_rows(&maps.q, p.Q, d, p.h_q, p.n_q, p.G, qpt) || !encode_keys(&maps.kv, &bxs, p, d, d, n_cells))
        return SFA_ERR_CUDA;
    return d == 128 ? launch_narrow_d<128, TREE>(p, maps, bxs, qpt, n_cells, st)
                    : launch_narrow_d<64, TREE>(p, maps, bxs, qpt, n_cells, st);
}

}  // namespace
}  // namespace chunk
}  // namespace sfa
