// chunk_wide.cu -- chunk attention with 512 value dims (576 / 512 head dims, bf16) on tcgen05
// CTA pairs.
//
// A pair of CTAs (a cluster of two, cta_group::2) owns 128 rows (query, head) of one KV head,
// 64 per CTA, and streams 128-key tiles:
//   S[128 x 128]  = Q K^T     K' = dkq, each CTA holding 64 of the keys;
//   O[128 x 512] += P V       two N = 256 products, each CTA holding 128 of their value dims.
// The shapes follow from tensor memory and shared memory.  128 rows x 512 fp32 dims of O would
// fill one CTA's tensor memory and leave none for S; a pair's M = 128 product puts a CTA's 64
// rows on all 128 lanes (the lanes' halves hold the two halves of the columns), so O takes 256
// columns and two S tiles 128.  And Q needs 72 KB a CTA instead of 144.
//
// Shared memory of a CTA: Q (9 slabs of [64 rows][64 dims], 128-byte swizzle), eight operand
// slots of 16 KB (two slabs [64 keys][64 dims]), one slab for dims 512..575, P (16 KB).  Slots 0-3
// hold S's operands, the CTA's own 64 keys, 128 dims each; slots 4-7 P V's, slot 4 + 2 half + n the
// 64 keys of `half` with value dims 256 n + 128 c ..  Where V is K a value slab is read from L2 a
// second time: keeping it from S to P V would take half the slots away from the loads in flight
// (measured: two tile buffers that keep them 4.65 us a tile, each load's latency in sight).
// Order of the products: S(t + 1), then P V (t): the softmax of tile t runs while S(t + 1) does,
// and its 16 KB of P are written once P V (t - 1) has left the buffer.
//
// For fp32 results the weights are carried as two bf16 halves (hi + lo, 2^-16 relative).  Beside
// 576-wide Q there is room for one key half's only: P V then runs by key half, the halves' hi and
// lo in the P buffer one after the other, S(t + 1) cut in two between them (beside 512-wide Q with
// both halves in place 512 tokens behind 1000 take 30 us, 36 so).  For bf16 results a weight is one bf16
// value: off by 2^-8 of itself at most, either sign, which leaves the result off by about as much as its
// own rounding does (1.7e-3 of its size each, at 64 keys as at 16384: the sum and its error shrink
// alike), and by up to 2^-8 where one key has nearly all the weight (the sum of the weights is of the
// unrounded ones).  A choice for speed: the second half doubles the products of P V.
//
// The running maximum moves only when a tile raises it by more than 2^8: weights up to 256 keep
// their relative precision in bf16 and fp32, and O in tensor memory is rescaled seldom.
//
// Pages: a key half is loaded in boxes of gcd(page, 64) rows.  Where the list ends inside one, in
// boxes of 8 rows and of one, those past the end from outside the tensor, which reads as
// zeros: cells that hold no attended token may hold NaN.
//
// Measured (576 wide, 16 heads): 512 tokens behind 8192 in 96 us, 1570 TFLOP/s, the tensor pipe 78%
// busy; 2048 behind 131072 in 5.5 ms, 1720 TFLOP/s, where the card's power is what holds it; 32 single
// tokens at 131072 in 0.89 ms, 5.4 TB/s; one at 4096 in 13.3 us, a chain of latencies.
//
// Warps 0-7: softmax, correction, result: a thread has one row, a quarter of its keys and a
// quarter of its value dims; warps 8-11: loads, one S and one P V operand of a tile each (a
// warp's barrier wait, expect and copy take about 330 cycles whatever the copy's size, a further
// copy 15: four warps reach 83 bytes a cycle and SM, one 25); warp 12: products (in the pair's
// first CTA).
#include "chunk_tc.cuh"

namespace sfa {
namespace chunk {
namespace {

constexpr int kT = 128;             // keys of a tile
constexpr int kSlab = 64 * 128;     // bytes of 64 rows x 64 dims
constexpr int kWideThreads = 416;
constexpr int kSlots = 8;           // operands of two slabs

template <int DKQ, bool HL>
struct Wide {
    static constexpr int kNSK = DKQ / 64;
    static constexpr bool kRope = kNSK > 8;
    // hi + lo weights of both key halves fit beside 512-wide Q only; else a half's at a time
    static constexpr bool kSplit = HL && kRope;
    static constexpr int kPSlabs = HL && !kRope ? 4 : 2;
    static constexpr int kOffQ = 0;
    static constexpr int kOffBuf = kNSK * kSlab;               // [kSlots][2] slabs
    static constexpr int kOffRope = kOffBuf + 2 * kSlots * kSlab;
    static constexpr int kOffP = kOffRope + (kRope ? kSlab : 0);
    static constexpr int kOffMax = kOffP + kPSlabs * kSlab;    // float [2][256]
    static constexpr int kOffItem = kOffMax + 2 * 256 * 4;     // Item and Group, 32 bytes each
    static constexpr int kOffBar = kOffItem + 64;
    static constexpr int kBars = 1 + 2 * kSlots + 2 + 2 + 2 + 2 + 1;
    static constexpr int kBytes = kOffBar + kBars * 8 + 16;
    static_assert(kBytes <= 227 * 1024, "fits one CTA per SM");
};

// What a pass works on: nq queries of a row tile, from its query r0 on (at position pos0 of q0), and keys k0 .. k1.
struct Work {
    Item it;
    int item, g, split, q0, pos0, len, k0;
    int r0, nq, k1, n_tiles;
    int tb, np;        // tiles and passes before: the barriers' phases go on
    uint32_t tmem;
};
// Queries that are done again (odd_group).
struct Group {
    int state, r0, nq, k1;
};

struct WideMaps {
    CUtensorMap q;
    KeyMaps kv;
};

// --------------------------------------------------------------- pair (cta_group::2) wrappers
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// This shared address in the pair's first CTA, as a shared::cluster address.
__device__ __forceinline__ uint32_t in_leader(uint32_t saddr) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(saddr));
    return r;
}
// Arrives on a barrier of the other CTA.  What it publishes is this CTA's own shared memory, for
// the async proxy (fenced before): no release at cluster scope, which would also wait for the
// thread's loads in flight (measured: 1.8 to 3.9 thousand cycles a tile).
__device__ __forceinline__ void arrive_cluster(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
                 : "memory");
}
// A word into this shared address of the pair's CTA `rank`.
__device__ __forceinline__ void store_in(uint32_t saddr, uint32_t rank, int v) {
    asm volatile(
        "{\n\t.reg .b32 a;\n\t"
        "mapa.shared::cluster.u32 a, %0, %1;\n\t"
        "st.shared::cluster.u32 [a], %2;\n\t}" ::"r"(saddr),
        "r"(rank), "r"(v)
        : "memory");
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void mma2(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// Arrives on this barrier of both CTAs when the products issued so far are done.
__device__ __forceinline__ void commit2(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}
// --------------------------------------------------------------------------------- the kernel
// The words behind the barriers: tensor memory's address; a wait ran out; a result of either CTA is not
// finite; in the first CTA: a wait of the other one's ran out.
enum { kWordTmem, kWordAbort, kWordOdd, kWordOtherAbort };

// Where a list has no key: zeros.
__device__ __forceinline__ void wide_zeros(const Params &p, const Work &wk, int qpc) {
    const int warp = threadIdx.x >> 5, c = (int)cluster_rank(), G = p.G;
    const int row = (warp & 1) * 32 + (threadIdx.x & 31), part = 2 * ((warp >> 1) & 1) + (warp >> 2);
    const int ql = row / G, h = row - ql * G;
    if (warp >= 8 || ql >= qpc || c * qpc + ql >= wk.nq) return;
    const int64_t orow = (int64_t)(wk.it.q.c0 + wk.q0 + wk.r0 + c * qpc + ql) * p.h_q + wk.g * G + h;
    for (int d = part * 128; d < (part + 1) * 128; d += 4) {
        if (p.o_bf16)
            *reinterpret_cast<uint2 *>(reinterpret_cast<__nv_bfloat16 *>(p.O) + orow * 512 + d) = make_uint2(0, 0);
        else
            *reinterpret_cast<float4 *>(reinterpret_cast<float *>(p.O) + orow * 512 + d) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (part == 0 && p.lse) p.lse[orow] = -INFINITY;
}

template <int DKQ, bool VK, bool HL>
__device__ __forceinline__ void wide_pass(const WideMaps &maps, const Params &p, int bxs, int qpc, int n_cells,
                                          uint8_t *smem, const Work &wk) {
    using L = Wide<DKQ, HL>;
    constexpr bool SPLIT = L::kSplit;
    float *sMax = reinterpret_cast<float *>(smem + L::kOffMax);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kOffBar);
    volatile int *words = reinterpret_cast<volatile int *>(bars + L::kBars), *abort_flag = words + kWordAbort;
    const uint32_t bar0 = smem_u32(bars);
    // barriers, as shared addresses
    const uint32_t b_q = bar0, b_full = bar0 + 8, b_empty = b_full + 8 * kSlots, b_rope = b_empty + 8 * kSlots,
                   b_ropeDone = b_rope + 8, b_s = b_ropeDone + 8, b_p = b_s + 16, b_pv = b_p + 16,
                   b_drain = b_pv + 16;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int c = (int)cluster_rank();
    const Item &it = wk.it;
    const int item = wk.item, g = wk.g, split = wk.split, q0 = wk.q0, r0 = wk.r0, nq = wk.nq, pos0 = wk.pos0;
    const int k0 = wk.k0, k1 = wk.k1, n_tiles = wk.n_tiles, tb = wk.tb, np = wk.np, G = p.G;
    const bool whole = wk.len <= p.split_keys;
    const uint32_t tmem = wk.tmem;

    // a softmax thread's row: query ql of this CTA's qpc, head h.  Both halves hh of the tensor
    // memory lanes have every row, and two warps (cg) share a lane's columns.
    const int row = (warp & 1) * 32 + lane, hh = (warp >> 1) & 1, cg = warp >> 2;
    const int ql = row / G, h = row - ql * G;
    const bool live = warp < 8 && ql < qpc && c * qpc + ql < nq;
    const int64_t orow = (int64_t)(it.q.c0 + q0 + r0 + c * qpc + ql) * p.h_q + g * G + h;

    const uint32_t tS = tmem, tO = tmem + 128;   // S: 2 x 64 columns, O: 2 x 128
    const uint32_t buf0 = smem_u32(smem + L::kOffBuf), sQ = smem_u32(smem + L::kOffQ),
                   sRope = smem_u32(smem + L::kOffRope), sP = smem_u32(smem + L::kOffP);
    // once a wait ran out no other is made
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (ok && !wait2(bar, parity)) {
            ok = false;
            *abort_flag = 1;
            set_status(p.status, SFA_DEV_TIMEOUT);
        }
    };
    const int32_t *table = p.table + (int64_t)it.seq * p.table_stride;

    if (warp >= 8 && warp < 12) {
        // ------------------------------------------------------------------------------- loads
        const int j = warp - 8, half = j >> 1, n = j & 1;
        const uint32_t lead = in_leader(bar0);
        if (j == 0 && elect_one()) {
            if (c == 0) mbar_arrive_expect_tx(bars, 2u * L::kNSK * 128u * (uint32_t)(qpc * G));
            for (int d = 0; d < L::kNSK; ++d)
                tma2_load(sQ + d * kSlab, &maps.q, d * 64, g * G, it.q.c0 + q0 + r0 + c * qpc, lead);
        }
        __syncwarp();
        const uint32_t s_full = b_full + j * 8, s_empty = b_empty + j * 8, v_full = s_full + 32, v_empty = s_empty + 32;
        const uint32_t s_at = buf0 + 2 * j * kSlab, v_at = s_at + 8 * kSlab;
        const CUtensorMap *vm = VK ? maps.kv.k : maps.kv.v;
        const int vx = 256 * n + 128 * c;
        // keys of S: this CTA's half; of P V: `half`.  Their table entries are read a tile ahead.
        if (bxs == 6) {
            // a half tile lies in one page: one thread does it all, the next slot looked at ahead
            if (elect_one()) {
                auto entry = [&](int pos) { return pos < k1 ? __ldg(table + p.page_div.div(pos)) : -1; };
                auto row = [&](int e, int pos) {
                    return e < 0 || e >= p.n_pages ? n_cells : e * p.page + (pos - p.page_div.div(pos) * p.page);
                };
                auto rows_in = [&](int r, int pos) { return r == n_cells ? 0 : max(0, min(64, k1 - pos)); };
                auto expect = [&](uint32_t full, uint32_t bytes) {
                    if (c == 0) mbar_arrive_expect_tx(bars + (full - bar0) / 8, bytes);
                };
                int ps = k0 + c * 64, pv = k0 + half * 64;
                int es = entry(ps), ev = entry(pv);
                bool there = tb == 0;
                for (int t = -1; t < n_tiles && ok; ++t) {
                    const int T = tb + t;
                    if (t + 1 < n_tiles) {
                        const int r = row(es, ps), v = rows_in(r, ps);
                        es = entry(ps + kT);
                        if (!there) wait(s_empty, T & 1);
                        if (!ok) break;
                        expect(s_full, 4u * kSlab);
                        load_slabs_one<2, kSlab, true>(r, v, s_at, maps.kv.k, 128 * j, g, n_cells, lead + (s_full - bar0));
                        if (L::kRope && j == 3) {
                            wait(b_ropeDone, T & 1);
                            if (!ok) break;
                            expect(b_rope, 2u * kSlab);
                            load_slabs_one<1, kSlab, true>(r, v, sRope, maps.kv.k, 512, g, n_cells, lead + (b_rope - bar0));
                        }
                        ps += kT;
                    }
                    if (t >= 0) {
                        there = mbar_test_wait(v_empty, (T & 1) ^ 1);
                        const int r = row(ev, pv), v = rows_in(r, pv);
                        ev = entry(pv + kT);
                        if (!there) wait(v_empty, (T & 1) ^ 1);
                        if (!ok) break;
                        there = t + 2 < n_tiles && mbar_test_wait(s_empty, (T + 1) & 1);
                        expect(v_full, 4u * kSlab);
                        load_slabs_one<2, kSlab, true>(r, v, v_at, vm, vx, g, n_cells, lead + (v_full - bar0));
                        pv += kT;
                    } else {
                        there = n_tiles > 1 && mbar_test_wait(s_empty, (T + 1) & 1);
                    }
                }
            }
            __syncwarp();
        } else {
            HalfRows hs, hv;
            read_entries(hs, p, table, k0 + c * 64, k1, bxs);
            read_entries(hv, p, table, k0 + half * 64, k1, bxs);
            auto slot_free = [&](uint32_t full, uint32_t empty, uint32_t parity, uint32_t bytes) {
                wait(empty, parity);
                ok = __all_sync(0xFFFFFFFFu, ok);   // the warp's lanes agree
                if (ok && c == 0 && elect_one()) mbar_arrive_expect_tx(bars + (full - bar0) / 8, bytes);
                __syncwarp();
            };
            for (int t = -1; t < n_tiles && ok; ++t) {
                const int T = tb + t;
                if (t + 1 < n_tiles) {
                    find_rows(hs, p, n_cells);
                    slot_free(s_full, s_empty, (T & 1), 4u * kSlab);
                    if (!ok) break;
                    load_slabs<2, kSlab, true>(hs, s_at, maps.kv.k, 128 * j, g, bxs, lead + (s_full - bar0));
                    if (L::kRope && j == 3) {
                        slot_free(b_rope, b_ropeDone, (T & 1), 2u * kSlab);
                        if (!ok) break;
                        load_slabs<1, kSlab, true>(hs, sRope, maps.kv.k, 512, g, bxs, lead + (b_rope - bar0));
                    }
                    read_entries(hs, p, table, k0 + (t + 2) * kT + c * 64, k1, bxs);
                }
                if (t >= 0) {
                    find_rows(hv, p, n_cells);
                    slot_free(v_full, v_empty, (T & 1) ^ 1, 4u * kSlab);
                    if (!ok) break;
                    load_slabs<2, kSlab, true>(hv, v_at, vm, vx, g, bxs, lead + (v_full - bar0));
                    read_entries(hv, p, table, k0 + (t + 1) * kT + half * 64, k1, bxs);
                }
            }
        }
    } else if (warp == 12) {
        // ----------------------------------------------------------------------------- products
        if (c == 0 && elect_one()) {
            const uint32_t idS = idesc_bf16_f32(128, 128);
            const uint32_t idPV = idesc_bf16_f32(128, 256) | (1u << 16);   // V: N-major
            const uint64_t dQ = sw128_desc(sQ, 16, 1024), dBuf = sw128_desc(buf0, 16, 1024),
                           dRope = sw128_desc(sRope, 16, 1024), dP = sw128_desc(sP, 16, 1024),
                           dV = sw128_desc(buf0 + 8 * kSlab, kSlab, 1024);
            // an operand's barrier is looked at before the products of the one ahead of it
            bool there = false;
            auto take = [&](uint32_t bar, uint32_t parity) {
                if (!there) wait(bar, parity);
                tc_fence_after();
            };
            auto s_ops = [&](int T, int i0, int i1) {
                for (int i = i0; i < i1; ++i) {
                    take(b_full + i * 8, T & 1);
                    if (!ok) return;
                    there = i < 3 ? mbar_test_wait(b_full + (i + 1) * 8, T & 1)
                                  : L::kRope && mbar_test_wait(b_rope, T & 1);
#pragma unroll
                    for (int s = 0; s < 2; ++s)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma2(tS + (T & 1) * 64, dQ + (uint64_t)(((2 * i + s) * kSlab + kk * 32) >> 4),
                                 dBuf + (uint64_t)(((2 * i + s) * kSlab + kk * 32) >> 4), idS,
                                 (i > 0 || s > 0 || kk > 0) ? 1u : 0u);
                    commit2(b_empty + i * 8);
                }
            };
            auto s_end = [&](int T) {
                if (L::kRope) {
                    take(b_rope, T & 1);
                    if (!ok) return;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma2(tS + (T & 1) * 64, dQ + (uint64_t)((8 * kSlab + kk * 32) >> 4),
                             dRope + (uint64_t)((kk * 32) >> 4), idS, 1u);
                    commit2(b_ropeDone);
                }
                commit2(b_s + (T & 1) * 8);
                there = false;
            };
            auto pv_ops = [&](int t, int half) {
                const int T = tb + t;
                if (SPLIT || half == 0) wait(b_p + half * 8, T & 1);
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const int i = 2 * half + n;
                    take(b_full + (4 + i) * 8, T & 1);
                    if (!ok) return;
                    there = n == 0 ? mbar_test_wait(b_full + (5 + i) * 8, T & 1) : false;
#pragma unroll
                    for (int x = 0; x < (HL ? 2 : 1); ++x)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma2(tO + n * 128, dP + (uint64_t)(((SPLIT ? x : HL ? 2 * half + x : half) * kSlab + kk * 32) >> 4),
                                 dV + (uint64_t)((2 * i * kSlab + kk * 2048) >> 4), idPV,
                                 ((HL ? t % kDrain : t) > 0 || half > 0 || x > 0 || kk > 0) ? 1u : 0u);
                    commit2(b_empty + (4 + i) * 8);
                }
                if (SPLIT || half == 1) commit2(b_pv + half * 8);
            };
            wait(b_q, np & 1);
            for (int t = -1; t < n_tiles && ok; ++t) {
                const bool more = t + 1 < n_tiles;
                if (more) s_ops(tb + t + 1, 0, SPLIT ? 2 : 4);
                if (!SPLIT && more && ok) s_end(tb + t + 1);
                if (SPLIT) there = false;
                if (t >= 0 && ok) pv_ops(t, 0);
                if (SPLIT && more && ok) {
                    s_ops(tb + t + 1, 2, 4);
                    if (ok) s_end(tb + t + 1);
                }
                if (t >= 0 && ok) pv_ops(t, 1);
            }
            if (!ok) {   // what was issued has to end before tensor memory is given back
                commit2(b_drain);
                wait2(b_drain, 0);
            }
        }
        __syncwarp();
    } else if (warp < 8) {
        // ------------------------------------------------------------------------------ softmax
        const int pos = pos0 + r0 + c * qpc + ql;             // the row's last key
        const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
        const bool neg = p.scale_log2 < 0.f;
        // a zero scale: weights of 1 to 1e-28
        const float sc = fmaxf(fabsf(p.scale_log2), 1e-30f);
        const uint32_t p_ready0 = in_leader(b_p), p_ready1 = p_ready0 + 8;
        float m = -INFINITY, l = 0.f;                         // base 2; l of this thread's keys only
        float m_sum = -INFINITY;                              // m of the sums that have moved on
        auto part_row = [&]() {
            return (((int64_t)item * p.h_kv + g) * p.n_split + split) * p.part_rows + (r0 + c * qpc + ql) * G + h;
        };
        auto drain = [&](bool first, bool back) {   // columns 128 cg ..: dims 256 cg + 128 hh ..
            drain_tile<128, 512>(whole ? reinterpret_cast<float *>(p.O) : p.part_o, tO + cg * 128 + lane_addr,
                                 whole ? orow : part_row(), live, cg * 256 + hh * 128, drain_keep(m_sum, m), first, back);
        };
        const int kq = k0 + hh * 64 + cg * 32;                // the thread's first key
        auto read_entry = [&](int key) { return key < k1 ? __ldg(table + p.page_div.div(key)) : 0; };
        int entry = read_entry(kq + lane);
        for (int t = 0; t < n_tiles; ++t) {
            const int T = tb + t;
            const uint32_t b = T & 1, par = (T >> 1) & 1;
            const int kb = kq + t * kT;
            // bit j: key kb + j has a cell (its entry was read a tile ago)
            const bool cell = kb + lane >= k1 || (entry >= 0 && entry < p.n_pages);
            if (!cell) set_status(p.status, SFA_DEV_BAD_CELL);
            const uint32_t cells = __ballot_sync(0xFFFFFFFFu, cell);
            entry = read_entry(kb + kT + lane);
            const int last = min(pos, k1 - 1) - kb;           // the last key attended, from kb
            if (HL && t > 0 && t % kDrain == 0) {   // here, where few registers are in use
                wait(b_pv + 8, (T - 1) & 1);
                tc_fence_after();
                drain(t == kDrain, false);
                m_sum = m;
            }
            wait(b_s + b * 8, par);
            tc_fence_after();
            uint32_t r[32];
            tmem_ld32(tS + b * 64 + cg * 32 + lane_addr, r);
            tmem_ld_wait();
            tc_fence_before();
            float s[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) s[j] = __uint_as_float(r[j]);
            if (neg) {
#pragma unroll
                for (int j = 0; j < 32; ++j) s[j] = -s[j];
            }
            if (last < 31 || cells != 0xFFFFFFFFu) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (j > last || !((cells >> j) & 1)) s[j] = -INFINITY;
            }
            float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int j = 4; j < 32; ++j) mx[j & 3] = fmaxf(mx[j & 3], s[j]);
            mx[0] = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            float *mb = sMax + b * 256;
            mb[tid] = mx[0];
            named_barrier(1, 256);
            mx[0] = fmaxf(fmaxf(mx[0], mb[tid ^ 64]), fmaxf(mb[tid ^ 128], mb[tid ^ 192])) * sc;
            float alpha = 1.f;
            if (mx[0] > m + kLazy || (m == -INFINITY && mx[0] > m)) {
                alpha = ex2(m - mx[0]);
                m = mx[0];
            }
            const float mm = m == -INFINITY ? 0.f : m;
            float sum[2] = {0.f, 0.f};
            uint32_t hi[16], lo[HL ? 16 : 1];
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
                const float e0 = ex2(fmaf(s[j], sc, -mm)), e1 = ex2(fmaf(s[j + 1], sc, -mm));
                sum[0] += e0;
                sum[1] += e1;
                hi[j / 2] = pack_bf16(e0, e1);
                if constexpr (HL)
                    lo[j / 2] = pack_bf16(e0 - __uint_as_float(hi[j / 2] << 16),
                                          e1 - __uint_as_float(hi[j / 2] & 0xFFFF0000u));
            }
            l = l * alpha + (sum[0] + sum[1]);
            // the products of the tile before are done with P and O
            if (t > 0) wait(b_pv + 8, (T - 1) & 1);
            if (t > 0 && __any_sync(0xFFFFFFFFu, alpha != 1.f)) {
                tc_fence_after();
#pragma unroll 1
                for (int x = 0; x < 4; ++x) {
                    tmem_ld32(tO + (cg * 4 + x) * 32 + lane_addr, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * alpha);
                    tmem_st32(tO + (cg * 4 + x) * 32 + lane_addr, r);
                }
                tmem_st_wait();
                tc_fence_before();
            }
            auto write = [&](const uint32_t *w, uint32_t slab) {
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                     slab + row * 128 + (((cg * 4 + x) ^ (row & 7)) << 4)),
                                 "r"(w[4 * x]), "r"(w[4 * x + 1]), "r"(w[4 * x + 2]), "r"(w[4 * x + 3])
                                 : "memory");
            };
            if constexpr (SPLIT) {
                if (hh == 1) {   // O is rescaled; then P's second half, when the first is used up
                    __syncwarp();
                    if (lane == 0) arrive_cluster(p_ready0);
                    wait(b_pv, T & 1);
                }
                write(hi, sP);
                write(lo, sP + kSlab);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) arrive_cluster(hh == 1 ? p_ready1 : p_ready0);
            } else {
                write(hi, sP + (HL ? 2 * hh : hh) * kSlab);
                if constexpr (HL) write(lo, sP + (2 * hh + 1) * kSlab);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) arrive_cluster(p_ready0);
            }
        }
        // -------------------------------------------------------------------------------- result
        {   // the buffer that the last tile's maxima did not use
            float *lb = sMax + ((tb + n_tiles) & 1) * 256;
            lb[tid] = l;
            named_barrier(1, 256);
            l = (l + lb[tid ^ 64]) + (lb[tid ^ 128] + lb[tid ^ 192]);
        }
        if (tid == 0 && p.n_split > 1) let_next_start();   // the merge: what else may follow is not known
        wait(b_pv + 8, (tb + n_tiles - 1) & 1);
        ok = __all_sync(0xFFFFFFFFu, ok);
        tc_fence_after();
        if (ok) {
            const bool any = l > 0.f || l != l;
            const float inv = whole ? (any ? 1.f / l : 0.f) : 1.f;
            if (HL && n_tiles > kDrain) drain(false, true);
            const int64_t part = part_row();
            // columns 128 cg ..: dims 256 cg + 128 hh ..; every operand is used up
            // NaN counts where there are keys that some query does not attend
            if (store_tile<128, 512>(p, buf0 + warp * 16384, tO + cg * 128 + lane_addr, inv, live, whole ? orow : part,
                                     whole, cg * 256 + hh * 128, live && k1 > pos0 + 1)) {
                store_in(smem_u32(bars + L::kBars) + 4 * kWordOdd, 0, 1);
                store_in(smem_u32(bars + L::kBars) + 4 * kWordOdd, 1, 1);
            }
            if (live && hh == 0 && cg == 0) {
                if (!whole) {
                    p.part_ml[part * 2] = m;
                    p.part_ml[part * 2 + 1] = l;
                } else if (p.lse) {
                    p.lse[orow] = any ? (m + log2f(l)) / kLog2e : -INFINITY;
                }
            }
        }
    }

    // ------------------------------------------------------------------------- the pass's end
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {   // copies in flight land in shared memory that is still ours
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 2000000ull) {
        }
    }
    __syncwarp();
    cluster_sync_all();   // neither CTA leaves while the other's products or arrivals need it
    tc_fence_after();
}

// The groups of queries that are done again (odd_group), until there is none: the pair's first CTA says
// which.  Inlined, with a pass of its own: a call that is not, or one loop over passes, takes the kernel's
// products and copies out of uniform registers (512 tokens behind 8192 took 103 to 107 us, and 100; 98 so,
// 97 without groups; one token at 4096 13.4, 13.0 without).
template <int DKQ, bool VK, bool HL>
__device__ __forceinline__ void wide_again(const WideMaps &maps, const Params &p, int bxs, int qpc, int n_cells, Work wk) {
    using L = Wide<DKQ, HL>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, c = (int)cluster_rank();
    volatile int *words = reinterpret_cast<volatile int *>(smem + L::kOffBar + 8 * L::kBars);
    const Group *group = reinterpret_cast<const Group *>(smem + L::kOffItem + 32);
    const int end = wk.k1;
    int done = 0;
    for (;;) {
        wk.tb += wk.n_tiles;
        wk.np += wk.n_tiles > 0;
        if (c == 1 && tid == 0)
            store_in(smem_u32(smem + L::kOffBar + 8 * L::kBars) + 4 * kWordOtherAbort, 0, words[kWordAbort]);
        fence_proxy_async_smem();   // the next pass's loads land where the results passed
        __syncwarp();
        cluster_sync_all();
        if (c == 0 && warp == 0) {
            Piece w;
            w.seq = wk.it.seq;
            w.g = wk.g;
            w.q0 = wk.q0;
            w.pos0 = wk.pos0;
            w.k0 = wk.k0;
            w.k1 = end;
            w.part = wk.len <= p.split_keys ? -1 : 0;
            const Piece f = odd_group<512>(p, w, done, VK ? DKQ : 512);
            if ((tid & 31) == 0) {
                const int v[4] = {words[kWordAbort] || words[kWordOtherAbort] ? (int)kEnd : f.state, f.r0, f.nq, f.k1};
                for (int i = 0; i < 8; ++i) store_in(smem_u32(group) + 4 * (i & 3), i >> 2, v[i & 3]);
            }
        }
        __syncwarp();
        cluster_sync_all();
        if (group->state == kEnd) return;
        wk.r0 = group->r0;
        wk.nq = group->nq;
        wk.k1 = group->k1;
        done = wk.r0 + wk.nq;
        wk.n_tiles = max(0, (wk.k1 - wk.k0 + kT - 1) / kT);
        if (wk.n_tiles > 0) wide_pass<DKQ, VK, HL>(maps, p, bxs, qpc, n_cells, smem, wk);
        else if (group->state == kRun) wide_zeros(p, wk, qpc);
    }
}

template <int DKQ, bool VK, bool HL>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWideThreads, 1)
    chunk_wide_kernel(const __grid_constant__ WideMaps maps, const Params p, int bxs, int qpc, int n_cells) {
    using L = Wide<DKQ, HL>;
    extern __shared__ __align__(1024) uint8_t smem[];
    Item *sItem = reinterpret_cast<Item *>(smem + L::kOffItem);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kOffBar);
    volatile int *words = reinterpret_cast<volatile int *>(bars + L::kBars);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Work wk;
    wk.item = blockIdx.x >> 1;
    wk.g = blockIdx.y;
    wk.split = blockIdx.z;
    // the barriers, tensor memory and the pair's meeting need nothing from global memory: they
    // overlap the search for the item
    if (tid == 0) {
        const int ip = 1 + 2 * kSlots + 2 + 2;   // b_p
        // P (half 0) ready: eight warps of each CTA; P half 1: four of each
        for (int i = 0; i < L::kBars; ++i) mbar_init(bars + i, i == ip ? 16 : i == ip + 1 ? 8 : 1);
        words[kWordAbort] = words[kWordOdd] = words[kWordOtherAbort] = 0;
        fence_mbar_init();
    }
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         smem_u32(bars + L::kBars))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    pdl_wait();
    if (warp == 0) {
        const Item it = find_item(p, wk.item, (blockIdx.x & 1) == 0 && wk.g == 0 && wk.split == 0);
        if (lane == 0) *sItem = it;
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    tc_fence_after();
    wk.tmem = (uint32_t)words[kWordTmem];
    auto leave = [&]() {   // both CTAs of the pair, with nothing in flight
        if (warp == 12)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(wk.tmem) : "memory");
    };
    wk.it = *sItem;
    if (wk.it.seq < 0) return leave();
    wk.q0 = wk.it.tile * p.item_q;                            // first query of the tile
    wk.r0 = 0;
    wk.nq = min(p.item_q, min(wk.it.q.n, p.n_new_max) - wk.q0);
    wk.pos0 = wk.it.q.total - wk.it.q.n + wk.q0;              // its position
    wk.len = max(0, min(key_limit(p, wk.it.q), wk.pos0 + wk.nq));
    wk.k0 = (int)min((int64_t)wk.len, (int64_t)wk.split * p.split_keys);
    wk.k1 = (int)min((int64_t)wk.len, (int64_t)wk.k0 + p.split_keys);
    if (wk.split > 0 && wk.k0 >= wk.k1) return leave();       // no such piece
    wk.n_tiles = (wk.k1 - wk.k0 + kT - 1) / kT;
    wk.tb = wk.np = 0;
    if (wk.n_tiles == 0) {   // nothing to attend
        wide_zeros(p, wk, qpc);
        return leave();
    }
    wide_pass<DKQ, VK, HL>(maps, p, bxs, qpc, n_cells, smem, wk);
    if (words[kWordOdd]) wide_again<DKQ, VK, HL>(maps, p, bxs, qpc, n_cells, wk);
    leave();
}

template <int DKQ, bool VK, bool HL>
int launch_wide_t(const Params &p, const WideMaps &maps, int bxs, int qpc, int64_t n_cells, cudaStream_t st) {
    if (!ensure_max_dynamic_smem(chunk_wide_kernel<DKQ, VK, HL>)) return SFA_ERR_CUDA;
    if (launch_pdl(chunk_wide_kernel<DKQ, VK, HL>, dim3(2 * p.items, p.h_kv, p.n_split), dim3(kWideThreads),
                   (size_t)Wide<DKQ, HL>::kBytes, st, maps, p, bxs, qpc, (int)n_cells) != cudaSuccess) {
        cudaGetLastError();
        return SFA_ERR_CUDA;
    }
    return SFA_OK;
}

}  // namespace

int launch_wide(const Params &p, int dkq, int64_t n_cells, cudaStream_t st) {
    const int qpc = wide_qpc(p.G);
    int bxs;
    WideMaps maps;
    if (!encode_rows(&maps.q, p.Q, dkq, p.h_q, p.n_q, p.G, qpc) ||
        !encode_keys(&maps.kv, &bxs, p, dkq, 512, n_cells))
        return SFA_ERR_CUDA;
    const bool hl = !p.o_bf16;
    if (dkq == 576)
        return hl ? launch_wide_t<576, true, true>(p, maps, bxs, qpc, n_cells, st)
                  : launch_wide_t<576, true, false>(p, maps, bxs, qpc, n_cells, st);
    if (p.V)
        return hl ? launch_wide_t<512, false, true>(p, maps, bxs, qpc, n_cells, st)
                  : launch_wide_t<512, false, false>(p, maps, bxs, qpc, n_cells, st);
    return hl ? launch_wide_t<512, true, true>(p, maps, bxs, qpc, n_cells, st)
              : launch_wide_t<512, true, false>(p, maps, bxs, qpc, n_cells, st);
}

}  // namespace chunk
}  // namespace sfa
