// chunk_f32_tree.cu -- attention of drafted trees over fp32 caches.
//
// Both products run on binary16 operands (mma.sync, twice tf32's rate for each of its steps): a row is brought
// to a largest value of 2^10 .. 2^11 by a power of two and cut in hi + lo of 11 bits each, which leaves 2^-22 of a
// value (2^-35 of the row's largest at least), and of the four products the three larger ones are taken.
//   scores: the rows' powers of two come back with the scale;
//   values: a key's power goes into its weight, relative to a power u of the row (query, head) that its largest
//           weights 2^-sv_k p_k set: sum_k (p_k 2^(-sv_k - u)) (2^sv_k v_k) = 2^-u sum_k p_k v_k.  So a token of large
//           values costs only those rows precision to whose result it adds much.
// The running maximum moves by more than 2^8 only, u by more than 2^4 (weights stay below 2^15).
// A row is read, scaled and cut once for all 64 rows (query, head) of the CTA's tile; the next tile's rows are on
// their way to registers meanwhile.  Scores: a warp has 16 rows and 16 keys, wide heads' by a quarter (a half) of
// the dims, which the warps of a row group add up through shared memory; then a row's softmax is one warp's.
// Values: a warp has 32 dims of all rows (with values apart 64; narrow heads: of 32 or 16 rows), sixteen keys' sum
// is added with rounding.
// Values that are not finite are taken out of the operands: a score with one is a plain product instead, and such
// values are added one by one to the rows that attend them.
// 17 trees of 3 behind 27053, 576 wide, 16 heads: 863 us, 55 TFLOP/s of the rows alone (1679 by three tf32 products on
// 32 rows; 1010 with eight warps, each with its 16 rows' scores of 8 keys, which read the queries twice as often).
// 15 of 20 behind 17048, 128 wide, 16 heads on 4: 1101 us (2626).  It is bound by its phases, rows to shared memory,
// scores, softmax and values, which follow one another with a barrier each: scores at shared memory's rate (the
// queries are read for each tile), the others at instructions' latency.  16 warps need all 64 thousand registers: with
// values apart they would spill (1 tree of 133 behind 10852: 1167 us, eight warps 892).
#include "chunk_common.cuh"

namespace sfa {
namespace chunk {
namespace {

constexpr int kTop = 10;   // the exponent of a scaled row's largest value

template <int DKQ, int DV, bool VK>
struct F32T {
    static constexpr int kWarps = DV == 512 && VK ? 16 : 8;           // with values apart: registers
    static constexpr int kTK = DV == 512 ? 16 : 32;                   // keys of a tile
    static constexpr int kWG = kWarps / 4;                            // warps of 16 rows' scores: a tile of 16 keys
    static constexpr int kParts = kWG / (kTK / 16);                   // by so many parts of the dims each
    static constexpr int kLR = 2 * kWG;                               // softmax: lanes of a row
    static constexpr int kPQ = DKQ + 8, kPV = DV + 8, kPS = kTK + 8;  // pitches: ldmatrix without bank conflicts
    static constexpr int kOffK = 2 * kF32Rows * kPQ * 2;              // hi, lo of the queries before
    static constexpr int kOffV = kOffK + 2 * kTK * kPQ * 2;
    static constexpr int kOffP = kOffV + (VK ? 0 : 2 * kTK * kPV * 2);
    static constexpr int kOffS = kOffP + 2 * kF32Rows * kPS * 2;      // float [kParts][64][kPS]
    static constexpr int kOffCell = kOffS + kParts * kF32Rows * kPS * 4;   // int64 [2][kTK]: this tile's and the next one's
    static constexpr int kOffUnit = kOffCell + 2 * kTK * 8;           // float2: keys' and values' powers of two, undone
    static constexpr int kOffRow = kOffUnit + (VK ? 1 : 2) * kTK * 8; // int: rows' powers of two
    static constexpr int kOffAlpha = kOffRow + kF32Rows * 4;
    static constexpr int kOffOdd = kOffAlpha + kF32Rows * 4;          // int [64] of queries, [kTK]: 1 key, 2 value
    static constexpr int kBytes = kOffOdd + (kF32Rows + kTK) * 4;
    static constexpr int kBlocks = DV / 32;                           // values: blocks of 32 dims and row tiles of a warp
    static constexpr int kBW = kBlocks >= kWarps ? kBlocks / kWarps : 1, kMW = kBlocks >= kWarps ? 4 : 4 * kBlocks / kWarps;
    static_assert(kBytes + 64 <= 227 * 1024, "shared memory");
    static_assert(kOffCell % 8 == 0, "aligned");
};

__device__ __forceinline__ bool finite(float x) { return x - x == 0.f; }
// 2^e for e within [-126, 127]; below: 0.
__device__ __forceinline__ float pow2(int e) { return e < -126 ? 0.f : __uint_as_float((uint32_t)(127 + e) << 23); }
// mma_f16_16816 onto zeros.
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// 2^e as two factors, which may be out of range together.
__device__ __forceinline__ float2 pow2_halves(int e) { return make_float2(pow2(e >> 1), pow2(e - (e >> 1))); }
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void split_f16(float x, float y, __half2 &hi, __half2 &lo) {
    hi = __floats2half2_rn(x, y);
    const float2 h = __half22float2(hi);
    lo = __floats2half2_rn(x - h.x, y - h.y);
}

// One row, N pairs a lane (elements 64 i + 2 lane): scaled and cut into hi (at `to`) and lo (`apart` behind).
// Returns its power of two; odd: it has values that are not finite, which become zeros.  By one whole warp.
template <int N>
__device__ __forceinline__ int put_row(float2 (&v)[N], __half *to, int apart, bool &odd) {
    const int lane = threadIdx.x & 31;
    auto largest = [&]() {   // its bits
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
            top = max(top, max(__float_as_uint(v[i].x) & 0x7FFFFFFFu, __float_as_uint(v[i].y) & 0x7FFFFFFFu));
        return __reduce_max_sync(0xFFFFFFFFu, top);
    };
    uint32_t top = largest();
    odd = top >= 0x7F800000u;
    if (odd) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (!finite(v[i].x)) v[i].x = 0.f;
            if (!finite(v[i].y)) v[i].y = 0.f;
        }
        top = largest();
    }
    const int e = min(126, kTop - ((int)(top >> 23) - 127));   // a row of zeros: 126
    const float f = pow2(e);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        __half2 hi, lo;
        split_f16(v[i].x * f, v[i].y * f, hi, lo);
        *reinterpret_cast<__half2 *>(to + 64 * i + 2 * lane) = hi;
        *reinterpret_cast<__half2 *>(to + apart + 64 * i + 2 * lane) = lo;
    }
    return e;
}

template <int DKQ, int DV, bool VK>
__global__ void __launch_bounds__(32 * F32T<DKQ, DV, VK>::kWarps, DV == 512 ? 1 : 2) chunk_f32_tree_kernel(const Params p) {
    using L = F32T<DKQ, DV, VK>;
    constexpr int TK = L::kTK, WG = L::kWG, LR = L::kLR, PQ = L::kPQ, PV = VK ? L::kPQ : L::kPV, PS = L::kPS, BW = L::kBW, MW = L::kMW;
    constexpr int NQ = DKQ / 64, NV = DV / 64, RW = TK / L::kWarps;   // a lane's pairs of a row; a warp's rows of a tile
    extern __shared__ __align__(16) uint8_t smem[];
    __half *sQ = reinterpret_cast<__half *>(smem), *sK = reinterpret_cast<__half *>(smem + L::kOffK);
    __half *sV = VK ? sK : reinterpret_cast<__half *>(smem + L::kOffV), *sP = reinterpret_cast<__half *>(smem + L::kOffP);
    int64_t *sCells = reinterpret_cast<int64_t *>(smem + L::kOffCell);
    float2 *sUk = reinterpret_cast<float2 *>(smem + L::kOffUnit), *sUv = VK ? sUk : sUk + TK;
    int *sEq = reinterpret_cast<int *>(smem + L::kOffRow);
    float *sS = reinterpret_cast<float *>(smem + L::kOffS), *sAlpha = reinterpret_cast<float *>(smem + L::kOffAlpha);
    int *sOddQ = reinterpret_cast<int *>(smem + L::kOffOdd),
        *sOdd = sOddQ + kF32Rows;
    __shared__ Item s_item;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, fr = lane >> 2, fc = lane & 3;
    const int split = blockIdx.z, g = blockIdx.y;
    const float *Qg = reinterpret_cast<const float *>(p.Q), *Kg = reinterpret_cast<const float *>(p.K),
                *Vg = reinterpret_cast<const float *>(VK ? p.K : p.V);
    constexpr int DVR = VK ? DKQ : DV;   // elements of a value row in memory
    pdl_wait();
    if (warp == 0) {
        const Item it = find_item(p, blockIdx.x, g == 0 && split == 0);
        if (lane == 0) s_item = it;
    }
    __syncthreads();
    const Item it = s_item;
    if (it.seq < 0) return;
    const int r0 = it.tile * kF32Rows;                     // first flattened row
    const int n = min(it.q.n, p.n_new_max);
    const int rows = min(kF32Rows, (int)((int64_t)n * p.G - r0));
    const int cached = it.q.total - it.q.n;
    const int len = list_end(p, it.q, 0), begin = list_begin(p, it.q, len);
    int k0, k1;
    piece_keys(p, blockIdx.x, g, split, begin, len, k0, k1);
    const bool whole = one_piece(p, blockIdx.x, g, len - begin);
    if (split > 0 && k0 >= k1) return;                     // no such piece
    auto row_of = [&](int row) {
        return (int64_t)(it.q.c0 + (r0 + row) / p.G) * p.h_q + g * p.G + (r0 + row) % p.G;
    };

    // a warp's rows of the tile of keys t0 .., on their way
    float2 kreg[RW][NQ], vreg[VK ? 1 : RW][NV];
    int entry = 0;   // the page of one of them, looked up a tile ahead
    auto look_up = [&](int t0) {
        const int t = t0 + warp * RW + lane % RW;
        if (t < k1) entry = __ldg(p.table + (int64_t)it.seq * p.table_stride + p.page_div.div(t));
    };
    auto fetch = [&](int t0, int64_t *cells) {
        const int t = t0 + warp * RW + lane % RW;
        const bool page = entry >= 0 && entry < p.n_pages;
        if (t < k1 && !page) set_status(p.status, SFA_DEV_BAD_CELL);
        const int64_t mine = t < k1 && page ? (int64_t)entry * p.page + (t - p.page_div.div(t) * p.page) : -1;
        if (lane < RW) cells[warp * RW + lane] = mine;
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            const int64_t cell = RW == 1 ? mine : __shfl_sync(0xFFFFFFFFu, mine, i);
            const int64_t row = cell * p.h_kv + g;
#pragma unroll
            for (int x = 0; x < NQ; ++x)
                kreg[i][x] = cell >= 0 ? __ldg(reinterpret_cast<const float2 *>(Kg + row * DKQ + 64 * x + 2 * lane))
                                       : make_float2(0.f, 0.f);
            if constexpr (!VK) {
#pragma unroll
                for (int x = 0; x < NV; ++x)
                    vreg[i][x] = cell >= 0 ? __ldg(reinterpret_cast<const float2 *>(Vg + row * DV + 64 * x + 2 * lane))
                                           : make_float2(0.f, 0.f);
            }
        }
    };
    auto put = [&]() {
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            const int key = warp * RW + i;
            bool odd_k, odd_v;
            const int e = put_row<NQ>(kreg[i], sK + key * PQ, TK * PQ, odd_k);
            int sv = e;
            odd_v = odd_k;   // V = K: perhaps of dims behind the values only
            if constexpr (!VK) sv = put_row<NV>(vreg[i], sV + key * PV, TK * PV, odd_v);
            if (lane == 0) {
                sUk[key] = pow2_halves(-e);
                if constexpr (!VK) sUv[key] = pow2_halves(-sv);
                sOdd[key] = (odd_k ? 1 : 0) | (odd_v ? 2 : 0);
            }
        }
    };
    const int n_tiles = (k1 - k0 + TK - 1) / TK;
    if (n_tiles > 0) {
        look_up(k0);
        fetch(k0, sCells);
        look_up(k0 + TK);
    }
#pragma unroll 1
    for (int row = warp; row < kF32Rows; row += L::kWarps) {   // queries
        float2 v[NQ];
#pragma unroll
        for (int x = 0; x < NQ; ++x)
            v[x] = row < rows ? *reinterpret_cast<const float2 *>(Qg + row_of(row) * DKQ + 64 * x + 2 * lane) : make_float2(0.f, 0.f);
        bool odd;
        const int e = put_row<NQ>(v, sQ + row * PQ, kF32Rows * PQ, odd);
        if (lane == 0) {
            sEq[row] = e;
            sOddQ[row] = odd;
        }
    }
    const int rg = warp / WG, wg = warp % WG;   // scores: rows 16 rg ..; keys k8 .., dims from 16 first on
    const int k8 = 16 * (wg / L::kParts), part = wg % L::kParts, first = part * (DKQ / 16 / L::kParts);
    const int row = 16 * rg + wg * (32 / LR) + lane / LR, x0 = 2 * (lane % LR);   // softmax: keys x0 + 2 LR i, + 1
    const uint32_t *mask = row < rows ? p.mask + (int64_t)(it.q.c0 + (r0 + row) / p.G) * p.mask_words : nullptr;
    float m = -INFINITY, l = 0.f;   // of that row, base 2; l of this lane's keys
    int u = -1000;                  // and the power of two of its sums of values
    // values: blocks BW bw .. of row tiles MW mw ..
    const int bw = warp % (L::kBlocks / BW), mw = warp / (L::kBlocks / BW);
    float acc[BW][MW][4][4];
#pragma unroll
    for (int b = 0; b < BW; ++b)
#pragma unroll
        for (int x = 0; x < MW; ++x)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[b][x][i][c] = 0.f;

    for (int t = 0; t < n_tiles; ++t) {
        const int t0 = k0 + t * TK;
        __syncthreads();   // the tile before is done with
        put();
        if (t + 1 < n_tiles) {
            fetch(t0 + TK, sCells + ((t + 1) & 1) * TK);
            look_up(t0 + 2 * TK);
        }
        __syncthreads();
        // the tile's keys that are, and that have odd values
        const int64_t *sCell = sCells + (t & 1) * TK;
        const unsigned live = __ballot_sync(0xFFFFFFFFu, sCell[lane % TK] >= 0);
        const int o = sOdd[lane % TK];
        const unsigned odd_k = __ballot_sync(0xFFFFFFFFu, o & 1), odd_v = __ballot_sync(0xFFFFFFFFu, lane < TK && (o & 2));
        if (16 * rg < rows) {
            float d[2][2][4] = {};   // the small products' sum and the large one's
            const uint32_t qa = smem_u32(sQ + (16 * rg + (lane & 15)) * PQ + 8 * (lane >> 4) + 16 * first);
            const uint32_t ka = smem_u32(sK + (k8 + (lane & 7) + 8 * (lane >> 4)) * PQ + 8 * ((lane >> 3) & 1) + 16 * first);
#pragma unroll(L::kParts == 1 ? 2 : 1)
            for (int i = 0; i < DKQ / 16 / L::kParts; ++i) {
                uint32_t Ah[4], Al[4], Bh[4], Bl[4];
                ldsm_x4(ka + 32 * i, Bh[0], Bh[1], Bh[2], Bh[3]);
                ldsm_x4(qa + kF32Rows * PQ * 2 + 32 * i, Al[0], Al[1], Al[2], Al[3]);
                ldsm_x4(qa + 32 * i, Ah[0], Ah[1], Ah[2], Ah[3]);
                ldsm_x4(ka + TK * PQ * 2 + 32 * i, Bl[0], Bl[1], Bl[2], Bl[3]);
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    mma_f16_16816(d[nt][0], Al, Bh[2 * nt], Bh[2 * nt + 1]);
                    mma_f16_16816(d[nt][1], Ah, Bh[2 * nt], Bh[2 * nt + 1]);
                    mma_f16_16816(d[nt][0], Ah, Bl[2 * nt], Bl[2 * nt + 1]);
                }
            }
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int x = 2 * y;
                    *reinterpret_cast<float2 *>(sS + (part * kF32Rows + 16 * rg + fr + 8 * y) * PS + k8 + 8 * nt + 2 * fc) =
                        make_float2(d[nt][1][x] + d[nt][0][x], d[nt][1][x + 1] + d[nt][0][x + 1]);
                }
        }
        named_barrier(1 + rg, 32 * WG);   // the warps of these rows
        if (16 * rg < rows) {
            constexpr int KL = TK / LR;   // keys of a lane
            const uint32_t node = live & tree_bits(p, mask, cached, t0);
            const float2 uq = pow2_halves(-sEq[row]);
            const bool odd_q = sOddQ[row] != 0;
            float s[KL], mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < KL; i += 2) {
                float2 v = *reinterpret_cast<const float2 *>(sS + row * PS + x0 + LR * i);
#pragma unroll
                for (int j = 1; j < L::kParts; ++j) {
                    const float2 w = *reinterpret_cast<const float2 *>(sS + (j * kF32Rows + row) * PS + x0 + LR * i);
                    v.x += w.x;
                    v.y += w.y;
                }
                s[i] = v.x;
                s[i + 1] = v.y;
            }
#pragma unroll
            for (int i = 0; i < KL; ++i) {
                const int key = x0 + LR * (i & ~1) + (i & 1);
                const bool on = (node >> key) & 1;
                const float2 uk = sUk[key];
                float x = s[i] * uk.x * uq.x * uk.y * uq.y;
                if (on && (odd_q || ((odd_k >> key) & 1)) && row < rows) {   // the plain product
                    const float *q = Qg + row_of(row) * DKQ, *k = Kg + (sCell[key] * p.h_kv + g) * DKQ;
                    x = 0.f;
                    for (int j = 0; j < DKQ; ++j) x = fmaf(q[j], k[j], x);
                }
                s[i] = on ? x * p.scale_log2 : -INFINITY;
                mx = fmaxf(mx, s[i]);
            }
#pragma unroll
            for (int o = LR / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
            const float mn = mx > m + 8.f ? mx : m, base = mn == -INFINITY ? 0.f : mn;
            const float dm = m == -INFINITY || mn == m ? 0.f : m - mn;
            const int whole_dm = (int)floorf(fmaxf(dm, -300.f));
            unsigned odd_on = 0;
            if (odd_v & node) {
#pragma unroll
                for (int i = 0; i < KL; ++i)
                    odd_on |= s[i] != -INFINITY ? odd_v & (1u << (x0 + LR * (i & ~1) + (i & 1))) : 0u;
            }
            float sum = 0.f, w[KL], large = 0.f;   // the weights of the values as they were, the largest
#pragma unroll
            for (int i = 0; i < KL; ++i) {
                const float2 uv = sUv[x0 + LR * (i & ~1) + (i & 1)];
                const float e = ex2(s[i] - base);
                sum += e;
                w[i] = e * uv.x * uv.y;
                large = fmaxf(large, w[i]);
            }
#pragma unroll
            for (int o = LR / 2; o > 0; o >>= 1) large = fmaxf(large, __shfl_xor_sync(0xFFFFFFFFu, large, o));
            const int top = large > 0.f ? (int)(__float_as_uint(large) >> 23) - 126 : -2000, u0 = u + whole_dm;
            u = top > u0 + 4 ? top : u0;
            const float2 uw = pow2_halves(min(kTop - u, 252));
#pragma unroll
            for (int i = 0; i < KL; i += 2) {
                const int key = x0 + LR * i;
                float e[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    e[c] = w[i + c] * uw.x * uw.y;
                    // a value that is not finite counts by any weight (its finite ones are off by 2^-34 at most)
                    if ((odd_on >> (key + c)) & 1) e[c] = fmaxf(e[c], 0x1p-24f);
                }
                __half2 hi, lo;
                split_f16(e[0], e[1], hi, lo);
                *reinterpret_cast<__half2 *>(sP + row * PS + key) = hi;
                *reinterpret_cast<__half2 *>(sP + (kF32Rows + row) * PS + key) = lo;
            }
            m = mn;
            l = l * exp2f(dm) + sum;
            if (lane % LR == 0) sAlpha[row] = exp2f(dm - whole_dm) * pow2(u0 - u);
        }
        __syncthreads();
#pragma unroll
        for (int x = 0; x < MW; ++x) {
            if (16 * (MW * mw + x) >= rows) break;   // row tiles without rows
            const float al0 = sAlpha[16 * (MW * mw + x) + fr], al1 = sAlpha[16 * (MW * mw + x) + fr + 8];
            if (__any_sync(0xFFFFFFFFu, al0 != 1.f || al1 != 1.f)) {
#pragma unroll
                for (int b = 0; b < BW; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        acc[b][x][i][0] *= al0;
                        acc[b][x][i][1] *= al0;
                        acc[b][x][i][2] *= al1;
                        acc[b][x][i][3] *= al1;
                    }
            }
        }
#pragma unroll
        for (int ks = 0; ks < TK / 16; ++ks)
#pragma unroll
            for (int b = 0; b < BW; ++b) {
                const int d0 = 32 * (BW * bw + b);
                uint32_t hi[4][2], lo[4][2];   // of dims d0 + 8 i ..
                const uint32_t va = smem_u32(sV + (16 * ks + (lane & 15)) * PV + d0 + 8 * (lane >> 4));
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    ldsm_x4_t(va + 16 * i, hi[i][0], hi[i][1], hi[i + 1][0], hi[i + 1][1]);
                    ldsm_x4_t(va + TK * PV * 2 + 16 * i, lo[i][0], lo[i][1], lo[i + 1][0], lo[i + 1][1]);
                }
#pragma unroll
                for (int x = 0; x < MW; ++x) {
                    if (16 * (MW * mw + x) >= rows) break;
                    uint32_t ph[4], pl[4];
                    const uint32_t pa = smem_u32(sP + (16 * (MW * mw + x) + (lane & 15)) * PS + 16 * ks + 8 * (lane >> 4));
                    ldsm_x4(pa, ph[0], ph[1], ph[2], ph[3]);
                    ldsm_x4(pa + kF32Rows * PS * 2, pl[0], pl[1], pl[2], pl[3]);
                    // the tensor cores cut what they add to an accumulator towards zero: not to acc
                    float d[4][4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) mma_f16_zero(d[i], pl, hi[i][0], hi[i][1]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) mma_f16_16816(d[i], ph, lo[i][0], lo[i][1]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) mma_f16_16816(d[i], ph, hi[i][0], hi[i][1]);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int c = 0; c < 4; ++c) acc[b][x][i][c] += d[i][c];
                }
            }
        for (unsigned w = odd_v; w; w &= w - 1) {   // values that are not finite, to the rows that attend them
            const int key = __ffs(w) - 1;
            const float *v = Vg + (sCell[key] * p.h_kv + g) * DVR;
#pragma unroll
            for (int b = 0; b < BW; ++b)
#pragma unroll
                for (int x = 0; x < MW; ++x)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const float e = __half2float(sP[(16 * (MW * mw + x) + fr + 8 * (c >> 1)) * PS + key]);
                            const float y = v[32 * (BW * bw + b) + 8 * i + 2 * fc + (c & 1)];
                            if (!finite(y) && e != 0.f) acc[b][x][i][c] += y;
                        }
        }
    }
    // ------------------------------------------------------------------------------------ result
    __syncthreads();   // sAlpha is read
    const int64_t part0 = (int64_t)piece_part(p, blockIdx.x, g, split) * p.part_rows;
#pragma unroll
    for (int o = LR / 2; o > 0; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
    if (lane % LR == 0 && row < rows) {
        const bool any = l > 0.f || l != l;
        sAlpha[row] = whole ? (any ? 1.f / l : 0.f) : 1.f;
        sEq[row] = u - kTop;
        if (!whole) {
            p.part_ml[(part0 + row) * 2] = m;
            p.part_ml[(part0 + row) * 2 + 1] = l;
        } else if (p.lse) {
            p.lse[row_of(row)] = any ? (m + log2f(l)) / kLog2e : -INFINITY;
        }
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < MW; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const int row = 16 * (MW * mw + x) + fr + 8 * y;
            if (row >= rows) continue;
            const float inv = sAlpha[row];
            const int unit = sEq[row];
#pragma unroll
            for (int b = 0; b < BW; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int d = 32 * (BW * bw + b) + 8 * i + 2 * fc;
                    const float u = ldexpf(acc[b][x][i][2 * y] * inv, unit), v = ldexpf(acc[b][x][i][2 * y + 1] * inv, unit);
                    if (whole && p.o_bf16)
                        *reinterpret_cast<uint32_t *>(reinterpret_cast<__nv_bfloat16 *>(p.O) + row_of(row) * DV + d) = pack_bf16(u, v);
                    else
                        *reinterpret_cast<float2 *>(whole ? reinterpret_cast<float *>(p.O) + row_of(row) * DV + d
                                                          : p.part_o + (part0 + row) * DV + d) = make_float2(u, v);
                }
        }
}

template <int DKQ, int DV, bool VK>
int launch(const Params &p, cudaStream_t st) {
    if (!ensure_max_dynamic_smem(chunk_f32_tree_kernel<DKQ, DV, VK>)) return SFA_ERR_CUDA;
    if (launch_pdl(chunk_f32_tree_kernel<DKQ, DV, VK>, dim3(p.items, p.h_kv, p.n_split), dim3(32 * F32T<DKQ, DV, VK>::kWarps),
                   (size_t)F32T<DKQ, DV, VK>::kBytes, st, p) != cudaSuccess) {
        cudaGetLastError();
        return SFA_ERR_CUDA;
    }
    return SFA_OK;
}

}  // namespace

int launch_f32_tree(const Params &p, int dkq, cudaStream_t st) {
    switch (dkq) {
        case 576: return launch<576, 512, true>(p, st);
        case 512: return p.V ? launch<512, 512, false>(p, st) : launch<512, 512, true>(p, st);
        case 128: return p.V ? launch<128, 128, false>(p, st) : launch<128, 128, true>(p, st);
        default: return p.V ? launch<64, 64, false>(p, st) : launch<64, 64, true>(p, st);
    }
}

}  // namespace chunk
}  // namespace sfa
