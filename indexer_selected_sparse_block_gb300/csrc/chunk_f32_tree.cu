// chunk_f32_tree.cu -- attention of drafted trees over fp32 caches.
//
// Both products run on binary16 operands (mma.sync, twice tf32's rate for each of its steps): a row is brought
// to a largest value of 2^10 .. 2^11 by a power of two and cut in hi + lo of 11 bits each, which leaves 2^-22 of a
// value (2^-35 of the row's largest at least), and of the four products the three larger ones are taken.
//   scores: the rows' powers of two come back with the scale;
//   values: a key's power goes into its weight, relative to the smallest one so far (S: the largest values),
//           so that sum_k (p_k 2^(S - sv_k)) (2^sv_k v_k) = 2^S sum_k p_k v_k.
// A row is read, scaled and cut once for all 64 rows (query, head) of the CTA's tile; the next tile's rows are on
// their way to registers meanwhile.  Scores: a warp has 16 rows and half the tile's keys.  Values: a warp has 64
// dims of all rows (narrow heads: 32 dims of 32 or 16 rows), sixteen keys' sum is added with rounding.
// Values that are not finite are taken out of the operands: a score with one is a plain product instead, and such
// values are added one by one to the rows that attend them.
// XXX
#include "chunk_common.cuh"

namespace sfa {
namespace chunk {
namespace {

constexpr int kThreads = 256;
constexpr int kTop = 10;   // the exponent of a scaled row's largest value

template <int DKQ, int DV, bool VK>
struct F32T {
    static constexpr int kTK = DV == 512 ? 16 : 32, kNT = kTK / 16;   // keys of a tile; a warp's score tiles of 8 keys
    static constexpr int kPQ = DKQ + 8, kPV = DV + 8, kPS = kTK + 8;  // pitches: ldmatrix without bank conflicts
    static constexpr int kOffK = 2 * kF32Rows * kPQ * 2;              // hi, lo of the queries before
    static constexpr int kOffV = kOffK + 2 * kTK * kPQ * 2;
    static constexpr int kOffP = kOffV + (VK ? 0 : 2 * kTK * kPV * 2);
    static constexpr int kOffCell = kOffP + 2 * kF32Rows * kPS * 2;   // int64 [kTK]
    static constexpr int kOffUnit = kOffCell + kTK * 8;               // int: rows' and keys' powers of two
    static constexpr int kOffMax = kOffUnit + (kF32Rows + kTK) * 4;   // float [2][64]
    static constexpr int kOffAlpha = kOffMax + 2 * kF32Rows * 4;
    static constexpr int kOffSv = kOffAlpha + kF32Rows * 4;           // int [kTK]
    static constexpr int kOffOdd = kOffSv + kTK * 4;                  // int [64] of queries, [kTK]: 1 key, 2 value
    static constexpr int kOffSwap = (kOffOdd + (kF32Rows + kTK) * 4 + 15) / 16 * 16;   // float4 [8][32]: scores of halves
    static constexpr int kBytes = kOffSwap + (kNT == 1 ? 8 * 32 * 16 : 0);
    static_assert(kNT == 1 || kNT == 2, "two warps' score tiles: 16 or 32 keys");
    static constexpr int kBlocks = DV / 32, kBW = kBlocks >= 8 ? kBlocks / 8 : 1, kMW = kBlocks >= 8 ? 4 : kBlocks / 2;
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
    float top = 0.f;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (!finite(v[i].x)) {
            v[i].x = 0.f;
            bad = true;
        }
        if (!finite(v[i].y)) {
            v[i].y = 0.f;
            bad = true;
        }
        top = fmaxf(top, fmaxf(fabsf(v[i].x), fabsf(v[i].y)));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    odd = __any_sync(0xFFFFFFFFu, bad);
    const int e = min(126, kTop - ((int)(__float_as_uint(top) >> 23) - 127));   // a row of zeros: 126
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
__global__ void __launch_bounds__(kThreads, DV == 512 ? 1 : 2) chunk_f32_tree_kernel(const Params p) {
    using L = F32T<DKQ, DV, VK>;
    constexpr int TK = L::kTK, NT = L::kNT, PQ = L::kPQ, PV = VK ? L::kPQ : L::kPV, PS = L::kPS, BW = L::kBW, MW = L::kMW;
    constexpr int NQ = DKQ / 64, NV = DV / 64, RW = TK / 8;   // a lane's pairs of a row; a warp's rows of a tile
    extern __shared__ __align__(16) uint8_t smem[];
    __half *sQ = reinterpret_cast<__half *>(smem), *sK = reinterpret_cast<__half *>(smem + L::kOffK);
    __half *sV = VK ? sK : reinterpret_cast<__half *>(smem + L::kOffV), *sP = reinterpret_cast<__half *>(smem + L::kOffP);
    int64_t *sCell = reinterpret_cast<int64_t *>(smem + L::kOffCell);
    int *sEq = reinterpret_cast<int *>(smem + L::kOffUnit), *sEk = sEq + kF32Rows;
    float *sMax = reinterpret_cast<float *>(smem + L::kOffMax), *sAlpha = reinterpret_cast<float *>(smem + L::kOffAlpha);
    int *sSv = reinterpret_cast<int *>(smem + L::kOffSv), *sOddQ = reinterpret_cast<int *>(smem + L::kOffOdd),
        *sOdd = sOddQ + kF32Rows;
    float4 *sSwap = reinterpret_cast<float4 *>(smem + L::kOffSwap);
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
    int64_t cells[RW];
    auto fetch = [&](int t0) {
        const int t = t0 + warp * RW + lane % RW;
        const int64_t mine = t < k1 ? cell_of(p, it.seq, t) : -1;
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            cells[i] = __shfl_sync(0xFFFFFFFFu, mine, i);
            const int64_t row = cells[i] * p.h_kv + g;
#pragma unroll
            for (int x = 0; x < NQ; ++x)
                kreg[i][x] = cells[i] >= 0 ? __ldg(reinterpret_cast<const float2 *>(Kg + row * DKQ + 64 * x + 2 * lane))
                                           : make_float2(0.f, 0.f);
            if constexpr (!VK) {
#pragma unroll
                for (int x = 0; x < NV; ++x)
                    vreg[i][x] = cells[i] >= 0 ? __ldg(reinterpret_cast<const float2 *>(Vg + row * DV + 64 * x + 2 * lane))
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
                sCell[key] = cells[i];
                sEk[key] = e;
                sSv[key] = sv;
                sOdd[key] = (odd_k ? 1 : 0) | (odd_v ? 2 : 0);
            }
        }
    };
    const int n_tiles = (k1 - k0 + TK - 1) / TK;
    if (n_tiles > 0) fetch(k0);
    for (int i = 0; i < kF32Rows / 8; ++i) {   // queries: a warp has eight rows
        const int row = warp * (kF32Rows / 8) + i;
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
    const int rg = warp >> 1, kh = warp & 1, key0 = 8 * NT * kh;   // scores: rows 16 rg .., keys key0 ..
    const uint32_t *mask[2];
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};   // rows 16 rg + fr and 8 more, base 2; l of this lane's keys
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        const int row = 16 * rg + fr + 8 * y;
        mask[y] = row < rows ? p.mask + (int64_t)(it.q.c0 + (r0 + row) / p.G) * p.mask_words : nullptr;
    }
    // values: blocks BW bw .. of row tiles MW mw ..
    const int bw = L::kBlocks >= 8 ? warp : warp % L::kBlocks, mw = L::kBlocks >= 8 ? 0 : warp / L::kBlocks;
    float acc[BW][MW][4][4];
#pragma unroll
    for (int b = 0; b < BW; ++b)
#pragma unroll
        for (int x = 0; x < MW; ++x)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[b][x][i][c] = 0.f;
    int S = 127;   // the values' power of two so far

    for (int t = 0; t < n_tiles; ++t) {
        const int t0 = k0 + t * TK;
        __syncthreads();   // the tile before is done with
        put();
        if (t + 1 < n_tiles) fetch(t0 + TK);
        __syncthreads();
        float s[NT][4];   // keys key0 + 8 nt + 2 fc, + 1 of both rows
        {
            constexpr int W = 2 / NT;   // warps a sum: halves of the dims, of both tiles of keys, or one warp
            constexpr int kSteps = DKQ / 16 / W;
            float d[2][3][4] = {};   // a sum for each product: chains of their own
            const int first = W == 2 ? kh * kSteps : 0, k8 = W == 2 ? 0 : key0;
            const uint32_t qa = smem_u32(sQ + (16 * rg + (lane & 15)) * PQ + 8 * (lane >> 4) + 16 * first);
            const uint32_t ka = smem_u32(sK + (k8 + (lane & 7) + 8 * (lane >> 4)) * PQ + 8 * ((lane >> 3) & 1) + 16 * first);
#pragma unroll 2
            for (int i = 0; i < (16 * rg < rows ? kSteps : 0); ++i) {
                uint32_t Ah[4], Al[4], Bh[4], Bl[4];
                ldsm_x4(ka + 32 * i, Bh[0], Bh[1], Bh[2], Bh[3]);
                ldsm_x4(qa + kF32Rows * PQ * 2 + 32 * i, Al[0], Al[1], Al[2], Al[3]);
                ldsm_x4(qa + 32 * i, Ah[0], Ah[1], Ah[2], Ah[3]);
                ldsm_x4(ka + TK * PQ * 2 + 32 * i, Bl[0], Bl[1], Bl[2], Bl[3]);
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    mma_f16_16816(d[nt][0], Al, Bh[2 * nt], Bh[2 * nt + 1]);
                    mma_f16_16816(d[nt][2], Ah, Bh[2 * nt], Bh[2 * nt + 1]);
                    mma_f16_16816(d[nt][1], Ah, Bl[2 * nt], Bl[2 * nt + 1]);
                }
            }
            float sum[2][4];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int x = 0; x < 4; ++x) sum[nt][x] = d[nt][2][x] + (d[nt][0][x] + d[nt][1][x]);
            if constexpr (W == 2) {   // a warp keeps the tile kh and gives the other
                float4 *swap = sSwap + (rg * 2 + kh) * 32 + lane;
                *swap = kh ? make_float4(sum[0][0], sum[0][1], sum[0][2], sum[0][3])
                           : make_float4(sum[1][0], sum[1][1], sum[1][2], sum[1][3]);
                named_barrier(1 + rg, 64);
                const float4 o = sSwap[(rg * 2 + (kh ^ 1)) * 32 + lane];
#pragma unroll
                for (int x = 0; x < 4; ++x) s[0][x] = kh ? sum[1][x] : sum[0][x];
                s[0][0] += o.x;
                s[0][1] += o.y;
                s[0][2] += o.z;
                s[0][3] += o.w;
            } else {
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                    for (int x = 0; x < 4; ++x) s[nt][x] = sum[nt][x];
            }
        }
        float mx[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const int row = 16 * rg + fr + 8 * y;
            const uint32_t node = tree_bits(p, mask[y], cached, t0);
            const int eq = sEq[row];
            const bool odd_q = sOddQ[row] != 0;
            mx[y] = -INFINITY;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int key = key0 + 8 * nt + 2 * fc + c;
                    float &x = s[nt][2 * y + c];
                    const bool on = sCell[key] >= 0 && ((node >> key) & 1);
                    const int e = -eq - sEk[key];   // in two steps: either may be out of range
                    x = x * pow2(e >> 1) * pow2(e - (e >> 1));
                    if (on && (odd_q || (sOdd[key] & 1)) && row < rows) {   // the plain product
                        const float *q = Qg + row_of(row) * DKQ, *k = Kg + (sCell[key] * p.h_kv + g) * DKQ;
                        x = 0.f;
                        for (int i = 0; i < DKQ; ++i) x = fmaf(q[i], k[i], x);
                    }
                    x = on ? x * p.scale_log2 : -INFINITY;
                    mx[y] = fmaxf(mx[y], x);
                }
            mx[y] = fmaxf(mx[y], __shfl_xor_sync(0xFFFFFFFFu, mx[y], 1));
            mx[y] = fmaxf(mx[y], __shfl_xor_sync(0xFFFFFFFFu, mx[y], 2));
            if (fc == 0) sMax[kh * kF32Rows + row] = mx[y];
        }
        // the tile's smallest power of two, and whether it has odd values: the same in every warp
        int low = sSv[lane % TK];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) low = min(low, __shfl_xor_sync(0xFFFFFFFFu, low, o));
        const unsigned odd_v = __ballot_sync(0xFFFFFFFFu, lane < TK && (sOdd[lane % TK] & 2));
        const int S1 = min(S, low);
        const float down = t == 0 ? 1.f : pow2(S1 - S);
        S = S1;
        named_barrier(1 + rg, 64);   // the two warps of these rows
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const int row = 16 * rg + fr + 8 * y;
            const float mn = fmaxf(m[y], fmaxf(mx[y], sMax[(kh ^ 1) * kF32Rows + row]));
            const float al = m[y] == -INFINITY ? (mn == -INFINITY ? 1.f : 0.f) : exp2f(m[y] - mn);
            float sum = 0.f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int key = key0 + 8 * nt + 2 * fc;
                float e[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float x = s[nt][2 * y + c];
                    e[c] = x == -INFINITY ? 0.f : exp2f(x - mn);
                    sum += e[c];
                    e[c] *= pow2(S - sSv[key + c] + kTop);
                    // a value that is not finite counts by any weight (its finite ones are off by 2^-34 at most)
                    if ((odd_v >> (key + c)) & 1 && x != -INFINITY) e[c] = fmaxf(e[c], 0x1p-24f);
                }
                __half2 hi, lo;
                split_f16(e[0], e[1], hi, lo);
                *reinterpret_cast<__half2 *>(sP + row * PS + key) = hi;
                *reinterpret_cast<__half2 *>(sP + (kF32Rows + row) * PS + key) = lo;
            }
            m[y] = mn;
            l[y] = l[y] * al + sum;
            if (kh == 0 && fc == 0) sAlpha[row] = al * down;
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
    __syncthreads();   // sMax and sAlpha are read
    const int64_t part0 = (int64_t)piece_part(p, blockIdx.x, g, split) * p.part_rows;
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        l[y] += __shfl_xor_sync(0xFFFFFFFFu, l[y], 1);
        l[y] += __shfl_xor_sync(0xFFFFFFFFu, l[y], 2);
        if (fc == 0) sMax[kh * kF32Rows + 16 * rg + fr + 8 * y] = l[y];
    }
    named_barrier(1 + rg, 64);
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        const int row = 16 * rg + fr + 8 * y;
        const float sum = sMax[row] + sMax[kF32Rows + row];
        const bool any = sum > 0.f || sum != sum;
        if (kh == 0 && fc == 0) {
            sAlpha[row] = whole ? (any ? 1.f / sum : 0.f) : 1.f;
            if (row < rows) {
                if (!whole) {
                    p.part_ml[(part0 + row) * 2] = m[y];
                    p.part_ml[(part0 + row) * 2 + 1] = sum;
                } else if (p.lse) {
                    p.lse[row_of(row)] = any ? (m[y] + log2f(sum)) / kLog2e : -INFINITY;
                }
            }
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
#pragma unroll
            for (int b = 0; b < BW; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int d = 32 * (BW * bw + b) + 8 * i + 2 * fc;
                    const float u = ldexpf(acc[b][x][i][2 * y] * inv, -S - kTop), v = ldexpf(acc[b][x][i][2 * y + 1] * inv, -S - kTop);
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
    if (launch_pdl(chunk_f32_tree_kernel<DKQ, DV, VK>, dim3(p.items, p.h_kv, p.n_split), dim3(kThreads),
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
