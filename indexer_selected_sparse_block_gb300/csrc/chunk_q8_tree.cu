// chunk_q8_tree.cu -- attention of drafted trees over q8_0 caches.
//
// An element of a q8_0 row is scale * code, one scale (binary16) a block of 32.  The codes are exact in
// binary16 and bf16, so the products run on them as they are and the scales come in around the products:
//   s_ik  = sum_b scale_kb (sum_{j in b} q_ij code_kj)   a block's sum, two m16n8k16 steps, then one fp32
//           multiply-add: exact products, fp32 sums;
//   o_id += sum_k p_ik (scale_kb code_kd)                weights and values as two bf16 parts each (2^-17), the
//           three larger products of the four; a lane expands the values where it needs them, in registers.
// bf16 queries are binary16 times a power of two of their row, its largest value brought to 2^14 .. 2^15: exact down
// to 2^-17, which is 2^-31 of the row's largest at most; a smaller value is off by 2^-25, 2^-39 of the largest.  No
// value is ever expanded in memory: a tile is its raw rows.
//
// One CTA: 64 rows (query, head) of one KV head against 32 keys at a time, three tiles of raw rows by
// asynchronous copies.  Scores: a warp has 16 rows and 16 keys.  Values: a warp has 64 dims of all rows (narrow
// heads: 32 dims of 32 or 16 rows).  The dims of a lane's operands are eight (four) neighbours of a block: any
// order does for the contraction, and a lane's results are eight neighbouring dims.
// 2 trees of 13 nodes behind 34715, 576 wide, 16 heads: 342 us, 92 TFLOP/s of the rows alone (1091 by three tf32
// products on rows expanded in shared memory).  It is bound by instructions and the latency of short chains, on
// eight warps with all registers: schedulers issue half the time, mma.sync is a third of its 600 TFLOP/s.  With 16
// warps of half the value dims, scores by halves of the dims and a row's softmax in one warp 361; 39 trees of 19
// behind 786, 512 wide: 290, 297; 27 of 104 behind 54: 397, 377.
// Row tiles without rows are left out (128 wide, 1 tree of 3 behind 126486, 16 heads on 16: 554 us, 688 with them),
// of wide heads' the last two at once: a test for each costs full tiles 4%.
#include "chunk_common.cuh"

namespace sfa {
namespace chunk {
namespace {

constexpr int kThreads = 256, kKeys = 32, kBufs = 3;
constexpr int kPS = kKeys + 8;   // pitch of the weights' rows, in bf16: 16-byte rows without bank conflicts
// Pitch of a raw row in shared memory: four rows' 32 bytes, a quarter of the bank line each.
constexpr int raw_pitch(int bytes) { return bytes % 128 == 32 || bytes % 128 == 96 ? bytes : raw_pitch(bytes + 16); }
// Where key k of sixteen stands in the contraction with the values: lane fc has those of 2 fc, 2 fc + 1, 2 fc + 8
// and 2 fc + 9, which are the keys fc, fc + 4, fc + 8 and fc + 12.
__device__ __forceinline__ int key_slot(int k) { return 2 * (k & 3) + ((k >> 2) & 1) + 8 * (k >> 3); }

template <int DKQ, int DV, bool VK>
struct Q8 {
    static constexpr int kRK = q8_row_bytes(DKQ), kRV = q8_row_bytes(DV);
    static constexpr int kPK = raw_pitch(kRK), kPV = VK ? kPK : raw_pitch(kRV);
    static constexpr int kPQ = DKQ + 32;                              // pitch of the queries' rows
    static constexpr int kOffK = kQ8Rows * kPQ * 2;
    static constexpr int kOffV = kOffK + kBufs * kKeys * kPK;
    static constexpr int kOffP = kOffV + (VK ? 0 : kBufs * kKeys * kPV);   // bf16 [2][64][kPS]
    static constexpr int kOffOk = kOffP + 2 * kQ8Rows * kPS * 2;       // int [kBufs][kKeys]: the key has a cell
    static constexpr int kOffMax = kOffOk + kBufs * kKeys * 4;        // float [2][64]
    static constexpr int kOffAlpha = kOffMax + 2 * kQ8Rows * 4;
    static constexpr int kOffUnit = kOffAlpha + kQ8Rows * 4;           // a row's scores' unit
    static constexpr int kBytes = kOffUnit + kQ8Rows * 4;
    // value dims: blocks of 32 and row tiles of 16 a warp
    static constexpr int kBlocks = DV / 32, kBW = kBlocks >= 8 ? kBlocks / 8 : 1, kMW = kBlocks >= 8 ? 4 : kBlocks / 2;
};

// Four codes to two pairs of binary16: the bytes 128 + code become 1152 + code.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t &a, uint32_t &b) {
    w ^= 0x80808080u;
    const __half2 off = __half2half2(__ushort_as_half(0x6480));   // 1152
    uint32_t x = __byte_perm(w, 0x64646464u, 0x4140), y = __byte_perm(w, 0x64646464u, 0x4342);
    const __half2 u = __hsub2(*reinterpret_cast<__half2 *>(&x), off), v = __hsub2(*reinterpret_cast<__half2 *>(&y), off);
    a = *reinterpret_cast<const uint32_t *>(&u);
    b = *reinterpret_cast<const uint32_t *>(&v);
}
// Byte i of w (128 + code) as a float.
template <int I>
__device__ __forceinline__ float code_f32(uint32_t w) {
    return __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440 + I)) - 8388736.f;
}
// mma_f16_16816 onto zeros.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// mma_bf16_16816 onto zeros.
__device__ __forceinline__ void mma_bf16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// Two values to bf16, and what is left of them.
__device__ __forceinline__ void split_bf16(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16(x, y);
    lo = pack_bf16(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xFFFF0000u));
}
__device__ __forceinline__ float scale_at(const uint8_t *row, int d, int block) {
    return __half2float(*reinterpret_cast<const __half *>(row + d + 2 * block));
}

// ROUND, fp32 results: sixteen keys' sum is added to acc with rounding.  The tensor cores cut what they add to an
// accumulator towards zero: 1.1e-9 of a result for a key of a piece's, which bf16 results do not show (3e-5 at 30000
// keys; it costs 8%: 373 us for the 342 above).
template <int DKQ, int DV, bool VK, bool ROUND>
__global__ void __launch_bounds__(kThreads, DV == 512 ? 1 : 2) chunk_q8_tree_kernel(const Params p) {
    using L = Q8<DKQ, DV, VK>;
    constexpr int RK = L::kRK, RV = L::kRV, PK = L::kPK, PV = L::kPV, DVS = VK ? DKQ : DV;   // DVS: where a value row's scales are
    constexpr int BW = L::kBW, MW = L::kMW;
    extern __shared__ __align__(16) uint8_t smem[];
    __half *sQ = reinterpret_cast<__half *>(smem);
    __nv_bfloat16 *sP = reinterpret_cast<__nv_bfloat16 *>(smem + L::kOffP);
    float *sMax = reinterpret_cast<float *>(smem + L::kOffMax);
    float *sAlpha = reinterpret_cast<float *>(smem + L::kOffAlpha), *sUnit = reinterpret_cast<float *>(smem + L::kOffUnit);
    int *sOk = reinterpret_cast<int *>(smem + L::kOffOk);
    __shared__ Item s_item;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, fr = lane >> 2, fc = lane & 3;
    const int split = blockIdx.z, g = blockIdx.y;
    pdl_wait();
    if (warp == 0) {
        const Item it = find_item(p, blockIdx.x, g == 0 && split == 0);
        if (lane == 0) s_item = it;
    }
    __syncthreads();
    const Item it = s_item;
    if (it.seq < 0) return;
    const int r0 = it.tile * kQ8Rows;                       // first flattened row
    const int n = min(it.q.n, p.n_new_max);
    const int rows = min(kQ8Rows, (int)((int64_t)n * p.G - r0));
    const int cached = it.q.total - it.q.n;
    const int len = list_end(p, it.q, 0), begin = list_begin(p, it.q, len);
    int k0, k1;
    piece_keys(p, blockIdx.x, g, split, begin, len, k0, k1);
    const bool whole = one_piece(p, blockIdx.x, g, len - begin);
    if (split > 0 && k0 >= k1) return;                     // no such piece

    // raw rows of the tile of keys t0 ..: a warp has four keys'
    auto fetch = [&](int t0, int b) {
        const int key = warp * 4 + (lane & 3), t = t0 + key;
        const int64_t mine = t < k1 ? cell_of(p, it.seq, t) : -1;
        if (lane < 4) sOk[b * kKeys + key] = mine >= 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t cell = __shfl_sync(0xFFFFFFFFu, mine, i);
            const int64_t row = (cell < 0 ? 0 : cell) * p.h_kv + g;
            const uint32_t on = cell < 0 ? 0u : 16u;
            const uint32_t k = smem_u32(smem + L::kOffK + (b * kKeys + warp * 4 + i) * PK);
            for (int c = lane; c < RK / 16; c += 32)
                cp_async16(k + 16 * c, reinterpret_cast<const uint8_t *>(p.K) + row * RK + 16 * c, on);
            if constexpr (!VK) {
                const uint32_t v = smem_u32(smem + L::kOffV + (b * kKeys + warp * 4 + i) * PV);
                for (int c = lane; c < RV / 16; c += 32)
                    cp_async16(v + 16 * c, reinterpret_cast<const uint8_t *>(p.V) + row * RV + 16 * c, on);
            }
        }
    };
    const int n_tiles = (k1 - k0 + kKeys - 1) / kKeys;
#pragma unroll
    for (int t = 0; t < kBufs - 1; ++t) {
        if (t < n_tiles) fetch(k0 + t * kKeys, t);
        cp_async_commit();
    }
    // queries: a warp has eight rows, each brought to a largest value of 2^14 .. 2^15
    for (int i = 0; i < kQ8Rows / 8; ++i) {
        const int row = warp * (kQ8Rows / 8) + i;
        constexpr int N = (DKQ + 63) / 64;   // pairs of a lane
        float2 v[N];
        float top = 0.f;
        const int64_t at = row < rows ? ((int64_t)(it.q.c0 + (r0 + row) / p.G) * p.h_q + g * p.G + (r0 + row) % p.G) * DKQ : 0;
#pragma unroll
        for (int x = 0; x < N; ++x) {
            const uint32_t u = row < rows ? *reinterpret_cast<const uint32_t *>(reinterpret_cast<const __nv_bfloat16 *>(p.Q) +
                                                                                 at + 64 * x + 2 * lane)
                                          : 0u;
            v[x] = make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
            top = fmaxf(top, fmaxf(fabsf(v[x].x), fabsf(v[x].y)));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        // 2^e, -113 to 126: a row of zeros, or with an infinity, keeps its values' size
        const int e = top > 0.f && top < INFINITY ? min(126, 14 - ((int)(__float_as_uint(top) >> 23) - 127)) : 0;
        const float f = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
        for (int x = 0; x < N; ++x)
            *reinterpret_cast<__half2 *>(sQ + row * L::kPQ + 64 * x + 2 * lane) = __floats2half2_rn(v[x].x * f, v[x].y * f);
        if (lane == 0) sUnit[row] = __uint_as_float((uint32_t)(127 - e) << 23);
    }
    const int rg = warp >> 1, kh = warp & 1;   // scores: rows 16 rg .., keys 16 kh ..
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

    int buf = 0;
    for (int t = 0; t < n_tiles; ++t) {
        const int t0 = k0 + t * kKeys;
        cp_async_wait<kBufs - 2>();
        __syncthreads();   // the tile is there, for all; the one before is done with
        if (t + kBufs - 1 < n_tiles) fetch(t0 + (kBufs - 1) * kKeys, buf == 0 ? kBufs - 1 : buf - 1);
        cp_async_commit();
        const uint8_t *rK = smem + L::kOffK + buf * kKeys * PK;
        const uint8_t *rV = VK ? rK : smem + L::kOffV + buf * kKeys * PV;
        float s[2][4] = {};   // keys 16 kh + 8 nt + 2 fc, + 1 of both rows
        {
            const __half *qa = sQ + (16 * rg + fr) * L::kPQ + 8 * fc;
            const uint8_t *kc = rK + (16 * kh + fr) * PK + 8 * fc, *ks = rK + (16 * kh + 2 * fc) * PK + DKQ;
#pragma unroll 1
            for (int b0 = 0; b0 < (16 * rg < rows ? DKQ / 32 : 0); b0 += 2) {
                float2 c[2][2];   // scales of both blocks, of keys 8 nt + 2 fc and the next
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        c[nt][x] = __half22float2(*reinterpret_cast<const __half2 *>(ks + (8 * nt + x) * PK + 2 * b0));
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int b = b0 + y;
                    const uint4 u = *reinterpret_cast<const uint4 *>(qa + 32 * b),
                                v = *reinterpret_cast<const uint4 *>(qa + 8 * L::kPQ + 32 * b);
                    const uint32_t A0[4] = {u.x, v.x, u.y, v.y}, A1[4] = {u.z, v.z, u.w, v.w};
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) {
                        const uint2 w = *reinterpret_cast<const uint2 *>(kc + 8 * nt * PK + 32 * b);
                        uint32_t h[4];
                        codes_f16(w.x, h[0], h[1]);
                        codes_f16(w.y, h[2], h[3]);
                        float d[4];
                        mma_f16_first(d, A0, h[0], h[1]);
                        mma_f16_16816(d, A1, h[2], h[3]);
                        const float c0 = y ? c[nt][0].y : c[nt][0].x, c1 = y ? c[nt][1].y : c[nt][1].x;
                        s[nt][0] = fmaf(d[0], c0, s[nt][0]);
                        s[nt][1] = fmaf(d[1], c1, s[nt][1]);
                        s[nt][2] = fmaf(d[2], c0, s[nt][2]);
                        s[nt][3] = fmaf(d[3], c1, s[nt][3]);
                    }
                }
            }
        }
        float mx[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const int row = 16 * rg + fr + 8 * y;
            const uint32_t node = tree_bits(p, mask[y], cached, t0);
            const float unit = sUnit[row] * p.scale_log2;
            mx[y] = -INFINITY;
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int key = 16 * kh + 8 * nt + 2 * fc + c;
                    float &x = s[nt][2 * y + c];
                    x = sOk[buf * kKeys + key] && ((node >> key) & 1) ? x * unit : -INFINITY;
                    mx[y] = fmaxf(mx[y], x);
                }
            mx[y] = fmaxf(mx[y], __shfl_xor_sync(0xFFFFFFFFu, mx[y], 1));
            mx[y] = fmaxf(mx[y], __shfl_xor_sync(0xFFFFFFFFu, mx[y], 2));
            if (fc == 0) sMax[kh * kQ8Rows + row] = mx[y];
        }
        named_barrier(1 + rg, 64);   // the two warps of these rows
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const int row = 16 * rg + fr + 8 * y;
            const float mn = fmaxf(m[y], fmaxf(mx[y], sMax[(kh ^ 1) * kQ8Rows + row]));
            const float al = m[y] == -INFINITY ? (mn == -INFINITY ? 1.f : 0.f) : exp2f(m[y] - mn);
            float sum = 0.f;
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float x = s[nt][2 * y + c];
                    float e = x == -INFINITY ? 0.f : exp2f(x - mn);
                    sum += e;
                    // a scale that is not finite counts by any weight, however small
                    if (x != -INFINITY && e < 0x1p-126f) e = 0x1p-126f;
                    const __nv_bfloat16 hi = __float2bfloat16_rn(e);
                    __nv_bfloat16 *to = sP + row * kPS + 16 * kh + key_slot(8 * nt + 2 * fc + c);
                    to[0] = hi;
                    to[kQ8Rows * kPS] = __float2bfloat16_rn(e - __bfloat162float(hi));
                }
            }
            m[y] = mn;
            l[y] = l[y] * al + sum;
            if (kh == 0 && fc == 0) sAlpha[row] = al;
        }
        __syncthreads();
#pragma unroll
        for (int x = 0; x < MW; ++x) {
            if ((MW < 4 || x == 2) && 16 * (MW * mw + x) >= rows) break;
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
        for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
            for (int b = 0; b < BW; ++b) {
                const int blk = BW * bw + b;
                const uint8_t *v0 = rV + (16 * ks + fc) * PV;   // keys fc, + 4, + 8, + 12
                uint32_t w[4];
                float c[4];
                bool odd = false;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const uint8_t *v = v0 + 4 * x * PV;
                    w[x] = *reinterpret_cast<const uint32_t *>(v + 32 * blk + 4 * fr) ^ 0x80808080u;
                    c[x] = scale_at(v, DVS, blk);
                    // a scale that is not finite: not in the products, where a zero weight would not cancel it
                    if (c[x] - c[x] != 0.f) {
                        c[x] = 0.f;
                        odd = true;
                    }
                }
                uint32_t hi[4][2], lo[4][2];   // of dims 4 fr + i
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint32_t u = w[2 * x], v = w[2 * x + 1];
                    const float cu = c[2 * x], cv = c[2 * x + 1];
                    split_bf16(code_f32<0>(u) * cu, code_f32<0>(v) * cv, hi[0][x], lo[0][x]);
                    split_bf16(code_f32<1>(u) * cu, code_f32<1>(v) * cv, hi[1][x], lo[1][x]);
                    split_bf16(code_f32<2>(u) * cu, code_f32<2>(v) * cv, hi[2][x], lo[2][x]);
                    split_bf16(code_f32<3>(u) * cu, code_f32<3>(v) * cv, hi[3][x], lo[3][x]);
                }
#pragma unroll
                for (int x = 0; x < MW; ++x) {
                    if ((MW < 4 || x == 2) && 16 * (MW * mw + x) >= rows) break;
                    uint32_t ph[4], pl[4];
                    const uint32_t pa = smem_u32(sP + (16 * (MW * mw + x) + (lane & 15)) * kPS + 16 * ks + 8 * (lane >> 4));
                    ldsm_x4(pa, ph[0], ph[1], ph[2], ph[3]);
                    ldsm_x4(pa + kQ8Rows * kPS * 2, pl[0], pl[1], pl[2], pl[3]);
                    if constexpr (ROUND) {
                        float d[4][4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) mma_bf16_first(d[i], pl, hi[i][0], hi[i][1]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) mma_bf16_16816(d[i], ph, lo[i][0], lo[i][1]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) mma_bf16_16816(d[i], ph, hi[i][0], hi[i][1]);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int y = 0; y < 4; ++y) acc[b][x][i][y] += d[i][y];
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) mma_bf16_16816(acc[b][x][i], pl, hi[i][0], hi[i][1]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) mma_bf16_16816(acc[b][x][i], ph, lo[i][0], lo[i][1]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) mma_bf16_16816(acc[b][x][i], ph, hi[i][0], hi[i][1]);
                    }
                }
                if (__any_sync(0xFFFFFFFFu, odd)) {   // such keys one by one, to the rows that attend them
                    for (int k = 0; k < 16; ++k) {
                        const uint8_t *v = rV + (16 * ks + k) * PV;
                        const float sc = scale_at(v, DVS, blk);
                        if (sc - sc == 0.f) continue;
#pragma unroll
                        for (int x = 0; x < MW; ++x)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
#pragma unroll
                                for (int y = 0; y < 4; ++y) {   // row fr + 8 (y / 2), dim 8 fc + 4 (y % 2) + i
                                    const int row = 16 * (MW * mw + x) + fr + 8 * (y >> 1);
                                    const float e = __bfloat162float(sP[row * kPS + 16 * ks + key_slot(k)]);
                                    const float code = (float)(int8_t)v[32 * blk + 8 * fc + 4 * (y & 1) + i];
                                    if (e != 0.f) acc[b][x][i][y] += e * (sc * code);
                                }
                    }
                }
            }
        }
        buf = buf == kBufs - 1 ? 0 : buf + 1;
    }
    // ------------------------------------------------------------------------------------ result
    cp_async_wait<0>();
    __syncthreads();   // sMax and sAlpha are read
    const int64_t part0 = (int64_t)piece_part(p, blockIdx.x, g, split) * p.part_rows;
    auto row_of = [&](int row) {
        return (int64_t)(it.q.c0 + (r0 + row) / p.G) * p.h_q + g * p.G + (r0 + row) % p.G;
    };
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        l[y] += __shfl_xor_sync(0xFFFFFFFFu, l[y], 1);
        l[y] += __shfl_xor_sync(0xFFFFFFFFu, l[y], 2);
        if (fc == 0) sMax[kh * kQ8Rows + 16 * rg + fr + 8 * y] = l[y];
    }
    named_barrier(1 + rg, 64);
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        const int row = 16 * rg + fr + 8 * y;
        const float sum = sMax[row] + sMax[kQ8Rows + row];
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
            for (int b = 0; b < BW; ++b) {
                const int d = 32 * (BW * bw + b) + 8 * fc;
                float o[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    o[i] = acc[b][x][i][2 * y] * inv;
                    o[4 + i] = acc[b][x][i][2 * y + 1] * inv;
                }
                if (whole && p.o_bf16) {
                    *reinterpret_cast<uint4 *>(reinterpret_cast<__nv_bfloat16 *>(p.O) + row_of(row) * DV + d) =
                        make_uint4(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7]));
                } else {
                    float4 *to = reinterpret_cast<float4 *>(whole ? reinterpret_cast<float *>(p.O) + row_of(row) * DV + d
                                                                  : p.part_o + (part0 + row) * DV + d);
                    to[0] = make_float4(o[0], o[1], o[2], o[3]);
                    to[1] = make_float4(o[4], o[5], o[6], o[7]);
                }
            }
        }
}

template <int DKQ, int DV, bool VK, bool ROUND>
int launch(const Params &p, cudaStream_t st) {
    if (!ensure_max_dynamic_smem(chunk_q8_tree_kernel<DKQ, DV, VK, ROUND>)) return SFA_ERR_CUDA;
    if (launch_pdl(chunk_q8_tree_kernel<DKQ, DV, VK, ROUND>, dim3(p.items, p.h_kv, p.n_split), dim3(kThreads),
                   (size_t)Q8<DKQ, DV, VK>::kBytes, st, p) != cudaSuccess) {
        cudaGetLastError();
        return SFA_ERR_CUDA;
    }
    return SFA_OK;
}
template <int DKQ, int DV, bool VK>
int launch(const Params &p, cudaStream_t st) {
    return p.o_bf16 ? launch<DKQ, DV, VK, false>(p, st) : launch<DKQ, DV, VK, true>(p, st);
}

}  // namespace

int launch_q8_tree(const Params &p, int dkq, cudaStream_t st) {
    switch (dkq) {
        case 576: return launch<576, 512, true>(p, st);
        case 512: return p.V ? launch<512, 512, false>(p, st) : launch<512, 512, true>(p, st);
        case 128: return p.V ? launch<128, 128, false>(p, st) : launch<128, 128, true>(p, st);
        default: return p.V ? launch<64, 64, false>(p, st) : launch<64, 64, true>(p, st);
    }
}

}  // namespace chunk
}  // namespace sfa
