// chunk.cu -- causal attention of each sequence's chunk of new tokens over its pages
// (sfa_chunk_attend_paged), and the attention of its drafted tree (sfa_tree_attend_paged): the kernel
// of fp32 and q8_0 caches, the merge of split lists, the launch plan and the C entry points.
#include "chunk_common.cuh"

namespace sfa {
namespace chunk {
namespace {

// ------------------------------------------------------------------------------ fp32 kernel
// fp32 and q8_0 caches.  One CTA: 32 rows (query, head) of one KV head against TK keys at a time.
// Both products run on the tensor cores as three tf32 ones (mma.sync): each operand is cut in
// hi + lo of 11 bits each (hi = x rounded, lo = x - hi cut: at most 2^-21 of x is lost), and
// hi hi + hi lo + lo hi, summed in fp32, leaves at most 2^-22 of the product out.  Eight warps (wide
// heads: two times eight, a half of the rows each) score an eighth of the head dim, the eight sums
// and the softmax meet in shared memory in fp32, and each warp has its part of the value dims.  The
// wide heads' fp32 rows come by asynchronous copies into a second buffer while the tile before is
// worked on; the narrow ones leave room for two CTAs an SM.
// The rate of mma.sync bounds it (the warps wait for that pipe most): 300 tokens behind 4096, 576
// wide, 40 TFLOP/s, 120 of tf32; plain fp32 multiplications in the same frame made 25.  512 wide with
// V apart 1158 us with 16 warps, 1243 with eight; 576 wide the same with either.
constexpr int kRows = 32;

template <int DKQ, int DV, bool VK>
struct F32 {
    static constexpr int TK = DKQ > 128 ? 16 : 32;
    static constexpr int kSides = DKQ > 128 ? 2 : 1;          // the scores' warps: 8 dim groups x row halves
    static constexpr int kThreads = 256 * kSides;
    static constexpr int PK = DKQ + 4, PV = DV + 4;   // row pitches: conflict-free 16-byte reads
    static constexpr int kTile = TK * PK + (VK ? 0 : TK * PV);
    // two tiles where they fit beside Q
    static constexpr int kPP = TK + 4;                // pitch of the weights' rows
    static constexpr int kBase = kRows * PK + 8 * kRows * TK + kRows * kPP + 3 * kRows;
    static constexpr int kBufs = DKQ > 128 && (kBase + 2 * kTile) * 4 + 2 * TK * 8 <= 226 * 1024 ? 2 : 1;
    static constexpr int kFloats = kBase + kBufs * kTile;
    static constexpr size_t bytes() { return kFloats * 4 + kBufs * TK * 8; }
};

__device__ __forceinline__ float4 load4(const void *base, int64_t elem, int dtype) {
    if (dtype == SFA_F32) return *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(base) + elem);
    const uint2 u = *reinterpret_cast<const uint2 *>(reinterpret_cast<const __nv_bfloat16 *>(base) + elem);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u),
                       __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xFFFF0000u));
}

// Rows (cell, g) of a cache into shared memory as fp32: D elements at pitch D + 4, zeros where
// the cell is -1.
template <int D, int THREADS>
__device__ __forceinline__ void load_rows(float *dst, const void *src, int dtype, const int64_t *cells,
                                          int n, int h_kv, int g) {
    constexpr int C = D / 4;
    for (int e = threadIdx.x; e < n * C; e += THREADS) {
        const int r = e / C, c = e - r * C;
        const int64_t cell = cells[r];
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (cell >= 0) {
            const int64_t row = cell * h_kv + g;
            if (dtype == SFA_Q8_0) {
                const uint8_t *y = reinterpret_cast<const uint8_t *>(src) + row * q8_row_bytes(D);
                const char4 q = *reinterpret_cast<const char4 *>(y + 4 * c);
                const float s = __half2float(*reinterpret_cast<const __half *>(y + D + 2 * (c / 8)));
                v = make_float4(s * q.x, s * q.y, s * q.z, s * q.w);
            } else {
                v = load4(src, row * D + 4 * c, dtype);
            }
        }
        *reinterpret_cast<float4 *>(dst + r * (D + 4) + 4 * c) = v;
    }
}

// The same of an fp32 cache by asynchronous copies.
template <int D, int THREADS>
__device__ __forceinline__ void copy_rows(float *dst, const void *src, const int64_t *cells, int n, int h_kv, int g) {
    constexpr int C = D / 4;
    const uint32_t to = smem_u32(dst);
    for (int e = threadIdx.x; e < n * C; e += THREADS) {
        const int r = e / C, c = e - r * C;
        const int64_t cell = cells[r];
        const float *row = reinterpret_cast<const float *>(src) + (cell < 0 ? 0 : cell * h_kv + g) * D;
        cp_async16(to + (r * (D + 4) + 4 * c) * 4, row + 4 * c, cell < 0 ? 0u : 16u);
    }
}

// Writes four value dims of one row: the result, or a partial one of a split list.
__device__ __forceinline__ void store4(const Params &p, int64_t row, int dv, int d, float4 v) {
    if (p.o_bf16)
        *reinterpret_cast<uint2 *>(reinterpret_cast<__nv_bfloat16 *>(p.O) + row * dv + d) =
            make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
    else
        *reinterpret_cast<float4 *>(reinterpret_cast<float *>(p.O) + row * dv + d) = v;
}

// x as hi + lo, tf32 both, by two integer and two fp32 operations (with cvt.rna.tf32 the kernel took
// 1308 us at 300 tokens behind 4096, 576 wide, when it took 1083 so).  A NaN that the addition carries out of
// the exponent is NaN in lo.
__device__ __forceinline__ void split_tf32(float x, uint32_t &hi, uint32_t &lo) {
    hi = (__float_as_uint(x) + 0x1000u) & 0xFFFFE000u;
    lo = __float_as_uint(x - __uint_as_float(hi)) & 0xFFFFE000u;
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
__device__ __forceinline__ void mma_split(float (&d)[4], const uint32_t (&ah)[4], const uint32_t (&al)[4],
                                          const uint32_t (&bh)[2], const uint32_t (&bl)[2]) {
    mma_tf32(d, al, bh);
    mma_tf32(d, ah, bl);
    mma_tf32(d, ah, bh);
}

template <int DKQ, int DV, bool VK>
__global__ void __launch_bounds__(F32<DKQ, DV, VK>::kThreads) chunk_f32_kernel(const Params p, int dtype) {
    using L = F32<DKQ, DV, VK>;
    constexpr int TK = L::TK, PK = L::PK, PV = VK ? L::PK : L::PV, BUFS = L::kBufs, PP = L::kPP;
    constexpr int kThreads = L::kThreads, SIDES = L::kSides, RT = 2 / SIDES;   // RT: 16-row tiles of a scoring warp
    extern __shared__ __align__(16) float sm[];
    float *sQ = sm, *sTile = sQ + kRows * PK;    // [BUFS] x (K rows, V rows)
    float *sRed = sTile + BUFS * L::kTile;
    float *sP = sRed + 8 * kRows * TK;           // [row][key slot]
    float *sM = sP + kRows * PP, *sL = sM + kRows, *sA = sL + kRows;
    int64_t *sCells = reinterpret_cast<int64_t *>(sA + kRows);   // [BUFS][TK]
    __shared__ Item s_item;
    __shared__ unsigned s_odd;   // keys of the tile with values that are not finite
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int fr = lane >> 2, fc = lane & 3;   // a fragment's row and column of this lane
    const int split = blockIdx.z, g = blockIdx.y;
    pdl_wait();
    if (warp == 0) {
        const Item it = find_item(p, blockIdx.x, g == 0 && split == 0);
        if (lane == 0) s_item = it;
    }
    __syncthreads();
    const Item it = s_item;
    if (it.seq < 0) return;
    const int r0 = it.tile * kRows;                        // first flattened row
    const int n = min(it.q.n, p.n_new_max);
    const int rows = min(kRows, (int)((int64_t)n * p.G - r0));
    const int pos0 = it.q.total - it.q.n;                  // position of the chunk's first query
    const int p_last = pos0 + (r0 + rows - 1) / p.G;
    const int len = max(0, min(key_limit(p, it.q), p_last + 1));
    const int k0 = (int)min((int64_t)len, (int64_t)split * p.split_keys);
    const int k1 = (int)min((int64_t)len, (int64_t)k0 + p.split_keys);
    const bool whole = len <= p.split_keys;                // this piece is the whole list
    if (split > 0 && k0 >= k1) return;                     // no such piece

    for (int e = tid; e < kRows * (DKQ / 4); e += kThreads) {
        const int r = e / (DKQ / 4), c = e - r * (DKQ / 4);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows) {
            const int q = (r0 + r) / p.G, h = g * p.G + (r0 + r) % p.G;
            v = load4(p.Q, ((int64_t)(it.q.c0 + q) * p.h_q + h) * DKQ + 4 * c,
                      dtype == SFA_F32 ? SFA_F32 : SFA_BF16);
        }
        *reinterpret_cast<float4 *>(sQ + r * PK + 4 * c) = v;
    }
    if (tid < kRows) {
        sM[tid] = -INFINITY;
        sL[tid] = 0.f;
    }
    constexpr int NT = DV / (kThreads / 4);   // 8-wide column tiles of a warp's value dims
    float acc[2][NT][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[i][n][c] = 0.f;

    // the tile of keys t0 .. into buffer b: its cells, then its rows (ahead: by asynchronous copies)
    const bool ahead = BUFS == 2 && dtype == SFA_F32;
    auto find_cells = [&](int t0, int b) {
        if (tid < TK) sCells[b * TK + tid] = t0 + tid < k1 ? cell_of(p, it.seq, t0 + tid) : -1;
    };
    auto fetch = [&](int b) {
        float *k = sTile + b * L::kTile;
        const int64_t *cells = sCells + b * TK;
        if (ahead) {
            copy_rows<DKQ, kThreads>(k, p.K, cells, TK, p.h_kv, g);
            if constexpr (!VK) copy_rows<DV, kThreads>(k + TK * PK, p.V, cells, TK, p.h_kv, g);
            cp_async_commit();
        } else {
            load_rows<DKQ, kThreads>(k, p.K, dtype, cells, TK, p.h_kv, g);
            if constexpr (!VK) load_rows<DV, kThreads>(k + TK * PK, p.V, dtype, cells, TK, p.h_kv, g);
        }
    };
    const int first_pos = pos0 + r0 / p.G;   // the rows' first position
    if (ahead && k0 < k1) {
        find_cells(k0, 0);
        __syncthreads();
        fetch(0);
    }
    int buf = 0;
    for (int t0 = k0; t0 < k1; t0 += TK) {
        if (ahead) {
            if (t0 + TK < k1) find_cells(t0 + TK, buf ^ 1);
            __syncthreads();   // the previous tile is done with its buffer; the cells are there
            if (t0 + TK < k1) {
                fetch(buf ^ 1);
                cp_async_wait<1>();
            } else {
                cp_async_wait<0>();
            }
        } else {
            __syncthreads();   // the previous tile is done with shared memory
            find_cells(t0, 0);
            __syncthreads();
            fetch(0);
        }
        const float *sK = sTile + buf * L::kTile, *sV = VK ? sK : sK + TK * PK;
        const int64_t *sCell = sCells + buf * TK;
        __syncthreads();
        {   // scores: warp w takes dims [x DKQ / 8, (x + 1) DKQ / 8), x = w mod 8, of its rows
            constexpr int KN = TK / 8;
            const int x = warp & 7, row0 = (warp >> 3) * 16;
            float sc[RT][KN][4];
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int n = 0; n < KN; ++n)
#pragma unroll
                    for (int c = 0; c < 4; ++c) sc[i][n][c] = 0.f;
            const float *q = sQ + (row0 + fr) * PK + x * (DKQ / 8) + fc, *k = sK + fr * PK + x * (DKQ / 8) + fc;
#pragma unroll
            for (int d = 0; d < DKQ / 8; d += 8) {
                uint32_t ah[RT][4], al[RT][4], bh[KN][2], bl[KN][2];
#pragma unroll
                for (int i = 0; i < RT; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        split_tf32(q[(16 * i + 8 * (c & 1)) * PK + d + 4 * (c >> 1)], ah[i][c], al[i][c]);
#pragma unroll
                for (int n = 0; n < KN; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) split_tf32(k[8 * n * PK + d + 4 * c], bh[n][c], bl[n][c]);
#pragma unroll
                for (int i = 0; i < RT; ++i)
#pragma unroll
                    for (int n = 0; n < KN; ++n) mma_split(sc[i][n], ah[i], al[i], bh[n], bl[n]);
            }
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int n = 0; n < KN; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        *reinterpret_cast<float2 *>(sRed + (x * kRows + row0 + 16 * i + 8 * c + fr) * TK + 8 * n + 2 * fc) =
                            make_float2(sc[i][n][2 * c], sc[i][n][2 * c + 1]);
        }
        if (tid == 0) s_odd = 0;
        __syncthreads();
        {   // softmax of row tid / TPR, KPT keys a thread
            constexpr int TPR = kThreads / kRows, KPT = TK / TPR;
            const int r = tid / TPR, kk = tid % TPR;
            const int pos = pos0 + (r0 + r) / p.G;
            float s[KPT], mx = -INFINITY;
#pragma unroll
            for (int b = 0; b < KPT; ++b) {
                const int k = kk + TPR * b;
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < 8; ++w) v += sRed[(w * kRows + r) * TK + k];
                const bool on = sCell[k] >= 0 && t0 + k <= pos;
                if (on && v - v != 0.f) {   // halves of an infinity cancel to NaN: the plain product instead
                    v = 0.f;
                    for (int d = 0; d < DKQ; ++d) v += sQ[r * PK + d] * sK[k * PK + d];
                }
                s[b] = on ? v * p.scale_log2 : -INFINITY;
                mx = fmaxf(mx, s[b]);
            }
#pragma unroll
            for (int o = TPR / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
            const float mo = sM[r], mn = fmaxf(mo, mx);
            float sum = 0.f;
#pragma unroll
            for (int b = 0; b < KPT; ++b) {
                const float e = s[b] == -INFINITY ? 0.f : exp2f(s[b] - mn);
                const int k = kk + TPR * b;   // key slots: see below
                sP[r * PP + (k & ~7) + (k & 1) * 4 + ((k & 7) >> 1)] = e;
                sum += e;
            }
#pragma unroll
            for (int o = TPR / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
            const float al = mn == -INFINITY ? 1.f : exp2f(mo - mn);
            __syncwarp();
            if (kk == 0) {
                sM[r] = mn;
                sL[r] = sL[r] * al + sum;
                sA[r] = al;
            }
        }
        // every key of the tile is attended by every row: no zero weight in front of a NaN
        const bool plain = __syncthreads_and(t0 + TK <= min(k1, first_pos + 1) && (tid >= TK || sCell[tid] >= 0));
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float al = sA[16 * i + 8 * (c >> 1) + fr];
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[i][n][c] *= al;
            }
        const int d0 = warp * (NT * 8);   // the warp's value dims
        if (!plain) {
            // Keys that some rows do not attend may hold NaN and infinities there, which a zero
            // weight does not cancel: such values are taken out of the tile, and added one by one to
            // the rows that attend them.
            float *v = sTile + buf * L::kTile + (VK ? 0 : TK * PK);
            for (int e = tid; e < TK * DV; e += kThreads) {
                const float x = v[(e / DV) * PV + e % DV];
                if (x - x != 0.f) atomicOr(&s_odd, 1u << (e / DV));
            }
            __syncthreads();
            const unsigned odd = s_odd;
            if (odd) {
                for (int k = 0; k < TK; ++k) {
                    if (!((odd >> k) & 1)) continue;
                    const int at = (k & ~7) + (k & 1) * 4 + ((k & 7) >> 1);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                const float x = v[k * PV + d0 + 8 * n + 2 * fc + (c & 1)];
                                const float e = sP[(16 * i + 8 * (c >> 1) + fr) * PP + at];
                                if (x - x != 0.f && e != 0.f) acc[i][n][c] += e * x;
                            }
                }
                __syncthreads();
                for (int e = tid; e < TK * DV; e += kThreads) {
                    float &x = v[(e / DV) * PV + e % DV];
                    if (x - x != 0.f) x = 0.f;
                }
                __syncthreads();
            }
        }
        // Slot j < 4 of eight keys is key 2 j, slot j + 4 key 2 j + 1: the lanes' reads of V then fall
        // in different banks.  A tile's sum is added to acc with rounding: the tensor cores cut towards
        // zero what they add to an accumulator, which a long list would show.
        uint32_t ah[TK / 8][2][4], al[TK / 8][2][4];
#pragma unroll
        for (int k = 0; k < TK / 8; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    split_tf32(sP[(16 * i + 8 * (c & 1) + fr) * PP + 8 * k + fc + 4 * (c >> 1)], ah[k][i][c], al[k][i][c]);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float add[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) add[i][c] = 0.f;
#pragma unroll
            for (int k = 0; k < TK / 8; ++k) {
                uint32_t bh[2], bl[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) split_tf32(sV[(8 * k + 2 * fc + c) * PV + d0 + 8 * n + fr], bh[c], bl[c]);
#pragma unroll
                for (int i = 0; i < 2; ++i) mma_split(add[i], ah[k][i], al[k][i], bh, bl);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[i][n][c] += add[i][c];
        }
        buf = ahead ? buf ^ 1 : 0;
    }
    __syncthreads();
    const int64_t part0 = (int64_t)piece_part(p, blockIdx.x, g, split) * p.part_rows;
#pragma unroll
    for (int i = 0; i < 4; ++i) {   // the lane's rows
        const int row = 16 * (i >> 1) + 8 * (i & 1) + fr;
        if (row >= rows) continue;
        const float l = sL[row], m = sM[row];
        const bool any = l > 0.f || l != l;   // no key: zeros; NaN stays
        const float inv = whole ? (any ? 1.f / l : 0.f) : 1.f;
        const int64_t o = (int64_t)(it.q.c0 + (r0 + row) / p.G) * p.h_q + g * p.G + (r0 + row) % p.G;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int d = warp * (NT * 8) + 8 * n + 2 * fc;
            const float x = acc[i >> 1][n][2 * (i & 1)] * inv, y = acc[i >> 1][n][2 * (i & 1) + 1] * inv;
            if (whole && p.o_bf16)
                *reinterpret_cast<uint32_t *>(reinterpret_cast<__nv_bfloat16 *>(p.O) + o * DV + d) = pack_bf16(x, y);
            else
                *reinterpret_cast<float2 *>((whole ? reinterpret_cast<float *>(p.O) + o * DV : p.part_o + (part0 + row) * DV) + d) =
                    make_float2(x, y);
        }
        if (warp == 0 && fc == 0) {
            if (!whole) {
                p.part_ml[(part0 + row) * 2] = m;
                p.part_ml[(part0 + row) * 2 + 1] = l;
            } else if (p.lse) {
                p.lse[o] = any ? (m + log2f(l)) / kLog2e : -INFINITY;
            }
        }
    }
}

// ----------------------------------------------------------------------------- split merge
// The rows of the lists that were cut: a warp for a row, four in turn (32 to a CTA), or, where a list may have
// many pieces, eight warps for one, each with every eighth piece, summed in the warps' order.  Lane c
// holds where piece c, c + 32, .. left its partial results and the row's (m, l) there.  The kernel is
// a chain of latencies (the list, then its partial results), so the first pieces' rows are asked
// for before the weights are known, 16 bytes a lane.  Lists of one piece were written by the
// attention kernel itself.
constexpr int kMaxPieces = 160;   // of a list
constexpr int kManyPieces = 8;    // from here on eight warps for a row

template <int DV, int WPR>
__global__ void __launch_bounds__(256) chunk_combine_kernel(const Params p) {
    constexpr int W = kMaxPieces / 32, C = (DV + 127) / 128, ROWS = WPR == 8 ? 1 : 32, B = 4;
    __shared__ float s_acc[WPR == 8 ? 8 : 1][WPR == 8 ? DV : 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row0 = blockIdx.z * ROWS + (WPR == 8 ? 0 : warp), first = WPR == 8 ? warp : 0;
    pdl_wait();
    // the list: its rows, and the row tile of partial results of each piece (-1: none)
    int rows, r0, c0, g, n_pieces;
    int part[W];
#pragma unroll
    for (int x = 0; x < W; ++x) part[x] = -1;
    if (p.slots > 0) {   // the work was dealt out: the list that slot blockIdx.x has the start of
        const int c = blockIdx.x;
        const int4 start = p.slot_info[2 * c + 1];
        rows = start.z * p.G;
        if (!start.x || row0 >= rows) return;
        n_pieces = 0;
        bool ended = false;   // a list may end in the last of 32 slots: their number does not say
#pragma unroll
        for (int x = 0; x < W; ++x) {   // lane 0: the start; lane l: the slot l behind it
            if (ended) break;
            const int d = c + lane + 32 * x;
            const int4 head = d > c && d < p.slots ? p.slot_info[2 * d] : make_int4(0, d >= p.slots, 0, 0);
            const unsigned ends = __ballot_sync(0xFFFFFFFFu, head.y != 0);
            ended = ends != 0;
            n_pieces += ended ? __ffs(ends) : 32;
            if (d == c) part[x] = 2 * c + 1;
            else if (head.x && lane + 32 * x < n_pieces) part[x] = 2 * d;
        }
        r0 = 0;
        c0 = start.y;
        g = start.w;
    } else {
        g = blockIdx.y;
        const Item it = find_item(p, blockIdx.x, false);
        if (it.seq < 0) return;
        const int n = min(it.q.n, p.n_new_max);
        if (p.item_q > 0) {
            const int q0 = it.tile * p.item_q;
            r0 = q0 * p.G;
            rows = min(p.item_q, n - q0) * p.G;
        } else {
            r0 = it.tile * p.item_rows;
            rows = min(p.item_rows, (int)((int64_t)n * p.G - r0));
        }
        if (row0 >= rows) return;
        const int p_last = it.q.total - it.q.n + (r0 + rows - 1) / p.G;
        const int end = list_end(p, it.q, p_last + 1), len = end - list_begin(p, it.q, end);
        n_pieces = sfa::chunk::n_pieces(p, blockIdx.x, g, len);
        if (n_pieces == 1) return;
#pragma unroll
        for (int x = 0; x < W; ++x)
            if (lane + 32 * x < n_pieces) part[x] = piece_part(p, blockIdx.x, g, lane + 32 * x);
        c0 = it.q.c0;
    }
    // B of this warp's pieces from piece c on
    auto where = [&](int c) {
        int at = -1;
#pragma unroll
        for (int x = 0; x < W; ++x) {
            const int v = __shfl_sync(0xFFFFFFFFu, part[x], c & 31);
            if (c >> 5 == x) at = v;
        }
        return at;
    };
    auto load = [&](int row, int c, float4 (&v)[B][C]) {
#pragma unroll
        for (int y = 0; y < B; ++y) {
            const int at = where(c + y * WPR);
            const float *src = p.part_o + ((int64_t)max(at, 0) * p.part_rows + row) * DV + lane * 4;
#pragma unroll
            for (int k = 0; k < C; ++k)
                v[y][k] = at >= 0 && k * 128 + lane * 4 < DV ? *reinterpret_cast<const float4 *>(src + k * 128)
                                                            : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    };
#pragma unroll 1
    for (int row = row0; row < min(rows, (int)(blockIdx.z + 1) * ROWS); row += 8) {
        float4 v[B][C];
        load(row, first, v);
        float m[W], w[W], M = -INFINITY, l = 0.f;
#pragma unroll
        for (int x = 0; x < W; ++x) {
            const float2 ml = part[x] >= 0 ? *reinterpret_cast<const float2 *>(p.part_ml + ((int64_t)part[x] * p.part_rows + row) * 2)
                                           : make_float2(-INFINITY, 0.f);
            m[x] = ml.x;
            w[x] = ml.y;
            M = fmaxf(M, m[x]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
#pragma unroll
        for (int x = 0; x < W; ++x) {   // the piece's share of the sum, then its weight
            const bool none = m[x] == -INFINITY && w[x] == 0.f;   // the row attends no key of it
            const float e = m[x] == -INFINITY ? 0.f : exp2f(m[x] - M);
            l += w[x] == 0.f ? 0.f : (m[x] == -INFINITY ? w[x] : e * w[x]);
            w[x] = none ? -1.f : e;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
        float4 acc[C];
#pragma unroll
        for (int c = 0; c < C; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = first; c < n_pieces; c += B * WPR) {
            if (c != first) load(row, c, v);
#pragma unroll
            for (int y = 0; y < B; ++y) {
                const int cy = c + y * WPR;
                float e = 0.f;
#pragma unroll
                for (int x = 0; x < W; ++x) {
                    const float f = __shfl_sync(0xFFFFFFFFu, w[x], cy & 31);
                    if (cy >> 5 == x) e = f;
                }
                if (e < 0.f) continue;   // what its sums hold there may be NaN
#pragma unroll
                for (int k = 0; k < C; ++k) {
                    acc[k].x = fmaf(e, v[y][k].x, acc[k].x);
                    acc[k].y = fmaf(e, v[y][k].y, acc[k].y);
                    acc[k].z = fmaf(e, v[y][k].z, acc[k].z);
                    acc[k].w = fmaf(e, v[y][k].w, acc[k].w);
                }
            }
        }
        const bool any = l > 0.f || l != l;
        const float inv = any ? 1.f / l : 0.f;
        const int64_t o = (int64_t)(c0 + (r0 + row) / p.G) * p.h_q + g * p.G + (r0 + row) % p.G;
        if (lane == 0 && first == 0 && p.lse) p.lse[o] = any ? (M + log2f(l)) / kLog2e : -INFINITY;
        if constexpr (WPR == 8) {
#pragma unroll
            for (int k = 0; k < C; ++k)
                if (k * 128 + lane * 4 < DV) *reinterpret_cast<float4 *>(&s_acc[warp][k * 128 + lane * 4]) = acc[k];
            __syncthreads();
            for (int d = 4 * threadIdx.x; d < DV; d += 4 * 256) {
                float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int y = 0; y < 8; ++y) {
                    const float4 q = *reinterpret_cast<const float4 *>(&s_acc[y][d]);
                    t.x += q.x;
                    t.y += q.y;
                    t.z += q.z;
                    t.w += q.w;
                }
                store4(p, o, DV, d, make_float4(t.x * inv, t.y * inv, t.z * inv, t.w * inv));
            }
        } else {
#pragma unroll
            for (int k = 0; k < C; ++k)
                if (k * 128 + lane * 4 < DV)
                    store4(p, o, DV, k * 128 + lane * 4, make_float4(acc[k].x * inv, acc[k].y * inv, acc[k].z * inv, acc[k].w * inv));
        }
    }
}

// --------------------------------------------------------------------------------- the plan
enum Kernel { kF32, kWide, kNarrow, kNodes, kQ8Tree, kF32Tree };
struct Plan {
    Kernel kernel;
    int item_rows, item_q, items, part_rows;
    int slots;                 // > 0: the work dealt out evenly (Share)
    int n_split, first_keys, split_keys, whole_lists;   // else: pieces of a list
};

// Row tiles of n_q queries in n_seq chunks of at most n_new_max, at most.
int64_t items_bound(int n_seq, int n_q, int G, int n_new_max, int item_rows, int item_q) {
    const int64_t per = item_q > 0 ? ((int64_t)n_new_max + item_q - 1) / item_q
                                   : ((int64_t)n_new_max * G + item_rows - 1) / item_rows;
    const int64_t all = (item_q > 0 ? n_q / item_q : (int64_t)n_q * G / item_rows) + n_seq;
    return per * n_seq < all ? per * n_seq : all;
}

// A tree's row tiles all have lists as long as its sequence: those that are left after the whole waves keep
// few SMs busy for as long as a wave.  Only they are cut: into equal pieces, or, where they are nearly a
// wave themselves, a long first piece each and the rest in m pieces, of which `rounds` follow one another
// on the `spare` places while the long ones run.  Chunks, whose row tiles are many, keep their equal cuts.
// 576 wide, bf16 results: 56 lists of 30000 keys on 76 pairs 283 us whole, 270 so; 80 of 20000 329, 308; 160 of
// 8192 278, 257; 256 of 16384 745, 715.  With every SM busy the card's power lowers its clock by about a
// tenth, which a cut has to gain first (64 lists of 32768 369 us either way, 60 of 16384 186 and 191).
void plan_last_wave(Plan &pl, int64_t units, int64_t tiles, int64_t slots, double t_tile, double t_piece, double t_merge,
                    double part_us, double best_us) {
    const int64_t whole = units / slots * slots, left = units - whole;
    if (left == 0) return;
    const double before = units / slots * (tiles * t_tile + t_piece), t_exit = 1.;   // t_exit: a piece that is none
    auto take = [&](double us, int64_t n, int64_t first, int64_t other) {
        us = before + 1.1 * us + t_merge + left * n * part_us + (double)whole * (n - 1) / slots * t_exit;
        if (us >= best_us || (double)left * n * pl.part_rows * 514 * 4 > 1e9) return;
        best_us = us;
        pl.n_split = (int)n;
        pl.first_keys = (int)(first * 128);
        pl.split_keys = (int)(other * 128);
        pl.whole_lists = (int)whole;
    };
    for (int64_t n = 2; n <= tiles && n <= 64; ++n) {
        const int64_t per = (tiles + n - 1) / n;
        if ((tiles + per - 1) / per == n) take((left * n + slots - 1) / slots * (per * t_tile + t_piece), n, per, per);
    }
    const int64_t spare = slots - left;
    for (int64_t m = 1; m <= 4; ++m) {
        // first * t_tile + t_piece = rounds * (rest / m * t_tile + t_piece), first + rest = tiles
        const int64_t rounds = (left * m + spare - 1) / spare;
        const double rest = (tiles * t_tile - (rounds - 1) * t_piece) / (t_tile * (1. + (double)rounds / m));
        const int64_t cut = (int64_t)(rest / m + 0.5), first = tiles - cut * m;   // cut: tiles of a short piece
        if (cut < 4 || first < cut) continue;
        const double a = first * t_tile + t_piece, b = rounds * (cut * t_tile + t_piece);
        take(a > b ? a : b, 1 + m, first, cut);
    }
}

// Whether the drafted part is done node by node: what is faster by the waves of either, their times measured
// on trees (a node's time grows with the nodes it attends, a tile's with the tree).  32 trees of 64 nodes, 576
// wide, 16 heads, fp32 results: 28 us, 55 on tiles; one of 16: 5.2, 12.7; 128 wide, 16 heads on 4: one of 16 3.7,
// 11.3, and 32 of 64 30, 14 on tiles.  (Masks that name every node: 32 of 64, 576 wide, 65 and 55.)
bool use_nodes(int n_seq, int n_q, int G, int h_kv, bool wide, int n_new_max, int64_t items) {
    const int64_t groups = (int64_t)h_kv * ((G + 15) / 16), grid = (int64_t)n_seq * n_new_max, sms = device_sm_count();
    if (n_new_max > kNodesMax || grid > 0x7FFFFFFF || groups > 65535) return false;
    const int64_t nodes = (grid < n_q ? grid : n_q) * groups, at_once = wide ? sms / 2 : sms;
    const double one = wide ? 8.5 / (4. * sms) : 3.7 / (8. * sms), tiles = wide ? 13. : 11.;
    return nodes * one < (items * h_kv + at_once - 1) / at_once * tiles;
}

// The kernel, and how the lists are spread over the SMs: each whole or in equal pieces, a CTA
// (pair) for one, or, by the narrow heads' kernel, all of them dealt out evenly.  What the model
// says takes least time:
//   whole or cut:  waves of pieces (their key tiles, a piece's start and end), and the merge;
//   dealt out:     the tiles' share of a slot, its pieces' starts and ends, and the merge.
// (The wide kernel's pairs would, dealt out, read a cache at 76 places at a time, 147 KB in 1.4 us
// each: more than DRAM has where row tiles share a cache larger than L2.  As one loop over pieces it
// also ran 6% slower at 2048 tokens behind 131072.)
Plan make_plan(int dtype, int n_seq, int n_q, int G, int h_kv, int dv, int n_new_max, int64_t n_kv_max,
               int64_t n_cells, bool o_bf16, int tree) {
    Plan pl;
    const bool tc = dtype == SFA_BF16 && n_cells > 0, wide = tc && dv == 512;
    // (a tree of a bf16 cache of no cell attends nothing, like a chunk of it)
    const bool q8_tree = dtype == SFA_Q8_0 && tree, f32_tree = dtype == SFA_F32 && tree;
    pl.kernel = wide ? kWide : tc ? kNarrow : q8_tree ? kQ8Tree : f32_tree ? kF32Tree : kF32;
    pl.item_rows = wide ? 128 : tc ? 256 : q8_tree ? kQ8Rows : f32_tree ? kF32Rows : kRows;
    pl.item_q = wide ? 2 * wide_qpc(G) : tc ? 2 * narrow_qpt(G) : 0;
    const int64_t items = items_bound(n_seq, n_q, G, n_new_max, pl.item_rows, pl.item_q);
    pl.items = (int)(items > 0x3FFFFFFF ? 0x3FFFFFFF : items);
    if (tree == kDrafted && tc && use_nodes(n_seq, n_q, G, h_kv, wide, n_new_max, items)) {
        pl = Plan{};
        pl.kernel = kNodes;
        pl.n_split = 1;
        return pl;
    }
    const int64_t most = (int64_t)n_new_max * G;
    pl.part_rows = most < pl.item_rows ? (int)most : pl.item_rows;
    const int tile = 128;
    const int64_t tiles = n_kv_max > 0 ? (n_kv_max + tile - 1) / tile : 1, units = items * h_kv;
    int64_t slots = wide ? device_sm_count() / 2 : device_sm_count();
    if (slots > kMaxPieces) slots = kMaxPieces;
    // us: a tile, a piece's start and end in a launch of its own and behind another one, the merge
    double t_tile = wide ? (o_bf16 ? 1.35 : 2.) : tc ? (o_bf16 ? 1.8 : 2.4) : dv == 512 ? 30. : 8.;
    if (tree == kTree && pl.kernel == kNarrow && pl.part_rows <= 128) t_tile *= 0.7;   // one row tile
    if (q8_tree) t_tile = dv == 512 ? 17. : dv == 128 ? 5. : 3.;
    if (f32_tree) t_tile = dv == 512 ? 24. : dv == 128 ? 6. : 4.;
    const double t_piece = 7., t_next = 4., t_merge = 6.;
    const double part_us = (double)pl.part_rows * dv * 4 * 2 / 4e6;   // a partial, both ways
    int64_t best = 1;
    double best_us = 0;
    for (int64_t ns = 1; ns <= tiles && ns <= 128; ++ns) {
        const int64_t per = (tiles + ns - 1) / ns;
        if (ns > 1 && (tiles + per - 1) / per != ns) continue;
        if (ns > 1 && (double)units * ns * pl.part_rows * (dv + 2) * 4 > 1e9) break;
        const int64_t waves = (units * ns + slots - 1) / slots;
        const double us = waves * (per * t_tile + t_piece) + (ns > 1 ? t_merge + units * ns * part_us : 0.);
        if (ns == 1 || us < best_us) {
            best = ns;
            best_us = us;
        }
    }
    const int64_t per = (tiles + best - 1) / best;
    pl.split_keys = best > 1 ? (int)(per * tile) : 0x7FFFFF80;
    pl.n_split = (int)best;
    pl.first_keys = pl.split_keys;
    pl.slots = 0;
    pl.whole_lists = 0;
    if (tree == kTree && wide) plan_last_wave(pl, units, tiles, slots, t_tile, t_piece, t_merge, part_us, best_us);
    if (pl.kernel == kNarrow && units > 0 && tree != kDrafted) {
        // four tiles a slot at least: shorter pieces cost the merge more than they gain
        const int64_t few = (units * tiles + 3) / 4, ss = few < slots ? few : slots;
        // lists shorter than their bound leave whole ones' SMs idle, dealt out ones' not
        const bool ragged = n_q < (int64_t)n_seq * n_new_max;
        double us = (double)units * tiles / ss * t_tile * (ragged ? 0.7 : 1.) + t_piece +
                    (double)units / ss * t_next + (ss > 1 ? t_merge : 0.);
        // A tree's few rows leave a tile's time to the memory once every SM reads, and dealing out costs
        // more than the model of chunks says: pieces and partial results.  (128 wide, 16 heads on 4: 24
        // trees of 16 nodes behind 2048 whole 33 us, dealt out 41; behind 8192 92 and 89; 4 of 60 behind
        // 8192, in equal pieces, 44 and 50; 24 of 1 to 61 behind up to 8192 97 and 79.)
        if (tree == kTree) {
            const double t_read = 128. * 4 * dv / 6.5e6 * ss;   // a tile of K and V
            us += (double)units * tiles / ss * (ragged ? 0.7 : 1.) * (t_read > t_tile ? t_read - t_tile : 0.) + 10. +
                  2. * ss * part_us;
        }
        if (us < best_us) pl.slots = (int)ss;
    }
    return pl;
}

// Row tiles of partial results: each DV values and (m, l) a row; behind them the slots' own notes.
size_t plan_parts(const Plan &pl, int h_kv) {
    return pl.slots > 0 ? 2 * (size_t)pl.slots
                        : pl.n_split > 1 ? ((size_t)pl.items * h_kv - pl.whole_lists) * pl.n_split : 0;
}
size_t plan_workspace(const Plan &pl, int h_kv, int dv) {
    return plan_parts(pl, h_kv) * pl.part_rows * ((size_t)dv + 2) * sizeof(float) + 2 * (size_t)pl.slots * sizeof(int4);
}

bool shape_ok(int dkq, int dv, bool has_v) {
    return (dkq == 576 && dv == 512 && !has_v) || (dkq == 512 && dv == 512) ||
           (dkq == 128 && dv == 128) || (dkq == 64 && dv == 64);
}

template <int DKQ, int DV, bool VK>
int launch_f32(const Params &p, int dtype, cudaStream_t st) {
    if (!ensure_max_dynamic_smem(chunk_f32_kernel<DKQ, DV, VK>)) return SFA_ERR_CUDA;
    if (launch_pdl(chunk_f32_kernel<DKQ, DV, VK>, dim3(p.items, p.h_kv, p.n_split), dim3(F32<DKQ, DV, VK>::kThreads),
                   F32<DKQ, DV, VK>::bytes(), st, p, dtype) != cudaSuccess) {
        cudaGetLastError();
        return SFA_ERR_CUDA;
    }
    return SFA_OK;
}

template <int DV>
int launch_combine(const Params &p, cudaStream_t st) {
    const bool many = p.slots == 0 && p.n_split >= kManyPieces;
    const unsigned z = many ? p.part_rows : (p.part_rows + 31) / 32;
    if (launch_pdl(many ? chunk_combine_kernel<DV, 8> : chunk_combine_kernel<DV, 1>,
                   p.slots > 0 ? dim3(p.slots, 1, z) : dim3(p.items, p.h_kv, z), dim3(256), 0, st,
                   p) != cudaSuccess) {
        cudaGetLastError();
        return SFA_ERR_CUDA;
    }
    return SFA_OK;
}

// Sizes the plan and the workspace query share; SFA_OK, or what the entry point returns.
int check_sizes(int n_seq, int n_q, int h_q, int h_kv, int dkq, int dv, bool has_v, int n_new_max,
                int64_t n_kv_max) {
    if (n_seq < 0 || n_q < 0 || h_kv < 1 || h_q < 1 || h_q % h_kv != 0 || n_new_max < 0 ||
        n_kv_max < 0 || n_kv_max > 0x7FFFFFFF)
        return SFA_ERR_INVALID_ARG;
    if (!has_v && dv > dkq) return SFA_ERR_INVALID_ARG;
    if (!shape_ok(dkq, dv, has_v) || h_q / h_kv > 64 || h_kv > 65535) return SFA_ERR_UNSUPPORTED;
    if ((int64_t)n_q * h_q > 0x7FFFFFFF) return SFA_ERR_UNSUPPORTED;
    return SFA_OK;
}

// The keys that a list has at most: of the drafted part, the nodes and up to 127 keys before them.
int64_t plan_keys(int tree, int n_new_max, int64_t n_kv_max) {
    const int64_t few = (int64_t)n_new_max + 127;
    return tree == kDrafted && few < n_kv_max ? few : n_kv_max;
}

size_t attend_workspace(int dtype, int n_seq, int n_q, int h_q, int h_kv, int dkq, int dv, bool has_v, int n_new_max,
                        int64_t n_kv_max, int o_dtype, int tree) {
    if (check_sizes(n_seq, n_q, h_q, h_kv, dkq, dv, has_v, n_new_max, n_kv_max) != SFA_OK) return 0;
    if (n_seq == 0 || n_q == 0 || n_new_max == 0) return 0;
    return plan_workspace(make_plan(dtype, n_seq, n_q, h_q / h_kv, h_kv, dv, n_new_max,
                                    plan_keys(tree, n_new_max, n_kv_max), 1, o_dtype == SFA_BF16, tree), h_kv, dv);
}

int attend(const void *Q, const void *K, const void *V, int dtype, int64_t n_cells, const int32_t *page_table,
           int64_t table_stride, int page_size, int n_seq, int n_q, int h_q, int h_kv, int dkq, int dv, float scale,
           const int32_t *cu_new, const int32_t *len_total, int tree, const uint32_t *mask, int mask_words,
           int n_new_max, int64_t n_kv_max, void *O, int o_dtype, float *lse, void *workspace, size_t workspace_bytes,
           int32_t *dev_status, sfa_stream_t stream) {
    if (dtype != SFA_BF16 && dtype != SFA_F32 && dtype != SFA_Q8_0) return SFA_ERR_INVALID_ARG;
    if (o_dtype != SFA_BF16 && o_dtype != SFA_F32) return SFA_ERR_INVALID_ARG;
    const int rc = check_sizes(n_seq, n_q, h_q, h_kv, dkq, dv, V != nullptr, n_new_max, n_kv_max);
    if (rc != SFA_OK) return rc;
    if (tree) {
        if (mask_words < 1 || (int64_t)mask_words * 32 < n_new_max) return SFA_ERR_INVALID_ARG;
        if (mask_words > SFA_MAX_TREE / 32) return SFA_ERR_UNSUPPORTED;
    }
    if (page_size < 1 || table_stride < 0 || table_stride > 0x7FFFFFFF ||
        table_stride * page_size > 0x7FFFFFFF || n_cells < 0 || n_cells > 0x7FFFFFFF)
        return SFA_ERR_INVALID_ARG;
    if (!(scale == scale) || scale - scale != 0.f) return SFA_ERR_INVALID_ARG;
    if (n_seq == 0 || n_q == 0 || n_new_max == 0) return SFA_OK;
    if (!Q || !K || !page_table || !cu_new || !len_total || !O || (tree && !mask)) return SFA_ERR_INVALID_ARG;
    if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(O) || !aligned16(lse) ||
        !aligned16(workspace))
        return SFA_ERR_INVALID_ARG;
    // a cache of no cell: every page is a bad one, and any kernel's plan fits the workspace
    const Plan pl = make_plan(dtype, n_seq, n_q, h_q / h_kv, h_kv, dv, n_new_max,
                              n_cells > 0 ? plan_keys(tree, n_new_max, n_kv_max) : 0,
                              n_cells, o_dtype == SFA_BF16, tree);
    const size_t need = plan_workspace(pl, h_kv, dv);
    if (need > 0 && (!workspace || workspace_bytes < need)) return SFA_ERR_WORKSPACE;
    Params p{};
    p.Q = Q;
    p.K = K;
    p.V = V;
    p.table = page_table;
    p.cu = cu_new;
    p.total = len_total;
    p.O = O;
    p.lse = lse;
    p.tree = tree;
    p.mask = mask;
    p.mask_words = mask_words;
    p.part_o = reinterpret_cast<float *>(workspace);
    if (need > 0) {
        const size_t rows = plan_parts(pl, h_kv) * pl.part_rows;
        p.part_ml = p.part_o + rows * dv;
        p.slot_info = reinterpret_cast<int4 *>(p.part_ml + rows * 2);
    }
    p.status = dev_status;
    p.table_stride = table_stride;
    p.page = page_size;
    p.page_div.set(page_size);
    p.n_pages = (int)(n_cells / page_size);
    p.n_seq = n_seq;
    p.n_q = n_q;
    p.h_q = h_q;
    p.h_kv = h_kv;
    p.G = h_q / h_kv;
    p.o_bf16 = o_dtype == SFA_BF16;
    p.items = pl.items;
    p.item_rows = pl.item_rows;
    p.part_rows = pl.part_rows;
    p.item_q = pl.item_q;
    p.one_tile = pl.item_q > 0 ? n_new_max <= pl.item_q : (int64_t)n_new_max * p.G <= pl.item_rows;
    p.slots = pl.slots;
    p.n_split = pl.n_split;
    p.whole_lists = pl.whole_lists;
    p.first_keys = pl.first_keys;
    p.split_keys = pl.split_keys;
    p.n_new_max = n_new_max;
    p.n_kv_max = n_kv_max;
    p.scale_log2 = scale * kLog2e;
    cudaStream_t st = (cudaStream_t)stream;
    int r;
    if (pl.kernel == kWide) r = tree ? launch_wide_tree(p, dkq, n_cells, st) : launch_wide(p, dkq, n_cells, st);
    else if (pl.kernel == kNodes) r = launch_nodes(p, dkq, st);
    else if (pl.kernel == kQ8Tree) r = launch_q8_tree(p, dkq, st);
    else if (pl.kernel == kF32Tree) r = launch_f32_tree(p, dkq, st);
    else if (pl.kernel == kNarrow) r = tree ? launch_narrow_tree(p, dkq, n_cells, st) : launch_narrow(p, dkq, n_cells, st);
    else if (dkq == 576) r = launch_f32<576, 512, true>(p, dtype, st);
    else if (dkq == 512) r = V ? launch_f32<512, 512, false>(p, dtype, st) : launch_f32<512, 512, true>(p, dtype, st);
    else if (dkq == 128) r = V ? launch_f32<128, 128, false>(p, dtype, st) : launch_f32<128, 128, true>(p, dtype, st);
    else r = V ? launch_f32<64, 64, false>(p, dtype, st) : launch_f32<64, 64, true>(p, dtype, st);
    if (r != SFA_OK || need == 0 || pl.slots == 1) return r;
    return dv == 512 ? launch_combine<512>(p, st) : dv == 128 ? launch_combine<128>(p, st) : launch_combine<64>(p, st);
}

}  // namespace
}  // namespace chunk
}  // namespace sfa

extern "C" size_t sfa_chunk_attend_workspace_bytes(int dtype, int n_seq, int n_q, int h_q, int h_kv, int dkq, int dv,
                                                   int has_v, int n_new_max, int64_t n_kv_max, int o_dtype) {
    using namespace sfa::chunk;
    return attend_workspace(dtype, n_seq, n_q, h_q, h_kv, dkq, dv, has_v != 0, n_new_max, n_kv_max, o_dtype, kCausal);
}

extern "C" int sfa_chunk_attend_paged(const void *Q, const void *K, const void *V, int dtype, int64_t n_cells,
                                      const int32_t *page_table, int64_t table_stride, int page_size, int n_seq, int n_q,
                                      int h_q, int h_kv, int dkq, int dv, float scale, const int32_t *cu_new,
                                      const int32_t *len_total, int n_new_max, int64_t n_kv_max, void *O, int o_dtype,
                                      float *lse, void *workspace, size_t workspace_bytes, int32_t *dev_status,
                                      sfa_stream_t stream) {
    using namespace sfa::chunk;
    return attend(Q, K, V, dtype, n_cells, page_table, table_stride, page_size, n_seq, n_q, h_q, h_kv, dkq, dv, scale, cu_new,
                  len_total, kCausal, nullptr, 0, n_new_max, n_kv_max, O, o_dtype, lse, workspace, workspace_bytes,
                  dev_status, stream);
}

extern "C" size_t sfa_tree_attend_workspace_bytes(int dtype, int n_seq, int n_q, int h_q, int h_kv, int dkq, int dv, int has_v,
                                                  int part, int n_new_max, int64_t n_kv_max, int o_dtype) {
    using namespace sfa::chunk;
    if (part != SFA_PART_ALL && part != SFA_PART_DRAFTED) return 0;
    return attend_workspace(dtype, n_seq, n_q, h_q, h_kv, dkq, dv, has_v != 0, n_new_max, n_kv_max, o_dtype,
                            part == SFA_PART_ALL ? kTree : kDrafted);
}

extern "C" int sfa_tree_attend_paged(const void *Q, const void *K, const void *V, int dtype, int64_t n_cells,
                                     const int32_t *page_table, int64_t table_stride, int page_size, int n_seq, int n_q,
                                     int h_q, int h_kv, int dkq, int dv, float scale, const int32_t *cu_new,
                                     const int32_t *len_total, const uint32_t *mask, int mask_words, int part, int n_new_max,
                                     int64_t n_kv_max, void *O, int o_dtype, float *lse, void *workspace,
                                     size_t workspace_bytes, int32_t *dev_status, sfa_stream_t stream) {
    using namespace sfa::chunk;
    if (part != SFA_PART_ALL && part != SFA_PART_DRAFTED) return SFA_ERR_INVALID_ARG;
    return attend(Q, K, V, dtype, n_cells, page_table, table_stride, page_size, n_seq, n_q, h_q, h_kv, dkq, dv, scale, cu_new,
                  len_total, part == SFA_PART_ALL ? kTree : kDrafted, mask, mask_words, n_new_max, n_kv_max, O, o_dtype, lse,
                  workspace, workspace_bytes, dev_status, stream);
}
