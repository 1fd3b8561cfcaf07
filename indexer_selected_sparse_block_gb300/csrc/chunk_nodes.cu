// chunk_nodes.cu -- attention of drafted nodes over each other alone (SFA_PART_DRAFTED), bf16 caches.
//
// A node attends its ancestors: a handful of rows, where the tiles of chunk_wide.cuh would compute on every
// node of the tree.  One CTA has one node and 16 heads of one KV head, and gathers the rows that the
// node's mask names, 16 at a time: every row of its tile attends every key, so there is no mask in the
// products, and a value that is not finite reaches the nodes that attend it and no other.
//   S = Q K^T: each of the four warps over a quarter of the head dims, summed in shared memory;
//   O += P V:  each warp a quarter of the value dims, the weights as three bf16 parts (2^-27); keys with a score of
//              minus infinity take their sixteen there one by one.
// It is a chain of latencies a CTA (offsets, mask, page table, rows, scores, softmax, values) on the five CTAs that an
// SM's shared memory and registers hold.  32 trees of 64 nodes, 16 heads, 576 wide, fp32 results: 28.8 us, 3.6 TB/s
// of what has to move, Q and O (105 MB, 16 us); on tiles of all nodes 55.  Four CTAs 2.5 us more; stores of 8 bytes a
// lane and a barrier more, 0.3; operands from global memory straight into registers, values by movmatrix, 10.  The
// test for scores of minus infinity costs 0.3.
#include "chunk_common.cuh"

namespace sfa {
namespace chunk {
namespace {

constexpr int kThreads = 128, kKeys = 16, kHeads = 16;
constexpr int kPR = 18;   // pitch of the scores' rows
constexpr int kPP = 24;   // pitch of the weights' rows, in elements: 16-byte rows without bank conflicts

template <int DKQ, int DV, bool VK>
struct Nodes16 {
    static constexpr int kPQ = DKQ + 8, kPV = DV + 8;   // pitches, as above
    static constexpr int kOffK = kHeads * kPQ * 2;
    static constexpr int kOffV = kOffK + kKeys * kPQ * 2;
    static constexpr int kOffRed = kOffV + (VK ? 0 : kKeys * kPV * 2);   // float [4][16][kPR]
    static constexpr int kOffP = kOffRed + 4 * 16 * kPR * 4;              // bf16 [3][16][kPP]
    static constexpr int kOffCell = kOffP + 3 * 16 * kPP * 2;            // int64 [16]
    static constexpr int kOffAlpha = kOffCell + kKeys * 8;               // float [16]
    static constexpr int kOffList = kOffAlpha + 16 * 4;                  // uint16 [kNodesMax]
    static constexpr int kBytes = kOffList + kNodesMax * 2;
};

// Rows of D elements at pitch P from the cells; zeros where there is none.
template <int D, int P>
__device__ __forceinline__ void gather(uint32_t to, const void *src, const int64_t *cells, int h_kv, int g) {
    constexpr int C = D / 8;
    for (int e = threadIdx.x; e < kKeys * C; e += kThreads) {
        const int r = e / C, c = e - r * C;
        const int64_t cell = cells[r];
        cp_async16(to + r * P * 2 + c * 16,
                   reinterpret_cast<const __nv_bfloat16 *>(src) + ((cell < 0 ? 0 : cell) * h_kv + g) * D + c * 8,
                   cell < 0 ? 0u : 16u);
    }
}

// O += P V key by key, where a score is minus infinity: in the products its weight of zero would bring values
// that are not finite into that row.  The scores are in sRed still; a key without a cell is zeros.
template <int DV, int NT, int PV>
__device__ __forceinline__ void add_values(const Params &p, const float *sRed, const __nv_bfloat16 *sP, const float *sAlpha,
                                           const uint8_t *sV, bool more, float (&acc)[NT][4]) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const int r = (lane >> 2) + 8 * c;
        const float al = more ? sAlpha[r] : 1.f;
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            acc[x][2 * c] *= al;
            acc[x][2 * c + 1] *= al;
        }
#pragma unroll 1
        for (int k = 0; k < kKeys; ++k) {
            const float *f = sRed + r * kPR + k;
            if (((f[0] + f[16 * kPR]) + (f[2 * 16 * kPR] + f[3 * 16 * kPR])) * p.scale_log2 == -INFINITY) continue;
            const __nv_bfloat16 *w = sP + r * kPP + k;
            const float e = __bfloat162float(w[0]) + (__bfloat162float(w[16 * kPP]) + __bfloat162float(w[2 * 16 * kPP]));
            const __nv_bfloat162 *v = reinterpret_cast<const __nv_bfloat162 *>(sV) + (k * PV + warp * (DV / 4)) / 2 + (lane & 3);
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                const float2 y = __bfloat1622float2(v[4 * x]);
                acc[x][2 * c] = fmaf(e, y.x, acc[x][2 * c]);
                acc[x][2 * c + 1] = fmaf(e, y.y, acc[x][2 * c + 1]);
            }
        }
    }
}

template <int DKQ, int DV, bool VK>
__global__ void __launch_bounds__(kThreads, DV == 512 ? 5 : 8) drafted_nodes_kernel(const Params p) {
    using L = Nodes16<DKQ, DV, VK>;
    constexpr int NT = DV / 32;   // 8-wide column tiles of a warp's value dims
    extern __shared__ __align__(16) uint8_t smem[];
    float *sRed = reinterpret_cast<float *>(smem + L::kOffRed);
    __nv_bfloat16 *sP = reinterpret_cast<__nv_bfloat16 *>(smem + L::kOffP);
    int64_t *sCell = reinterpret_cast<int64_t *>(smem + L::kOffCell);
    float *sAlpha = reinterpret_cast<float *>(smem + L::kOffAlpha);
    uint16_t *sList = reinterpret_cast<uint16_t *>(smem + L::kOffList);
    __shared__ int s_count;
    __shared__ float sInv[16];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sQ = smem_u32(smem), sK = sQ + L::kOffK, sV = VK ? sK : sQ + L::kOffV;
    constexpr int PV = VK ? L::kPQ : L::kPV;
    pdl_wait();
    const int s = blockIdx.x / p.n_new_max, j = blockIdx.x - s * p.n_new_max;
    const int groups = (p.G + kHeads - 1) / kHeads, g = blockIdx.y / groups, h0 = (blockIdx.y - g * groups) * kHeads;
    const Seq q = load_seq(p, s, j == 0 && blockIdx.y == 0 && tid == 0);
    const int n = min(q.n, p.n_new_max);
    if (j >= n) return;
    const int heads = min(kHeads, p.G - h0), a = q.total - q.n;
    const int64_t row0 = (int64_t)(q.c0 + j) * p.h_q + g * p.G + h0;   // the tile's first (node, head)
    {   // the heads' queries, one run of memory
        const __nv_bfloat16 *src = reinterpret_cast<const __nv_bfloat16 *>(p.Q) + row0 * DKQ;
        constexpr int C = DKQ / 8;
        for (int e = tid; e < kHeads * C; e += kThreads) {
            const int r = e / C, c = e - r * C;
            cp_async16(sQ + r * L::kPQ * 2 + c * 16, src + (r < heads ? (int64_t)r * DKQ : 0) + c * 8, r < heads ? 16u : 0u);
        }
        cp_async_commit();
    }
    if (warp == 0) {   // the nodes that the mask names, below the sequence's end
        const int end = min(n, key_limit(p, q) - a);
        uint32_t bits = lane < p.mask_words && 32 * lane < end ? __ldg(p.mask + (int64_t)(q.c0 + j) * p.mask_words + lane) : 0u;
        if (end - 32 * lane < 32 && end > 32 * lane) bits &= (1u << (end - 32 * lane)) - 1u;
        int at = __popc(bits);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, at, o);
            if (lane >= o) at += y;
        }
        if (lane == 31) s_count = at;
        at -= __popc(bits);
        for (uint32_t b = bits; b; b &= b - 1) sList[at++] = (uint16_t)(32 * lane + __ffs(b) - 1);
        __syncwarp();
    }
    float m = -INFINITY, l = 0.f;   // of row tid / 8, base 2
    float acc[NT][4];               // value dims DV / 4 warp + 8 x + ..
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[x][c] = 0.f;
    int count = 0;
    for (int k0 = 0;; k0 += kKeys) {
        if (warp == 0 && lane < kKeys) {
            const bool on = k0 + lane < s_count;
            const int t = on ? a + sList[k0 + lane] : -1;
            sCell[lane] = t >= 0 ? cell_of(p, s, t) : -1;
        }
        __syncthreads();   // the chunk before is done with its rows; the cells are there
        count = s_count;
        if (k0 >= count) break;
        gather<DKQ, L::kPQ>(sK, p.K, sCell, p.h_kv, g);
        if constexpr (!VK) gather<DV, L::kPV>(sV, p.V, sCell, p.h_kv, g);
        cp_async_commit();
        cp_async_wait<0>();
        __syncthreads();
        {   // the warp's part of the scores
            float sc[2][4] = {};
            constexpr int NK = DKQ / 64;   // steps of 16 dims
            const uint32_t qa = sQ + ((lane & 15) * L::kPQ + warp * (DKQ / 4) + 8 * (lane >> 4)) * 2;
            const uint32_t ka = sK + (((lane & 7) + 8 * (lane >> 4)) * L::kPQ + warp * (DKQ / 4) + 8 * ((lane >> 3) & 1)) * 2;
#pragma unroll
            for (int i = 0; i < NK; ++i) {
                uint32_t A[4], B[2][2];
                ldsm_x4(qa + 32 * i, A[0], A[1], A[2], A[3]);
                ldsm_x4(ka + 32 * i, B[0][0], B[0][1], B[1][0], B[1][1]);
                mma_bf16_16816(sc[0], A, B[0][0], B[0][1]);
                mma_bf16_16816(sc[1], A, B[1][0], B[1][1]);
            }
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    *reinterpret_cast<float2 *>(sRed + (warp * 16 + (lane >> 2) + 8 * c) * kPR + 8 * x + 2 * (lane & 3)) =
                        make_float2(sc[x][2 * c], sc[x][2 * c + 1]);
        }
        __syncthreads();
        bool minus_inf = false;   // the score of a key that is
        {   // softmax of row tid / 8, keys tid % 8 and 8 more
            const int r = tid >> 3, k = tid & 7;
            float v[2], mx = -INFINITY;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float *f = sRed + r * kPR + k + 8 * x;
                v[x] = (f[0] + f[16 * kPR]) + (f[2 * 16 * kPR] + f[3 * 16 * kPR]);
                v[x] *= p.scale_log2;
                const bool key = sCell[k + 8 * x] >= 0;
                minus_inf = minus_inf || (key && v[x] == -INFINITY);
                v[x] = key ? v[x] : -INFINITY;
                mx = fmaxf(mx, v[x]);
            }
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
            const float mn = fmaxf(m, mx), al = m == -INFINITY ? 0.f : exp2f(m - mn);
            float sum = 0.f;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float e = v[x] == -INFINITY ? 0.f : exp2f(v[x] - mn);
                sum += e;
                float rest = e;
#pragma unroll
                for (int y = 0; y < 3; ++y) {
                    const __nv_bfloat16 b = __float2bfloat16_rn(rest);
                    sP[(y * 16 + r) * kPP + k + 8 * x] = b;
                    rest -= __bfloat162float(b);
                }
            }
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
            m = mn;
            l = l * al + sum;
            if (k == 0) sAlpha[r] = al;
        }
        if (__syncthreads_or(minus_inf)) {
            add_values<DV, NT, PV>(p, sRed, sP, sAlpha, smem + (VK ? L::kOffK : L::kOffV), k0 > 0, acc);
        } else {
            const float al0 = sAlpha[lane >> 2], al1 = sAlpha[(lane >> 2) + 8];
            uint32_t A[3][4];
            const uint32_t pa = smem_u32(sP) + ((lane & 15) * kPP + 8 * (lane >> 4)) * 2;
#pragma unroll
            for (int y = 0; y < 3; ++y) ldsm_x4(pa + y * 16 * kPP * 2, A[y][0], A[y][1], A[y][2], A[y][3]);
            const uint32_t va = sV + (((lane & 7) + 8 * ((lane >> 3) & 1)) * PV + warp * (DV / 4) + 8 * (lane >> 4)) * 2;
#pragma unroll
            for (int x = 0; x < NT; x += 2) {
                uint32_t B[2][2];
                ldsm_x4_t(va + 16 * x, B[0][0], B[0][1], B[1][0], B[1][1]);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float (&o)[4] = acc[x + i];
                    if (k0 > 0) {
                        o[0] *= al0;
                        o[1] *= al0;
                        o[2] *= al1;
                        o[3] *= al1;
                    }
#pragma unroll
                    for (int y = 2; y >= 0; --y) mma_bf16_16816(o, A[y], B[i][0], B[i][1]);
                }
            }
        }
        if (k0 + kKeys >= count) break;
    }
    // ------------------------------------------------------------------------------------ result
    const bool any = l > 0.f || l != l;
    if ((tid & 7) == 0) {
        const int r = tid >> 3;
        sInv[r] = any ? 1.f / l : 0.f;
        if (r < heads && p.lse) p.lse[row0 + r] = any ? (m + log2f(l)) / kLog2e : -INFINITY;
    }
    cp_async_wait<0>();   // a node that attends nothing has its queries in flight still
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const int r = (lane >> 2) + 8 * c;
        const float inv = sInv[r];
        // two lanes have a row's four neighbouring dims of two tiles: each takes one tile's
        const int64_t e = (row0 + r) * DV + warp * (DV / 4) + 4 * ((lane & 3) >> 1);
        const bool odd = lane & 1;
#pragma unroll
        for (int x = 0; x < NT; x += 2) {
            const float u0 = acc[x][2 * c] * inv, u1 = acc[x][2 * c + 1] * inv, v0 = acc[x + 1][2 * c] * inv,
                        v1 = acc[x + 1][2 * c + 1] * inv;
            if (p.o_bf16) {
                const uint32_t u = pack_bf16(u0, u1), v = pack_bf16(v0, v1), other = __shfl_xor_sync(0xFFFFFFFFu, odd ? u : v, 1);
                if (r < heads)
                    *reinterpret_cast<uint2 *>(reinterpret_cast<__nv_bfloat16 *>(p.O) + e + 8 * (x + odd)) =
                        odd ? make_uint2(other, v) : make_uint2(u, other);
            } else {
                const float o0 = __shfl_xor_sync(0xFFFFFFFFu, odd ? u0 : v0, 1), o1 = __shfl_xor_sync(0xFFFFFFFFu, odd ? u1 : v1, 1);
                if (r < heads)
                    *reinterpret_cast<float4 *>(reinterpret_cast<float *>(p.O) + e + 8 * (x + odd)) =
                        odd ? make_float4(o0, o1, v0, v1) : make_float4(u0, u1, o0, o1);
            }
        }
    }
}

template <int DKQ, int DV, bool VK>
int launch(const Params &p, cudaStream_t st) {
    using L = Nodes16<DKQ, DV, VK>;
    if (L::kBytes > 48 * 1024 && !ensure_max_dynamic_smem(drafted_nodes_kernel<DKQ, DV, VK>)) return SFA_ERR_CUDA;
    const int64_t x = (int64_t)p.n_seq * p.n_new_max;
    const int y = p.h_kv * ((p.G + kHeads - 1) / kHeads);
    if (launch_pdl(drafted_nodes_kernel<DKQ, DV, VK>, dim3((unsigned)x, (unsigned)y), dim3(kThreads), (size_t)L::kBytes, st,
                   p) != cudaSuccess) {
        cudaGetLastError();
        return SFA_ERR_CUDA;
    }
    return SFA_OK;
}

}  // namespace

int launch_nodes(const Params &p, int dkq, cudaStream_t st) {
    switch (dkq) {
        case 576: return launch<576, 512, true>(p, st);
        case 512: return p.V ? launch<512, 512, false>(p, st) : launch<512, 512, true>(p, st);
        case 128: return p.V ? launch<128, 128, false>(p, st) : launch<128, 128, true>(p, st);
        default: return p.V ? launch<64, 64, false>(p, st) : launch<64, 64, true>(p, st);
    }
}

}  // namespace chunk
}  // namespace sfa
