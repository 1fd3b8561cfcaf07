// rotate.cu -- rotary positions of rows (sfa_rope_frequencies, sfa_rope_init, sfa_rotate_rows).
#include <math.h>

#include "sfa_common.cuh"

namespace sfa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxRows = 8;        // rows of a CTA
constexpr int kTableBytes = kMaxRows * (SFA_MAX_ROT / 2) * (int)sizeof(float2);

enum Kind { kBf16, kRound, kF32 };   // bf16 rows, fp32 into bf16, fp32 rows

struct Rotation {
    const void *src;
    void *dst;
    int64_t src_stride, src_head, dst_stride, dst_head;
    FastDiv by_row, by_head;   // units of a row, of a head
    int row_units, head_units;
    int kind, vec, to_cells;
    int lo, rot;               // a head's units: lo copied ones, rot turned ones, copied ones
    int begin;                 // first dim that turns
    int skip;                  // in place: the copied ones are left out; lo = 0
};
struct Params {
    Rotation r[SFA_MAX_ROTATIONS];
    const int32_t *pos, *slot;
    int32_t *status;
    int64_t n_rows, n_cells;
    int n, rows;               // rows of a CTA
    int half;                  // pairs: n_rot / 2
    int pairs, inverse;
    float magnitude;
    uint64_t turns[SFA_MAX_ROT / 2];
};

// cos and sin of pos * f_j.  The product's low 64 bits are the fraction of a turn; what is left of the
// nearest quarter turn, at most an eighth, is exact to fp32's last bit when it meets sinpi and cospi.
__device__ __forceinline__ float2 turn(const Params &p, int pos, int j) {
    const uint64_t u = (uint64_t)(uint32_t)pos * p.turns[j];
    const uint32_t q = (uint32_t)((u + (1ull << 61)) >> 62);
    const int64_t rest = (int64_t)(u - ((uint64_t)q << 62));
    float s, c;
    sincospif((float)rest * 0x1p-63f, &s, &c);
    const float cc = (q & 1) ? s : c, ss = (q & 1) ? c : s;
    c = (((q + 1) & 2) ? -cc : cc) * p.magnitude;
    s = ((q & 2) ? -ss : ss) * p.magnitude;
    return make_float2(c, p.inverse ? -s : s);
}

// Eight elements of a row in registers, as they were loaded.
template <int KIND>
struct Eight {
    uint4 a[KIND == kBf16 ? 1 : 2];
    __device__ __forceinline__ void load(const void *base, int64_t e) {
        if constexpr (KIND == kBf16) {
            a[0] = __ldcs(reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(base) + e));
        } else {
            const uint4 *x = reinterpret_cast<const uint4 *>(reinterpret_cast<const float *>(base) + e);
            a[0] = __ldcs(x);
            a[1] = __ldcs(x + 1);
        }
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        if constexpr (KIND == kBf16) {
            const uint32_t w[4] = {a[0].x, a[0].y, a[0].z, a[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                f[4 * x] = __uint_as_float(a[x].x);
                f[4 * x + 1] = __uint_as_float(a[x].y);
                f[4 * x + 2] = __uint_as_float(a[x].z);
                f[4 * x + 3] = __uint_as_float(a[x].w);
            }
        }
    }
    __device__ __forceinline__ void put(const float (&f)[8]) {
        if constexpr (KIND == kF32) {
#pragma unroll
            for (int x = 0; x < 2; ++x)
                a[x] = make_uint4(__float_as_uint(f[4 * x]), __float_as_uint(f[4 * x + 1]),
                                  __float_as_uint(f[4 * x + 2]), __float_as_uint(f[4 * x + 3]));
        } else {
            a[0] = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
        }
    }
    __device__ __forceinline__ void store(void *base, int64_t e) const {
        if constexpr (KIND == kF32) {
            uint4 *y = reinterpret_cast<uint4 *>(reinterpret_cast<float *>(base) + e);
            y[0] = a[0];
            y[1] = a[1];
        } else {
            *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(base) + e) = a[0];
        }
    }
};

// A unit is eight elements that stay, eight that turn among themselves (adjacent pairs), or eight of the
// first half and their eight partners.  U of a thread's units are in flight at a time.
template <int KIND, bool PAIRS>
__device__ __forceinline__ void rotate_vec(const Params &p, const Rotation &r, int64_t row0, int rows, const int *sPos,
                                           const int64_t *sDst, const float2 *sTurn) {
    constexpr int U = (KIND == kBf16 ? 4 : 2) / (PAIRS ? 1 : 2);
    const int total = rows * r.row_units;
    for (int e0 = threadIdx.x; e0 < total; e0 += kThreads * U) {
        Eight<KIND> a[U], b[PAIRS ? 1 : U];
        int64_t to[U];
        int row[U], x[U];   // x: the unit's place among the turning ones, -1: it stays, -2: nothing to do
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int e = e0 + k * kThreads;
            x[k] = -2;
            row[k] = 0;
            to[k] = 0;
            if (e >= total) continue;
            row[k] = r.by_row.div(e);
            const int in_row = e - row[k] * r.row_units, h = r.by_head.div(in_row);
            const int u = in_row - h * r.head_units, y = u - r.lo;
            const int64_t d0 = sDst[row[k]];
            if (sPos[row[k]] < 0 || d0 < 0) continue;
            x[k] = y >= 0 && y < r.rot ? y : -1;
            const int dim = y < 0 ? u * 8 : y < r.rot ? r.begin + y * 8 : r.begin + 2 * p.half + (y - r.rot) * 8;
            const int64_t from = (row0 + row[k]) * r.src_stride + h * r.src_head + dim;
            to[k] = d0 * r.dst_stride + h * r.dst_head + dim;
            a[k].load(r.src, from);
            if constexpr (!PAIRS)
                if (x[k] >= 0) b[k].load(r.src, from + p.half);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (x[k] == -2) continue;
            if (KIND == kRound || x[k] >= 0) {
                float f[8];
                a[k].get(f);
                if (x[k] >= 0) {
                    const float2 *t = sTurn + row[k] * p.half + x[k] * (PAIRS ? 4 : 8);
                    if constexpr (PAIRS) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 cs = t[i];
                            const float u = f[2 * i], v = f[2 * i + 1];
                            f[2 * i] = u * cs.x - v * cs.y;
                            f[2 * i + 1] = u * cs.y + v * cs.x;
                        }
                    } else {
                        float g[8];
                        b[k].get(g);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float2 cs = t[i];
                            const float u = f[i], v = g[i];
                            f[i] = u * cs.x - v * cs.y;
                            g[i] = u * cs.y + v * cs.x;
                        }
                        b[k].put(g);
                        b[k].store(r.dst, to[k] + p.half);
                    }
                }
                a[k].put(f);
            }
            a[k].store(r.dst, to[k]);
        }
    }
}

__device__ __forceinline__ float load1(const void *base, int64_t e, int kind) {
    return kind == kBf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(base)[e])
                         : reinterpret_cast<const float *>(base)[e];
}
__device__ __forceinline__ void store1(void *base, int64_t e, int kind, float v) {
    if (kind == kF32) reinterpret_cast<float *>(base)[e] = v;
    else reinterpret_cast<__nv_bfloat16 *>(base)[e] = __float2bfloat16_rn(v);
}
// Rows of any alignment: a unit is an element that stays, or a pair.
__device__ __forceinline__ void rotate_any(const Params &p, const Rotation &r, int64_t row0, int rows, const int *sPos,
                                           const int64_t *sDst, const float2 *sTurn) {
    const int total = rows * r.row_units;
    for (int e = threadIdx.x; e < total; e += kThreads) {
        const int row = r.by_row.div(e);
        const int in_row = e - row * r.row_units, h = r.by_head.div(in_row);
        const int u = in_row - h * r.head_units, y = u - r.lo;
        const int64_t d0 = sDst[row];
        if (sPos[row] < 0 || d0 < 0) continue;
        const int64_t from = (row0 + row) * r.src_stride + h * r.src_head, to = d0 * r.dst_stride + h * r.dst_head;
        if (y >= 0 && y < r.rot) {
            const int a = r.begin + (p.pairs ? 2 * y : y), b = p.pairs ? a + 1 : a + p.half;
            const float2 cs = sTurn[row * p.half + y];
            const float f = load1(r.src, from + a, r.kind), g = load1(r.src, from + b, r.kind);
            store1(r.dst, to + a, r.kind, f * cs.x - g * cs.y);
            store1(r.dst, to + b, r.kind, f * cs.y + g * cs.x);
        } else {
            const int a = y < 0 ? u : r.begin + 2 * p.half + (y - r.rot);
            if (r.kind == kBf16)   // bit for bit: a conversion would quiet a NaN
                reinterpret_cast<uint16_t *>(r.dst)[to + a] = reinterpret_cast<const uint16_t *>(r.src)[from + a];
            else store1(r.dst, to + a, r.kind, reinterpret_cast<const float *>(r.src)[from + a]);
        }
    }
}

// A CTA has up to eight rows of every set: their cosines and sines, once for all heads and sets, then the
// rows themselves.
template <bool PAIRS>
__global__ void __launch_bounds__(kThreads, 3) rotate_rows_kernel(const __grid_constant__ Params p) {
    extern __shared__ float2 sTurn[];   // [rows][half]
    __shared__ int sPos[kMaxRows];
    __shared__ int64_t sRow[kMaxRows], sCell[kMaxRows];
    pdl_wait();
    const int64_t row0 = (int64_t)blockIdx.x * p.rows;
    const int rows = (int)min((int64_t)p.rows, p.n_rows - row0);
    if (threadIdx.x < rows) {
        const int64_t i = row0 + threadIdx.x;
        sPos[threadIdx.x] = p.pos[i];
        sRow[threadIdx.x] = i;
        int64_t c = p.slot ? p.slot[i] : -1;
        if (p.slot && c >= p.n_cells) {
            set_status(p.status, SFA_DEV_BAD_CELL);
            c = -1;
        }
        sCell[threadIdx.x] = c;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < rows * p.half; e += kThreads) {
        const int row = e / p.half;
        sTurn[e] = turn(p, sPos[row], e - row * p.half);
    }
    __syncthreads();
    for (int k = 0; k < p.n; ++k) {
        const Rotation &r = p.r[k];
        const int64_t *to = r.to_cells ? sCell : sRow;
        if (!r.vec) rotate_any(p, r, row0, rows, sPos, to, sTurn);
        else if (r.kind == kBf16) rotate_vec<kBf16, PAIRS>(p, r, row0, rows, sPos, to, sTurn);
        else if (r.kind == kRound) rotate_vec<kRound, PAIRS>(p, r, row0, rows, sPos, to, sTurn);
        else rotate_vec<kF32, PAIRS>(p, r, row0, rows, sPos, to, sTurn);
    }
}

// Whether no two heads of `n` rows overlap: heads within rows, or rows within heads.
bool apart(int64_t n, int64_t stride, int heads, int64_t head, int64_t d) {
    if (n <= 1) stride = 0;
    if (heads <= 1) head = 0;
    if ((n > 1 && stride < d) || (heads > 1 && head < d)) return false;
    if (n <= 1 || heads <= 1) return true;
    return (stride - d) / (heads - 1) >= head || (head - d) / (n - 1) >= stride;   // (n - 1) * stride + d <= head
}

}  // namespace
}  // namespace sfa

extern "C" int sfa_rope_frequencies(int n_rot, double base, double factor, double original_len,
                                    double beta_fast, double beta_slow, double *freq) {
    if (n_rot < 2 || n_rot > SFA_MAX_ROT || n_rot % 2 != 0 || !freq) return SFA_ERR_INVALID_ARG;
    if (!(base > 0.) || !(factor > 0.) || !(original_len >= 0.) || !isfinite(base) || !isfinite(factor) ||
        !isfinite(original_len))
        return SFA_ERR_INVALID_ARG;
    if (original_len > 0. && !(beta_fast > beta_slow && isfinite(beta_fast) && isfinite(beta_slow)))
        return SFA_ERR_INVALID_ARG;
    for (int j = 0; j < n_rot / 2; ++j) {
        const double f = pow(base, -2. * j / n_rot);
        double keep = 0.;
        if (original_len > 0.) {
            keep = (original_len * f / 6.283185307179586476925 - beta_slow) / (beta_fast - beta_slow);
            keep = keep < 0. ? 0. : keep > 1. ? 1. : keep;
        }
        freq[j] = f * keep + f / factor * (1. - keep);
    }
    return SFA_OK;
}

extern "C" int sfa_rope_init(sfa_rope *rope, int n_rot, int pairs, const double *freq, double magnitude) {
    if (!rope || !freq || n_rot < 2 || n_rot > SFA_MAX_ROT || n_rot % 2 != 0 || (pairs != 0 && pairs != 1))
        return SFA_ERR_INVALID_ARG;
    if (!isfinite(magnitude) || !isfinite((float)magnitude)) return SFA_ERR_INVALID_ARG;
    for (int j = 0; j < n_rot / 2; ++j)
        if (!isfinite(freq[j])) return SFA_ERR_INVALID_ARG;
    *rope = sfa_rope{};
    rope->n_rot = n_rot;
    rope->pairs = pairs;
    rope->magnitude = (float)magnitude;
    for (int j = 0; j < n_rot / 2; ++j) {
        const double t = freq[j] / 6.283185307179586476925, frac = t - floor(t);   // [0, 1]
        const double u = frac * 0x1p64;
        rope->turns[j] = u >= 0x1p64 ? 0 : (uint64_t)u;
    }
    return SFA_OK;
}

extern "C" int sfa_rotate_rows(int n, const sfa_row_rotation *rotations, const sfa_rope *rope, int inverse,
                               const int32_t *pos, int64_t n_rows, const int32_t *slot, int64_t n_cells,
                               int32_t *dev_status, sfa_stream_t stream) {
    using namespace sfa;
    if (n < 0 || n > SFA_MAX_ROTATIONS || (n > 0 && !rotations) || !rope || (inverse != 0 && inverse != 1) ||
        n_rows < 0 || n_rows > 0x7FFFFFFF || n_cells < 0 || n_cells > 0x7FFFFFFF)
        return SFA_ERR_INVALID_ARG;
    if (rope->n_rot < 2 || rope->n_rot > SFA_MAX_ROT || rope->n_rot % 2 != 0 || (rope->pairs != 0 && rope->pairs != 1) ||
        rope->magnitude - rope->magnitude != 0.f)
        return SFA_ERR_INVALID_ARG;
    Params p{};
    const int rot = rope->n_rot;
    constexpr int64_t kFar = (int64_t)1 << 40;
    bool cells = false;
    for (int k = 0; k < n; ++k) {
        const sfa_row_rotation &w = rotations[k];
        if ((w.src_dtype != SFA_BF16 && w.src_dtype != SFA_F32) || (w.dst_dtype != SFA_BF16 && w.dst_dtype != SFA_F32))
            return SFA_ERR_INVALID_ARG;
        if (w.src_dtype == SFA_BF16 && w.dst_dtype == SFA_F32) return SFA_ERR_UNSUPPORTED;
        if (w.n_heads < 1 || w.d < 1 || (int64_t)w.n_heads * w.d > (1 << 24) || w.rot_begin < 0 ||
            (int64_t)w.rot_begin + rot > w.d || (w.to_cells != 0 && w.to_cells != 1))
            return SFA_ERR_INVALID_ARG;
        if (w.src_stride < 0 || w.src_head_stride < 0 || w.dst_stride < 0 || w.dst_head_stride < 0 ||
            w.src_stride >= kFar || w.src_head_stride >= kFar || w.dst_stride >= kFar || w.dst_head_stride >= kFar)
            return SFA_ERR_INVALID_ARG;
        if (!apart(w.to_cells ? n_cells : n_rows, w.dst_stride, w.n_heads, w.dst_head_stride, w.d))
            return SFA_ERR_INVALID_ARG;
        const int ss = w.src_dtype == SFA_F32 ? 4 : 2, ds = w.dst_dtype == SFA_F32 ? 4 : 2;
        cells = cells || w.to_cells;
        Rotation &r = p.r[k];
        r.src = w.src;
        r.dst = w.dst;
        r.src_stride = w.src_stride;
        r.src_head = w.src_head_stride;
        r.dst_stride = w.dst_stride;
        r.dst_head = w.dst_head_stride;
        r.to_cells = w.to_cells;
        r.kind = w.src_dtype == SFA_BF16 ? kBf16 : w.dst_dtype == SFA_BF16 ? kRound : kF32;
        const bool same = w.src == w.dst;
        if (n_rows > 0) {
            if (!w.src || !w.dst || reinterpret_cast<uintptr_t>(w.src) % ss != 0 ||
                reinterpret_cast<uintptr_t>(w.dst) % ds != 0)
                return SFA_ERR_INVALID_ARG;
            if (same && (w.to_cells || ss != ds || (n_rows > 1 && w.src_stride != w.dst_stride) ||
                         (w.n_heads > 1 && w.src_head_stride != w.dst_head_stride)))
                return SFA_ERR_INVALID_ARG;
        }
        // strides of a single row or head do not count
        auto far16 = [](int64_t count, int64_t stride, int size) { return count <= 1 || stride * size % 16 == 0; };
        r.vec = aligned16(w.src) && aligned16(w.dst) && w.d % 8 == 0 && w.rot_begin % 8 == 0 &&
                rot % (rope->pairs ? 8 : 16) == 0 && far16(n_rows, w.src_stride, ss) &&
                far16(w.to_cells ? n_cells : n_rows, w.dst_stride, ds) && far16(w.n_heads, w.src_head_stride, ss) &&
                far16(w.n_heads, w.dst_head_stride, ds);
        const int v = r.vec ? 8 : 1;
        r.begin = w.rot_begin;
        r.lo = same ? 0 : w.rot_begin / v;
        r.rot = r.vec && rope->pairs ? rot / v : rot / 2 / v;
        r.head_units = r.lo + r.rot + (same ? 0 : (w.d - w.rot_begin - rot) / v);
        r.row_units = w.n_heads * r.head_units;
        r.by_head.set(r.head_units);
        r.by_row.set(r.row_units);
    }
    if (n == 0 || n_rows == 0) return SFA_OK;
    if (!pos || (cells && !slot)) return SFA_ERR_INVALID_ARG;
    p.pos = pos;
    p.slot = cells ? slot : nullptr;
    p.status = dev_status;
    p.n_rows = n_rows;
    p.n_cells = n_cells;
    p.n = n;
    p.half = rot / 2;
    p.pairs = rope->pairs;
    p.inverse = inverse;
    p.magnitude = rope->magnitude;
    for (int j = 0; j < rot / 2; ++j) p.turns[j] = rope->turns[j];
    // a row a CTA until every SM has several; then up to eight, which share a pass over the parameters
    int64_t rows = n_rows / (8 * (int64_t)device_sm_count());
    rows = rows < 1 ? 1 : rows > kMaxRows ? kMaxRows : rows;
    p.rows = (int)rows;
    const size_t smem = (size_t)rows * p.half * sizeof(float2);
    static_assert(kTableBytes <= 40 * 1024, "fits without a raised limit");
    if (launch_pdl(p.pairs ? rotate_rows_kernel<true> : rotate_rows_kernel<false>,
                   dim3((unsigned)((n_rows + rows - 1) / rows)), dim3(kThreads), smem, (cudaStream_t)stream, p) !=
        cudaSuccess) {
        cudaGetLastError();
        return SFA_ERR_CUDA;
    }
    return SFA_OK;
}
