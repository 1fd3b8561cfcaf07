// rotate.cu -- rotary positions of rows (sfa_rope_frequencies, sfa_rope_init, sfa_rotate_rows).
#include <math.h>

#include "sfa_common.cuh"

namespace sfa {
namespace {

constexpr int kThreads = 256;
constexpr int kTurns = 2048;       // of a block without 16-byte accesses: its rows times n_rot / 2

enum Kind { kBf16, kRound, kF32 };   // bf16 rows, fp32 into bf16, fp32 rows

struct Rotation {
    const void *src;
    void *dst;
    int64_t src_stride, src_head, dst_stride, dst_head;
    int kind, to_cells;
    int heads, begin;          // begin: first dim that turns
    int stay, lo;              // a head's units that stay, those before the turning ones (0: in place)
    FastDiv by_head, by_row;   // by stay, by heads * stay
    // 16-byte accesses: a row's `groups` threads have eight dims of the first half (or eight adjacent ones)
    // each, `subs` such teams every subs-th head; a block has `rows` rows
    int subs, rows;
    FastDiv by_team;           // by groups * subs
};
struct Params {
    Rotation r[SFA_MAX_ROTATIONS];
    const int32_t *pos, *slot;
    int32_t *status;
    int64_t n_rows, n_cells;
    int half;                  // pairs: n_rot / 2
    int groups;
    FastDiv by_groups;
    int pairs, inverse;
    float magnitude;
    uint64_t turns[SFA_MAX_ROT / 2];
};

// cos and sin of pos * f_j.  The product's low 64 bits are the fraction of a turn, as exact as the table's
// entry; what is left of the nearest quarter turn, at most an eighth, meets sinpi and cospi rounded to fp32.
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
// Where row i of a set goes, or -1: it is left out.
__device__ __forceinline__ int64_t target(const Params &p, const Rotation &r, int64_t i, int pos) {
    if (pos < 0) return -1;
    if (!r.to_cells) return i;
    const int c = p.slot[i];
    if (c >= p.n_cells) {
        set_status(p.status, SFA_DEV_BAD_CELL);
        return -1;
    }
    return c < 0 ? -1 : c;
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

// The rows of a block, where everything is aligned to 16 bytes.  A thread has the cosines and sines of its
// eight pairs (adjacent pairs: four) in registers and takes one head after the other, U of their loads in
// flight, the first ones before it makes the cosines: no thread waits for another.  Then the block's
// threads copy the dims that stay.
// The memory bounds it: 65536 rows of 20 heads of 128, bf16, 102 us (6.6 TB/s), 162 with the cosines of a
// block's rows in shared memory, made by all before any loads; 2048 rows of 17 heads, 64 of 576 dims turned,
// fp32 into bf16, 16.8 us, 30.4 so; 32 rows are latency, 2.5 us.
template <int KIND, bool PAIRS, int U>
__device__ __forceinline__ void rotate_vec(const Params &p, const Rotation &r, int64_t row0) {
    constexpr int NP = PAIRS ? 4 : 8;
    const int rows = (int)min((int64_t)r.rows, p.n_rows - row0), team = p.groups * r.subs;
    const int row = r.by_team.div(threadIdx.x), in = threadIdx.x - row * team;
    const int sub = p.by_groups.div(in), g = in - sub * p.groups;
    if (row < rows) {
        const int64_t i = row0 + row;
        const int pos = p.pos[i];
        const int64_t to = target(p, r, i, pos);
        const int dim = r.begin + g * 8;
        const int64_t from = i * r.src_stride + dim, at = to * r.dst_stride + dim;
        if (to >= 0) {
            float c[NP], s[NP];
            for (int h0 = sub; h0 < r.heads; h0 += U * r.subs) {
                Eight<KIND> a[U], b[PAIRS ? 1 : U];
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const int h = h0 + k * r.subs;
                    if (h >= r.heads) continue;
                    a[k].load(r.src, from + h * r.src_head);
                    if constexpr (!PAIRS) b[k].load(r.src, from + h * r.src_head + p.half);
                }
                if (h0 == sub) {
#pragma unroll
                    for (int x = 0; x < NP; ++x) {
                        const float2 cs = turn(p, pos, g * NP + x);
                        c[x] = cs.x;
                        s[x] = cs.y;
                    }
                }
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const int h = h0 + k * r.subs;
                    if (h >= r.heads) continue;
                    float f[8];
                    a[k].get(f);
                    if constexpr (PAIRS) {
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const float u = f[2 * x], v = f[2 * x + 1];
                            f[2 * x] = u * c[x] - v * s[x];
                            f[2 * x + 1] = u * s[x] + v * c[x];
                        }
                    } else {
                        float e[8];
                        b[k].get(e);
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
                            const float u = f[x], v = e[x];
                            f[x] = u * c[x] - v * s[x];
                            e[x] = u * s[x] + v * c[x];
                        }
                        b[k].put(e);
                        b[k].store(r.dst, at + h * r.dst_head + p.half);
                    }
                    a[k].put(f);
                    a[k].store(r.dst, at + h * r.dst_head);
                }
            }
        }
    }
    constexpr int C = 4;
    const int total = rows * r.heads * r.stay;
    for (int e0 = threadIdx.x; e0 < total; e0 += kThreads * C) {
        Eight<KIND> a[C];
        int64_t at[C];
#pragma unroll
        for (int k = 0; k < C; ++k) {
            const int e = e0 + k * kThreads;
            at[k] = -1;
            if (e >= total) continue;
            const int x = r.by_row.div(e), y = e - x * r.heads * r.stay, h = r.by_head.div(y), u = y - h * r.stay;
            const int64_t i = row0 + x, to = target(p, r, i, p.pos[i]);
            if (to < 0) continue;
            const int dim = 8 * u + (u < r.lo ? 0 : 2 * p.half);
            a[k].load(r.src, i * r.src_stride + h * r.src_head + dim);
            at[k] = to * r.dst_stride + h * r.dst_head + dim;
        }
#pragma unroll
        for (int k = 0; k < C; ++k) {
            if (at[k] < 0) continue;
            if constexpr (KIND == kRound) {
                float f[8];
                a[k].get(f);
                a[k].put(f);
            }
            a[k].store(r.dst, at[k]);
        }
    }
}

template <bool PAIRS, int U>
__global__ void __launch_bounds__(kThreads) rotate_rows_kernel(const __grid_constant__ Params p) {
    pdl_wait();
    const Rotation &r = p.r[blockIdx.y];
    const int64_t row0 = (int64_t)blockIdx.x * r.rows;
    if (row0 >= p.n_rows) return;
    if (r.kind == kBf16) rotate_vec<kBf16, PAIRS, U>(p, r, row0);
    else if (r.kind == kRound) rotate_vec<kRound, PAIRS, (U + 1) / 2>(p, r, row0);
    else rotate_vec<kF32, PAIRS, (U + 1) / 2>(p, r, row0);
}

__device__ __forceinline__ float load1(const void *base, int64_t e, int kind) {
    return kind == kBf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(base)[e])
                         : reinterpret_cast<const float *>(base)[e];
}
__device__ __forceinline__ void store1(void *base, int64_t e, int kind, float v) {
    if (kind == kF32) reinterpret_cast<float *>(base)[e] = v;
    else reinterpret_cast<__nv_bfloat16 *>(base)[e] = __float2bfloat16_rn(v);
}
// Rows of any alignment: a block has a few of them, their cosines and sines in shared memory, and then an
// element that stays or a pair at a time.
__global__ void __launch_bounds__(kThreads) rotate_any_kernel(const __grid_constant__ Params p) {
    __shared__ float2 sTurn[kTurns];   // [rows][half]
    pdl_wait();
    const Rotation &r = p.r[blockIdx.y];
    const int64_t row0 = (int64_t)blockIdx.x * r.rows;
    const int rows = (int)min((int64_t)r.rows, p.n_rows - row0);
    for (int e = threadIdx.x; e < rows * p.half; e += kThreads) {
        const int row = p.by_groups.div(e);
        sTurn[e] = turn(p, p.pos[row0 + row], e - row * p.half);
    }
    __syncthreads();
    const int units = p.half + r.stay;
    for (int row = 0; row < rows; ++row) {
        const int64_t i = row0 + row, d0 = target(p, r, i, p.pos[i]);
        if (d0 < 0) continue;
        for (int e = threadIdx.x; e < r.heads * units; e += kThreads) {
            const int h = r.by_head.div(e), y = e - h * units;
            const int64_t from = i * r.src_stride + h * r.src_head, to = d0 * r.dst_stride + h * r.dst_head;
            if (y < p.half) {
                const int a = r.begin + (p.pairs ? 2 * y : y), b = p.pairs ? a + 1 : a + p.half;
                const float2 cs = sTurn[row * p.half + y];
                const float f = load1(r.src, from + a, r.kind), g = load1(r.src, from + b, r.kind);
                store1(r.dst, to + a, r.kind, f * cs.x - g * cs.y);
                store1(r.dst, to + b, r.kind, f * cs.y + g * cs.x);
            } else {
                const int u = y - p.half, a = u + (u < r.lo ? 0 : 2 * p.half);
                if (r.kind == kBf16)   // bit for bit: a conversion would quiet a NaN
                    reinterpret_cast<uint16_t *>(r.dst)[to + a] = reinterpret_cast<const uint16_t *>(r.src)[from + a];
                else store1(r.dst, to + a, r.kind, reinterpret_cast<const float *>(r.src)[from + a]);
            }
        }
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
        // what is left of the nearest whole turn is exact, of either sign; -1/2 and 1/2 are the same
        const double t = freq[j] / 6.283185307179586476925, rest = t - nearbyint(t);
        const uint64_t u = (uint64_t)nearbyint(fabs(rest) * 0x1p64);
        rope->turns[j] = rest < 0. ? 0 - u : u;
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
    bool cells = false, vec = rot % (rope->pairs ? 8 : 16) == 0;
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
        vec = vec && aligned16(w.src) && aligned16(w.dst) && w.d % 8 == 0 && w.rot_begin % 8 == 0 &&
              far16(n_rows, w.src_stride, ss) && far16(w.to_cells ? n_cells : n_rows, w.dst_stride, ds) &&
              far16(w.n_heads, w.src_head_stride, ss) && far16(w.n_heads, w.dst_head_stride, ds);
        r.heads = w.n_heads;
        r.begin = w.rot_begin;
        r.lo = same ? 0 : w.rot_begin;
        r.stay = same ? 0 : w.d - rot;
    }
    if (n == 0 || n_rows == 0) return SFA_OK;
    if (!pos || (cells && !slot)) return SFA_ERR_INVALID_ARG;
    p.pos = pos;
    p.slot = cells ? slot : nullptr;
    p.status = dev_status;
    p.n_rows = n_rows;
    p.n_cells = n_cells;
    p.half = rot / 2;
    p.pairs = rope->pairs;
    p.inverse = inverse;
    p.magnitude = rope->magnitude;
    for (int j = 0; j < rot / 2; ++j) p.turns[j] = rope->turns[j];
    p.groups = vec ? (p.pairs ? rot / 8 : rot / 16) : p.half;
    p.by_groups.set(p.groups);
    // Four heads a thread, or one where that would leave threads of the device without any.
    int64_t threads = 0, blocks = 1;
    for (int k = 0; k < n; ++k) threads += n_rows * p.groups * p.r[k].heads;
    const int per = threads > 4 * 2048 * (int64_t)device_sm_count() ? 4 : 1;
    // few rows: a block on every SM before it has a second one
    const int few = n_rows >= kThreads * (int64_t)device_sm_count() ? kThreads
                    : n_rows > device_sm_count() ? (int)(n_rows / device_sm_count()) : 1;
    for (int k = 0; k < n; ++k) {
        Rotation &r = p.r[k];
        if (vec) {
            r.lo /= 8;
            r.stay /= 8;
            const int most = kThreads / p.groups;
            r.subs = (r.heads + per - 1) / per;
            if (r.subs > most) r.subs = most;
            r.rows = kThreads / (p.groups * r.subs);
            if (r.rows > few) r.rows = few;
            r.by_team.set(p.groups * r.subs);
            r.by_head.set(r.stay > 0 ? r.stay : 1);
            r.by_row.set(r.stay > 0 ? r.heads * r.stay : 1);
        } else {
            r.rows = kTurns / p.half < 8 ? kTurns / p.half : 8;
            r.by_head.set(p.half + r.stay);
        }
        const int64_t b = (n_rows + r.rows - 1) / r.rows;
        if (b > blocks) blocks = b;
    }
    auto kernel = !vec ? rotate_any_kernel
                  : per == 4 ? (p.pairs ? rotate_rows_kernel<true, 4> : rotate_rows_kernel<false, 4>)
                             : (p.pairs ? rotate_rows_kernel<true, 1> : rotate_rows_kernel<false, 1>);
    if (launch_pdl(kernel, dim3((unsigned)blocks, (unsigned)n), dim3(kThreads), 0, (cudaStream_t)stream, p) !=
        cudaSuccess) {
        cudaGetLastError();
        return SFA_ERR_CUDA;
    }
    return SFA_OK;
}
