// tree.cu -- drafted trees over a paged cache: their masks and positions (sfa_build_tree_maps), the path
// that the model agrees with (sfa_tree_accept), and what stays of it (sfa_tree_commit).
#include "sfa_common.cuh"

namespace sfa {
namespace {

// The tree of sequence s: its first row and its nodes.  Offsets that do not ascend within [0, n_rows] give
// an empty one.
struct Tree {
    int c0, n;
    bool bad;
};
__device__ __forceinline__ Tree load_tree(const int32_t *cu, int s, int64_t n_rows) {
    const int a = cu[s], b = cu[s + 1];
    Tree t;
    t.bad = a < 0 || b < a || b > n_rows;
    t.c0 = t.bad ? 0 : a;
    t.n = t.bad ? 0 : b - a;
    return t;
}

// ------------------------------------------------------------------------------------ tree maps
constexpr int kMapThreads = 128;

struct MapParams {
    const int32_t *parent, *cu, *total;
    uint32_t *mask;
    int32_t *q_pos, *cached_pos, *status;
    int64_t n_rows;
    int n_seq, words;
    FastDiv by_words;
};

// One CTA a tree, 32 nodes at a time: a thread has one word of one node's mask.  It goes up from the node
// to the first ancestor of an earlier group, whose mask is whole: at most 32 steps, and as a rule a
// tree's few levels.
__global__ void __launch_bounds__(kMapThreads) tree_maps_kernel(const MapParams p) {
    __shared__ int16_t sParent[SFA_MAX_TREE], sDepth[SFA_MAX_TREE];
    pdl_wait();
    const int tid = threadIdx.x;
    const int s = blockIdx.x;
    if (s < p.n_seq) {
        const Tree t = load_tree(p.cu, s, p.n_rows);
        int flags = t.bad ? SFA_DEV_BAD_QUERY : 0;
        const int total = p.total[s];
        if (total < t.n) flags |= SFA_DEV_BAD_QUERY;
        const int a = max(total - t.n, 0);
        const int n = min(t.n, 32 * p.words);
        if (n < t.n) flags |= SFA_DEV_BAD_TREE;
        for (int j = tid; j < n; j += kMapThreads) {
            int up = p.parent[t.c0 + j];
            if (up < -1 || up >= j) {
                flags |= SFA_DEV_BAD_TREE;
                up = -1;
            }
            sParent[j] = (int16_t)up;
        }
        __syncthreads();
        for (int g = 0; g < n; g += 32) {
            for (int e = tid; e < 32 * p.words; e += kMapThreads) {
                const int k = p.by_words.div(e), w = e - k * p.words, j = g + k;
                if (j >= n) break;
                uint32_t bits = 0;
                int cur = j, steps = 0;
                for (; cur >= g; cur = sParent[cur], ++steps) bits |= 1u << (cur & 31);
                if (w != g >> 5) bits = 0;
                const int64_t row = t.c0 + j;
                if (cur >= 0) bits |= p.mask[(int64_t)(t.c0 + cur) * p.words + w];
                p.mask[row * p.words + w] = bits;
                if (w == 0) {
                    const int depth = steps + (cur >= 0 ? sDepth[cur] : -1);
                    sDepth[j] = (int16_t)depth;
                    p.q_pos[row] = (int)min((int64_t)a + depth, (int64_t)0x7FFFFFFF);
                    if (p.cached_pos) p.cached_pos[row] = a - 1;
                }
            }
            __syncthreads();
        }
        for (int64_t e = (int64_t)n * p.words + tid; e < (int64_t)t.n * p.words; e += kMapThreads)
            p.mask[(int64_t)t.c0 * p.words + e] = 0;
        for (int j = n + tid; j < t.n; j += kMapThreads) {
            p.q_pos[t.c0 + j] = -1;
            if (p.cached_pos) p.cached_pos[t.c0 + j] = -1;
        }
        if (flags) set_status(p.status, flags);
    }
    // padding, a share of each CTA
    const int64_t end = p.n_seq > 0 ? min(max((int64_t)p.cu[p.n_seq], (int64_t)0), p.n_rows) : 0;
    const int64_t step = (int64_t)gridDim.x * kMapThreads, at = (int64_t)s * kMapThreads + tid;
    for (int64_t e = end * p.words + at; e < p.n_rows * p.words; e += step) p.mask[e] = 0;
    for (int64_t i = end + at; i < p.n_rows; i += step) {
        p.q_pos[i] = -1;
        if (p.cached_pos) p.cached_pos[i] = -1;
    }
}

// --------------------------------------------------------------------------------------- accept
struct AcceptParams {
    const int32_t *parent, *token, *target, *root_target, *cu;
    int32_t *path, *n_acc, *next, *status;
    int64_t n_rows, path_stride;
    int n_seq;
};

// One warp a tree.  Its nodes go to shared memory at once; then each step is a look at 32 nodes at a time
// from behind the last accepted one on.
__global__ void __launch_bounds__(32) tree_accept_kernel(const AcceptParams p) {
    __shared__ int32_t sParent[SFA_MAX_TREE], sToken[SFA_MAX_TREE], sTarget[SFA_MAX_TREE];
    pdl_wait();
    const int s = blockIdx.x, lane = threadIdx.x;
    const Tree t = load_tree(p.cu, s, p.n_rows);
    const int n = min(t.n, SFA_MAX_TREE);
    int flags = (t.bad ? SFA_DEV_BAD_QUERY : 0) | (n < t.n ? SFA_DEV_BAD_TREE : 0);
    const int root = p.root_target ? p.root_target[s] : 0;
    for (int j0 = lane; j0 < n; j0 += 64) {   // two nodes' loads in flight
        int v[2][3];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int j = j0 + 32 * x;
            if (j < n) {
                v[x][0] = p.parent[t.c0 + j];
                v[x][1] = p.token[t.c0 + j];
                v[x][2] = p.target[t.c0 + j];
            }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int j = j0 + 32 * x;
            if (j < n) {
                if (v[x][0] < -1 || v[x][0] >= j) {
                    flags |= SFA_DEV_BAD_TREE;
                    v[x][0] = -2;
                }
                sParent[j] = v[x][0];
                sToken[j] = v[x][1];
                sTarget[j] = v[x][2];
            }
        }
    }
    __syncwarp();
    int32_t *path = p.path + (int64_t)s * p.path_stride;
    int cur = -1, want = root;
    bool any = !p.root_target;
    int64_t k = 0;
    while (k < p.path_stride) {
        int hit = -1;
        for (int c0 = cur + 1; c0 < n && hit < 0; c0 += 32) {
            const int c = c0 + lane;
            const bool on = c < n && sParent[c] == cur && (any || sToken[c] == want);
            const unsigned all = __ballot_sync(0xFFFFFFFFu, on);
            if (all) hit = c0 + __ffs(all) - 1;
        }
        if (hit < 0) break;
        if (lane == 0) path[k] = hit;
        cur = hit;
        want = sTarget[hit];
        any = false;
        ++k;
    }
    for (int64_t i = k + lane; i < p.path_stride; i += 32) path[i] = -1;
    if (lane == 0) {
        p.n_acc[s] = (int)k;
        p.next[s] = k > 0 ? want : p.root_target ? root : -1;
    }
    if (flags) set_status(p.status, flags);
}

// --------------------------------------------------------------------------------------- commit
constexpr int kCommitThreads = 512;
constexpr int kAhead = 8;   // rows of a path in flight

struct CommitParams {
    uint8_t *rows[SFA_MAX_CELL_WRITES];
    int64_t row_bytes[SFA_MAX_CELL_WRITES];
    int unit[SFA_MAX_CELL_WRITES];          // bytes of a column: 16, or 2
    int col0[SFA_MAX_CELL_WRITES + 1];      // first column of each cache
    const int32_t *slot, *cu, *total, *path, *n_acc, *table, *head;
    int32_t *free_pages, *len_out, *head_out, *status;
    int64_t n_rows, n_cells, path_stride, table_stride, n_free;
    FastDiv page_div;
    int n, n_seq, page, n_pages;
};

// The accepted length that a path can have: at most its row, its tree and n_acc.
__device__ __forceinline__ int path_limit(const CommitParams &p, int s, const Tree &t, bool &bad) {
    const int m = p.n_acc[s];
    int64_t most = t.n;
    if (p.path_stride < most) most = p.path_stride;
    bad = m < 0 || m > most;
    return m < 0 ? 0 : m > most ? (int)most : m;
}
// Entries k0 .. of a path, those from `limit` on left out.
__device__ __forceinline__ void load_path(const CommitParams &p, int s, int k0, int limit, int (&x)[kAhead]) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) x[i] = k0 + i < limit ? p.path[(int64_t)s * p.path_stride + k0 + i] : -1;
}

// The free list, the lengths and the head, by one CTA: a thread has neighbouring sequences, a prefix sum of
// the pages they give back says where theirs go.
__device__ __forceinline__ void commit_lists(const CommitParams &p) {
    __shared__ int64_t s_warp[kCommitThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.n_seq + kCommitThreads - 1) / kCommitThreads;
    const int s0 = min(tid * per, p.n_seq), s1 = min(s0 + per, p.n_seq);
    int flags = 0;
    // length of sequence s afterwards, and the table entries [k0, k1) that it gives back
    auto after = [&](int s, int &k0, int &k1) {
        const Tree t = load_tree(p.cu, s, p.n_rows);
        const int held = p.total[s], total = max(held, 0);
        bool bad;
        const int most = path_limit(p, s, t, bad);
        const bool gone = t.n > 0 && held == 0;   // emptied since its tree was drafted
        const int limit = gone ? 0 : most;
        if (!gone && (t.bad || held < t.n)) flags |= SFA_DEV_BAD_QUERY;
        int m = 0, last = -1;
        for (int k = 0; k < limit && m == k; k += kAhead) {
            int x[kAhead];
            load_path(p, s, k, limit, x);
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (m == k + i && k + i < limit && x[i] > last && x[i] < t.n) {
                    last = x[i];
                    ++m;
                }
        }
        if (!gone && (bad || m < limit)) flags |= SFA_DEV_BAD_TREE;
        const int len = max(total - t.n, 0) + m;
        auto pages = [&](int n) { return n > 0 ? p.page_div.div(n - 1) + 1 : 0; };
        k0 = pages(len);
        k1 = (int)min((int64_t)pages(total), p.table_stride);
        return len;
    };
    auto is_page = [&](int s, int k) {
        const int e = p.table[(int64_t)s * p.table_stride + k];
        return e >= 0 && e < p.n_pages ? e : -1;
    };
    int64_t back = 0;
    for (int s = s0; s < s1; ++s) {
        int k0, k1;
        after(s, k0, k1);
        for (int k = k0; k < k1; ++k) back += is_page(s, k) >= 0;
    }
    int64_t x = back;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    const int64_t head = min(max((int64_t)*p.head, (int64_t)0), p.n_free);
    __syncthreads();
    int64_t before = 0, all = 0;
    for (int w = 0; w < kCommitThreads / 32; ++w) {
        if (w < warp) before += s_warp[w];
        all += s_warp[w];
    }
    int64_t at = head - all + before + x - back;
    for (int s = s0; s < s1; ++s) {
        int k0, k1;
        const int len = after(s, k0, k1);
        for (int k = k0; k < k1; ++k) {
            const int e = is_page(s, k);
            if (e < 0) continue;
            if (at >= 0) p.free_pages[at] = e;
            ++at;
        }
        p.len_out[s] = len;
    }
    if (tid == 0) {
        *p.head_out = (int32_t)max(head - all, (int64_t)0);
        if (head < all) flags |= SFA_DEV_BAD_LENGTH;   // more pages than were ever taken
    }
    if (flags) set_status(p.status, flags);
}

template <typename T>
__device__ __forceinline__ void commit_column(const CommitParams &p, int s, const Tree &t, int limit, T *base, int64_t pitch) {
    int last = -1;
    for (int k = 0; k < limit; k += kAhead) {
        int x[kAhead];
        load_path(p, s, k, limit, x);
        int64_t from[kAhead], to[kAhead];
        bool ended = false;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            from[i] = to[i] = -1;
            ended = ended || k + i >= limit || x[i] <= last || x[i] >= t.n;
            if (ended) continue;
            last = x[i];
            if (x[i] == k + i) continue;   // in place
            const int a = p.slot[t.c0 + x[i]], b = p.slot[t.c0 + k + i];
            if (a < 0 || b < 0 || a >= p.n_cells || b >= p.n_cells) {
                set_status(p.status, SFA_DEV_BAD_CELL);
                continue;
            }
            from[i] = a;
            to[i] = b;
        }
        T v[kAhead];
        // a path's nodes ascend, so no later row comes from a cell that an earlier one goes to, and within
        // a group everything is read first
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (from[i] >= 0) v[i] = base[from[i] * pitch];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (from[i] >= 0) base[to[i] * pitch] = v[i];
        if (ended) break;
    }
}

// CTA 0: the lists; the others: a thread has one column of one sequence's rows, so that rows move down the
// path in order with nobody to wait for.
__global__ void __launch_bounds__(kCommitThreads) tree_commit_kernel(const __grid_constant__ CommitParams p) {
    pdl_wait();
    if (blockIdx.x == 0) return commit_lists(p);
    const int cols = p.col0[p.n];
    const int64_t items = (int64_t)cols * p.n_seq;
    for (int64_t e = (int64_t)(blockIdx.x - 1) * kCommitThreads + threadIdx.x; e < items;
         e += (int64_t)(gridDim.x - 1) * kCommitThreads) {
        const int s = (int)(e / cols), col = (int)(e - (int64_t)s * cols);
        const Tree t = load_tree(p.cu, s, p.n_rows);
        bool bad;
        const int limit = path_limit(p, s, t, bad);
        int c = 0;
#pragma unroll
        for (int i = 1; i < SFA_MAX_CELL_WRITES; ++i)
            if (i < p.n && col >= p.col0[i]) c = i;
        uint8_t *at = p.rows[c] + (int64_t)(col - p.col0[c]) * p.unit[c];
        if (p.unit[c] == 16) commit_column(p, s, t, limit, reinterpret_cast<uint4 *>(at), p.row_bytes[c] / 16);
        else commit_column(p, s, t, limit, reinterpret_cast<uint16_t *>(at), p.row_bytes[c] / 2);
    }
}

}  // namespace
}  // namespace sfa

extern "C" int sfa_build_tree_maps(const int32_t *parent, const int32_t *cu_new, const int32_t *len_total,
                                   int n_seq, int64_t n_rows, uint32_t *mask, int mask_words, int32_t *q_pos,
                                   int32_t *cached_pos, int32_t *dev_status, sfa_stream_t stream) {
    using namespace sfa;
    if (n_seq < 0 || n_rows < 0 || n_rows > 0x7FFFFFFF || mask_words < 1) return SFA_ERR_INVALID_ARG;
    if (mask_words > SFA_MAX_TREE / 32) return SFA_ERR_UNSUPPORTED;
    if (n_rows == 0) return SFA_OK;
    if (!mask || !q_pos || (n_seq > 0 && (!parent || !cu_new || !len_total))) return SFA_ERR_INVALID_ARG;
    MapParams p{};
    p.parent = parent;
    p.cu = cu_new;
    p.total = len_total;
    p.mask = mask;
    p.q_pos = q_pos;
    p.cached_pos = cached_pos;
    p.status = dev_status;
    p.n_rows = n_rows;
    p.n_seq = n_seq;
    p.words = mask_words;
    p.by_words.set(mask_words);
    if (launch_pdl(tree_maps_kernel, dim3(n_seq > 0 ? n_seq : 1), dim3(kMapThreads), 0, (cudaStream_t)stream, p) !=
        cudaSuccess) {
        cudaGetLastError();
        return SFA_ERR_CUDA;
    }
    return SFA_OK;
}

extern "C" int sfa_tree_accept(const int32_t *parent, const int32_t *token, const int32_t *target,
                               const int32_t *root_target, const int32_t *cu_new, int n_seq, int64_t n_rows,
                               int32_t *path, int64_t path_stride, int32_t *n_acc, int32_t *next_token,
                               int32_t *dev_status, sfa_stream_t stream) {
    using namespace sfa;
    if (n_seq < 0 || n_rows < 0 || n_rows > 0x7FFFFFFF || path_stride < 1 || path_stride > 0x7FFFFFFF)
        return SFA_ERR_INVALID_ARG;
    if (n_seq == 0) return SFA_OK;
    if (!cu_new || !path || !n_acc || !next_token || (n_rows > 0 && (!parent || !token || !target)))
        return SFA_ERR_INVALID_ARG;
    AcceptParams p{};
    p.parent = parent;
    p.token = token;
    p.target = target;
    p.root_target = root_target;
    p.cu = cu_new;
    p.path = path;
    p.n_acc = n_acc;
    p.next = next_token;
    p.status = dev_status;
    p.n_rows = n_rows;
    p.path_stride = path_stride;
    p.n_seq = n_seq;
    if (launch_pdl(tree_accept_kernel, dim3(n_seq), dim3(32), 0, (cudaStream_t)stream, p) != cudaSuccess) {
        cudaGetLastError();
        return SFA_ERR_CUDA;
    }
    return SFA_OK;
}

extern "C" int sfa_tree_commit(int n, const sfa_cell_rows *caches, int64_t n_cells, const int32_t *slot,
                               const int32_t *cu_new, const int32_t *len_total, int n_seq, int64_t n_rows,
                               const int32_t *path, int64_t path_stride, const int32_t *n_acc, int page_size,
                               const int32_t *page_table, int64_t table_stride, int32_t *free_pages,
                               int64_t n_free, const int32_t *free_head, int32_t *len_out,
                               int32_t *free_head_out, int32_t *dev_status, sfa_stream_t stream) {
    using namespace sfa;
    if (n < 0 || n > SFA_MAX_CELL_WRITES || (n > 0 && !caches) || n_cells < 0 || n_cells > 0x7FFFFFFF || n_seq < 0 ||
        n_rows < 0 || n_rows > 0x7FFFFFFF || path_stride < 1 || path_stride > 0x7FFFFFFF || page_size < 1 ||
        table_stride < 0 || table_stride > 0x7FFFFFFF || table_stride * page_size > 0x7FFFFFFF || n_free < 0 ||
        n_free > 0x7FFFFFFF)
        return SFA_ERR_INVALID_ARG;
    CommitParams p{};
    for (int k = 0; k < n; ++k) {
        const sfa_cell_rows &c = caches[k];
        if (!c.rows || !aligned16(c.rows) || c.row_bytes < 2 || c.row_bytes % 2 != 0 || c.row_bytes > (1 << 24))
            return SFA_ERR_INVALID_ARG;
        p.rows[k] = reinterpret_cast<uint8_t *>(c.rows);
        p.row_bytes[k] = c.row_bytes;
        p.unit[k] = c.row_bytes % 16 == 0 ? 16 : 2;
        p.col0[k + 1] = p.col0[k] + (int)(c.row_bytes / p.unit[k]);
    }
    if (!free_head || !free_head_out || (n_free > 0 && !free_pages)) return SFA_ERR_INVALID_ARG;
    if (n_seq > 0 && (!cu_new || !len_total || !path || !n_acc || !len_out || (table_stride > 0 && !page_table) ||
                      (n_rows > 0 && !slot)))
        return SFA_ERR_INVALID_ARG;
    p.slot = slot;
    p.cu = cu_new;
    p.total = len_total;
    p.path = path;
    p.n_acc = n_acc;
    p.table = page_table;
    p.head = free_head;
    p.free_pages = free_pages;
    p.len_out = len_out;
    p.head_out = free_head_out;
    p.status = dev_status;
    p.n_rows = n_rows;
    p.n_cells = n_cells;
    p.path_stride = path_stride;
    p.table_stride = table_stride;
    p.n_free = n_free;
    p.page_div.set(page_size);
    p.n = n;
    p.n_seq = n_seq;
    p.page = page_size;
    p.n_pages = (int)(n_cells / page_size);
    const int64_t items = (int64_t)p.col0[n] * n_seq, most = 4 * (int64_t)device_sm_count();
    int64_t blocks = (items + kCommitThreads - 1) / kCommitThreads;
    if (blocks > most) blocks = most;
    if (launch_pdl(tree_commit_kernel, dim3((unsigned)(1 + blocks)), dim3(kCommitThreads), 0, (cudaStream_t)stream, p) !=
        cudaSuccess) {
        cudaGetLastError();
        return SFA_ERR_CUDA;
    }
    return SFA_OK;
}
