// Drafted trees: their layout (positions, ancestor words) and the commit of an accepted path.
//
// Both move a few integers or a few KB per request, so latency bounds them.  The layout takes
// the ancestors by pointer doubling (six rounds for 64 nodes) instead of walking each node's path.
// Measured: the layout 2 us, the commit of five tokens to one layer 5 us, of 32 layers x 32 requests (37 MB read and written) 10 us.
#include "msa_device.cuh"
#include "msa_internal.h"

namespace msa {
namespace {

// The rows of no request, by one CTA: those behind the last request, or, where a range is refused (they may then
// overlap or leave gaps anywhere), every row that no good range holds, found through a bitmap of them.
__device__ __forceinline__ void pad_rows(const int32_t *__restrict__ node_off, int n_rows, int n_req,
                                         int32_t *__restrict__ q_req, int32_t *__restrict__ q_pos,
                                         uint64_t *__restrict__ anc) {
    constexpr int kWindow = 32768;   // rows looked at together
    __shared__ uint32_t held[kWindow / 32];
    const int i = threadIdx.x;
    int r0, r1;
    bool bad = false;
    for (int x = i; x < n_req; x += kTreeMaxNodes) bad |= tree_range(node_off, x, n_rows, &r0, &r1) != 0;
    bad = __syncthreads_or(bad);
    // (without a bad range node_off rises from 0 to n_rows at most)
    for (long long w0 = bad ? 0 : node_off[n_req]; w0 < n_rows; w0 += kWindow) {
        const int rows = int(min((long long)kWindow, n_rows - w0));
        if (bad) {
            for (int x = i; x < kWindow / 32; x += kTreeMaxNodes) held[x] = 0;
            __syncthreads();
            for (int x = i; x < n_req; x += kTreeMaxNodes) {
                if (tree_range(node_off, x, n_rows, &r0, &r1)) continue;
                const int lo = int(max(0LL, r0 - w0)), hi = int(min((long long)rows, r1 - w0));
                for (int r = lo; r < hi; ++r) atomicOr(&held[r >> 5], 1u << (r & 31));
            }
            __syncthreads();
        }
        for (int r = i; r < rows; r += kTreeMaxNodes) {
            if (bad && (held[r >> 5] >> (r & 31) & 1)) continue;
            q_req[w0 + r] = -1;
            q_pos[w0 + r] = 0;
            anc[w0 + r] = 0;
        }
        __syncthreads();
    }
}

// CTA b < n_req: request b, one thread per node.  CTA n_req: the padding rows.
__global__ void __launch_bounds__(kTreeMaxNodes) k_tree_rows(
    const int32_t *__restrict__ node_off, const int32_t *__restrict__ parents, const int32_t *__restrict__ ctx_lens,
    int n_rows, int n_req, int max_blocks, int32_t *__restrict__ q_req, int32_t *__restrict__ q_pos,
    uint64_t *__restrict__ anc, int32_t *err) {
    __shared__ unsigned long long mask_s[kTreeMaxNodes];
    __shared__ int up_s[kTreeMaxNodes];
    const int b = blockIdx.x, i = threadIdx.x;
    pdl_trigger();
    if (b == n_req) {
        pad_rows(node_off, n_rows, n_req, q_req, q_pos, anc);
        return;
    }
    int row0;
    const int n = tree_rows_of(node_off, b, n_rows, err, i == 0, &row0);
    if (n == 0) return;   // no rows, or those of a refused request: padding
    // up: the node that this node's word reaches next (itself at the root)
    const int p = i < n ? parents[row0 + i] : 0;
    bool bad = i < n && (i == 0 ? p != -1 : (p < 0 || p >= i));
    int up = bad || i >= n || i == 0 ? i : p;
    unsigned long long mask = 1ull << i;
    mask_s[i] = mask;
    up_s[i] = up;
    __syncthreads();
#pragma unroll
    for (int round = 0; round < 6; ++round) {
        mask |= mask_s[up];
        up = up_s[up];
        __syncthreads();
        mask_s[i] = mask;
        up_s[i] = up;
        __syncthreads();
    }
    const long long ctx = ctx_lens[b];
    const long long pos = ctx + __popcll(mask) - 1;
    bad = bad || (i < n && (ctx < 0 || (pos >> 7) >= max_blocks));
    bad = __syncthreads_or(bad);
    if (bad && i == 0) raise_flag(err, MSA_FLAG_BOUNDS);
    if (i < n) {
        q_req[row0 + i] = bad ? -1 : b;
        q_pos[row0 + i] = bad ? 0 : int(pos);
        anc[row0 + i] = bad ? 0ull : mask;
    }
}

// 16-byte chunks of one token in K, V and the k-index, all groups: 2 * kv + ix.
__global__ void __launch_bounds__(256) k_commit_tree(
    const uint4 *__restrict__ k_new, const uint4 *__restrict__ v_new, const uint4 *__restrict__ ix_new,
    uint4 *__restrict__ k_cache, uint4 *__restrict__ v_cache, uint4 *__restrict__ ix_cache,
    const int32_t *__restrict__ block_table, const int32_t *__restrict__ ctx_lens,
    const int32_t *__restrict__ node_off, const int32_t *__restrict__ path, const int32_t *__restrict__ n_acc,
    int n_rows, int n_pages, int max_blocks, int kv, int ix, int32_t *__restrict__ new_lens, int32_t *err) {
    __shared__ long long src_s[kTreeMaxNodes];   // row of the k-th accepted node, -1: not written
    __shared__ long long dst_s[kTreeMaxNodes];   // its slot in the page pool (page * 128 + offset)
    const int b = blockIdx.x, layer = blockIdx.y, tid = threadIdx.x;
    const bool report = layer == 0;   // flags and lengths: one layer's CTA
    int row0;
    const int n = tree_rows_of(node_off, b, n_rows, err, report && tid == 0, &row0);
    int acc = n_acc[b];
    const int ctx = ctx_lens[b];
    if (acc < 0 || acc > n || ctx < 0) {
        if (report && tid == 0) raise_flag(err, MSA_FLAG_BOUNDS);
        acc = 0;
    }
    if (tid < acc) {
        const int node = path[row0 + tid];
        const long long pos = (long long)ctx + tid;
        int page = -1;
        if (node >= 0 && node < n && (pos >> 7) < max_blocks) page = block_table[size_t(b) * max_blocks + (pos >> 7)];
        const bool ok = page >= 0 && page < n_pages;
        if (!ok && report) raise_flag(err, MSA_FLAG_BOUNDS);
        src_s[tid] = ok ? row0 + node : -1;
        dst_s[tid] = (long long)page * 128 + (pos & 127);
    }
    if (report && tid == 0) new_lens[b] = ctx + acc;
    __syncthreads();
    const int per = 2 * kv + ix;
    const size_t new_kv = size_t(layer) * n_rows * kv, new_ix = size_t(layer) * n_rows * ix;
    const size_t pool_kv = size_t(layer) * n_pages * 128 * kv, pool_ix = size_t(layer) * n_pages * 128 * ix;
    // where 16-byte chunk i of the accepted tokens comes from and goes to; null: not written
    auto chunk = [&](int i, const uint4 *&from, uint4 *&to) {
        from = nullptr;
        if (i >= acc * per) return;
        const int t = i / per, c = i - t * per;
        const long long src = src_s[t], dst = dst_s[t];
        if (src < 0) return;
        if (c < kv) {
            from = k_new + new_kv + size_t(src) * kv + c;
            to = k_cache + pool_kv + size_t(dst) * kv + c;
        } else if (c < 2 * kv) {
            from = v_new + new_kv + size_t(src) * kv + c - kv;
            to = v_cache + pool_kv + size_t(dst) * kv + c - kv;
        } else {
            from = ix_new + new_ix + size_t(src) * ix + c - 2 * kv;
            to = ix_cache + pool_ix + size_t(dst) * ix + c - 2 * kv;
        }
    };
    // four loads in flight per thread: one at a time, a layer's few tokens take several times the latency
    for (int i = tid; i < acc * per; i += 4 * 256) {
        const uint4 *from[4];
        uint4 *to[4], v[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            chunk(i + x * 256, from[x], to[x]);
            if (from[x]) v[x] = __ldg(from[x]);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x)
            if (from[x]) *to[x] = v[x];
    }
}

}  // namespace

cudaError_t launch_tree_rows(const int32_t *node_off, const int32_t *parents, const int32_t *ctx_lens, int n_rows,
                             int n_req, int max_blocks, int32_t *q_req, int32_t *q_pos, uint64_t *anc, int32_t *err,
                             cudaStream_t st) {
    k_tree_rows<<<unsigned(n_req) + 1, kTreeMaxNodes, 0, st>>>(node_off, parents, ctx_lens, n_rows, n_req, max_blocks,
                                                               q_req, q_pos, anc, err);
    return cudaGetLastError();
}

cudaError_t launch_commit_tree(const void *k_new, const void *v_new, const void *kidx_new, int n_layers, void *k_cache,
                               void *v_cache, void *kidx_cache, const int32_t *block_table, const int32_t *ctx_lens,
                               const int32_t *node_off, const int32_t *path, const int32_t *n_acc, int n_rows,
                               int n_req, int n_pages, const Shape &s, int32_t *new_lens, int32_t *err,
                               cudaStream_t st) {
    const dim3 grid(static_cast<unsigned>(n_req), static_cast<unsigned>(n_layers));
    k_commit_tree<<<grid, 256, 0, st>>>(
        static_cast<const uint4 *>(k_new), static_cast<const uint4 *>(v_new), static_cast<const uint4 *>(kidx_new),
        static_cast<uint4 *>(k_cache), static_cast<uint4 *>(v_cache), static_cast<uint4 *>(kidx_cache), block_table,
        ctx_lens, node_off, path, n_acc, n_rows, n_pages, s.max_blocks, s.G * s.D / 8, s.G * s.Di / 8, new_lens, err);
    return cudaGetLastError();
}

}  // namespace msa
