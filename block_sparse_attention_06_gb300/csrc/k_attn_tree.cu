// Sparse attention of drafted trees over the paged cache.
//
// Row r of group g attends, with one softmax, the cached tokens of its selected blocks and those of
// its ancestors (and itself) whose block is selected:
//   o = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m),  s_t = sm_scale * q . k_t,  m = max_t s_t.
// One CTA per (row, group), one thread per token of a 128-token block, an online softmax over blocks.
#include "msa_device.cuh"
#include "msa_internal.h"

namespace msa {
namespace {

template <int D, int HPG>
__global__ void __launch_bounds__(128) k_attn_tree(
    const uint16_t *__restrict__ q, const uint16_t *__restrict__ k_cache, const uint16_t *__restrict__ v_cache,
    const uint16_t *__restrict__ k_new, const uint16_t *__restrict__ v_new, const int32_t *__restrict__ block_table,
    const int32_t *__restrict__ ctx_lens, const int32_t *__restrict__ node_off, const uint64_t *__restrict__ anc,
    const int32_t *__restrict__ sel, int n_rows, int n_req, int n_pages, int G, int topk, int max_blocks,
    float sm_scale, uint16_t *__restrict__ out, float *__restrict__ lse, int32_t *err) {
    __shared__ float q_s[HPG][D], p_s[HPG][128], red[HPG][4];
    __shared__ uint8_t see_s[128];
    const int r = blockIdx.x / G, g = blockIdx.x % G, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int lo = 0, hi = n_req;   // the request: the last b with node_off[b] <= r
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (node_off[mid + 1] <= r) lo = mid + 1;
        else hi = mid;
    }
    if (lo >= n_req) return;   // padding
    int row0;
    const int b = lo, n = tree_rows_of(node_off, b, n_rows, err, tid == 0, &row0);
    if (r < row0 || r >= row0 + n) return;
    const int ctx = ctx_lens[b];
    if (ctx < 0) {
        if (tid == 0) raise_flag(err, MSA_FLAG_BOUNDS);
        return;
    }
    for (int i = tid; i < HPG * D; i += 128)
        q_s[i / D][i % D] = bf16_lo(q[(size_t(r) * G + g) * HPG * D + i]);
    const uint64_t path = anc[r];
    const int32_t *srow = sel + (size_t(r) * G + g) * topk;
    constexpr int PER = HPG * D / 128;   // outputs per thread: column d, heads h0, h0 + step, ...
    const int d = tid % D, h0 = tid / D;
    constexpr int STEP = 128 / D;
    float o[PER], m[HPG], l[HPG];
#pragma unroll
    for (int i = 0; i < PER; ++i) o[i] = 0.f;
#pragma unroll
    for (int h = 0; h < HPG; ++h) m[h] = -INFINITY, l[h] = 0.f;
    __syncthreads();
    for (int x = 0; x <= topk; ++x) {   // the selected blocks, then the drafted tokens
        const uint16_t *kb = nullptr, *vb = nullptr;
        bool see = false;
        if (x < topk) {
            const int j = srow[x];
            if (j < 0) continue;
            if (j >= max_blocks) {
                if (tid == 0) raise_flag(err, MSA_FLAG_BOUNDS);
                continue;
            }
            if (j * 128 >= ctx) continue;
            const int page = block_table[size_t(b) * max_blocks + j];
            if (page < 0 || page >= n_pages) {
                if (tid == 0) raise_flag(err, MSA_FLAG_BOUNDS);
                continue;
            }
            see = j * 128 + tid < ctx;
            kb = k_cache + (size_t(page) * 128 * G + g) * D;
            vb = v_cache + (size_t(page) * 128 * G + g) * D;
        } else {
            if (tid < n && (path >> tid & 1)) {
                const int blk = (ctx + __popcll(anc[row0 + tid]) - 1) >> 7;
                for (int s = 0; s < topk; ++s) see = see || srow[s] == blk;
            }
            kb = k_new + (size_t(row0) * G + g) * D;
            vb = v_new + (size_t(row0) * G + g) * D;
        }
        float s[HPG];
#pragma unroll
        for (int h = 0; h < HPG; ++h) s[h] = 0.f;
        if (see) {
            const uint16_t *kt = kb + size_t(tid) * G * D;
            for (int c = 0; c < D; c += 8) {
                const uint4 w = *reinterpret_cast<const uint4 *>(kt + c);
                const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int h = 0; h < HPG; ++h) {
                        s[h] = fmaf(q_s[h][c + 2 * e], bf16_lo(ws[e]), s[h]);
                        s[h] = fmaf(q_s[h][c + 2 * e + 1], bf16_hi(ws[e]), s[h]);
                    }
            }
        }
        see_s[tid] = see;
#pragma unroll
        for (int h = 0; h < HPG; ++h) {
            s[h] = see ? s[h] * sm_scale : -INFINITY;
            float v = s[h];
            for (int off = 16; off; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
            if (lane == 0) red[h][warp] = v;
        }
        __syncthreads();
        float alpha[HPG];
#pragma unroll
        for (int h = 0; h < HPG; ++h) {
            const float mn = fmaxf(m[h], fmaxf(fmaxf(red[h][0], red[h][1]), fmaxf(red[h][2], red[h][3])));
            alpha[h] = mn == -INFINITY ? 1.f : expf(m[h] - mn);
            m[h] = mn;
            p_s[h][tid] = see ? expf(s[h] - mn) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int h = 0; h < HPG; ++h) l[h] *= alpha[h];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            float a = 1.f;
#pragma unroll
            for (int h = 0; h < HPG; ++h) a = h == h0 + i * STEP ? alpha[h] : a;
            o[i] *= a;
        }
        for (int t = 0; t < 128; ++t) {
            if (!see_s[t]) continue;
            const float v = bf16_lo(vb[size_t(t) * G * D + d]);
#pragma unroll
            for (int i = 0; i < PER; ++i) o[i] = fmaf(p_s[h0 + i * STEP][t], v, o[i]);
#pragma unroll
            for (int h = 0; h < HPG; ++h) l[h] += p_s[h][t];
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int h = h0 + i * STEP;
        float lh = 0.f, mh = 0.f;
#pragma unroll
        for (int e = 0; e < HPG; ++e)
            if (e == h) lh = l[e], mh = m[e];
        const size_t row = (size_t(r) * G + g) * HPG + h;
        out[row * D + d] = uint16_t(pack_bf16x2(lh > 0.f || lh != lh ? o[i] / lh : 0.f, 0.f) & 0xffffu);
        if (d == 0) lse[row] = lh > 0.f || lh != lh ? mh + logf(lh) : -INFINITY;
    }
}

template <int D, int HPG>
cudaError_t launch_t(const void *q, const void *k_cache, const void *v_cache, const void *k_new, const void *v_new,
                     const int32_t *bt, const int32_t *ctx, const int32_t *node_off, const uint64_t *anc,
                     const int32_t *sel, int n_rows, int n_req, int n_pages, const Shape &s, void *out, float *lse,
                     int32_t *err, cudaStream_t st) {
    k_attn_tree<D, HPG><<<unsigned(n_rows) * unsigned(s.G), 128, 0, st>>>(
        static_cast<const uint16_t *>(q), static_cast<const uint16_t *>(k_cache),
        static_cast<const uint16_t *>(v_cache), static_cast<const uint16_t *>(k_new),
        static_cast<const uint16_t *>(v_new), bt, ctx, node_off, anc, sel, n_rows, n_req, n_pages, s.G, s.topk,
        s.max_blocks, s.sm_scale, static_cast<uint16_t *>(out), lse, err);
    return cudaGetLastError();
}

}  // namespace

size_t tree_workspace_bytes(int, int, const Shape &) { return 16; }

cudaError_t launch_attn_tree(const void *q, const void *k_cache, const void *v_cache, const void *k_new,
                             const void *v_new, const int32_t *block_table, const int32_t *ctx_lens,
                             const int32_t *node_off, const uint64_t *anc, const int32_t *sel, int n_rows, int n_req,
                             int n_pages, const Shape &s, void *out, float *lse, void *, int32_t *err,
                             cudaStream_t st) {
#define MSA_AT_CASE(DD, HH)                                                                                      \
    if (s.D == DD && s.hpg == HH)                                                                                \
        return launch_t<DD, HH>(q, k_cache, v_cache, k_new, v_new, block_table, ctx_lens, node_off, anc, sel, n_rows, \
                                n_req, n_pages, s, out, lse, err, st);
    MSA_AT_CASE(128, 8) MSA_AT_CASE(128, 4) MSA_AT_CASE(64, 8) MSA_AT_CASE(64, 4)
#undef MSA_AT_CASE
    return cudaErrorNotSupported;
}

}  // namespace msa
