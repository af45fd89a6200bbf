// Verification of drafted trees against the target's probabilities.
//
// With r_c(t) = max(p(t) - c q(t), 0) the residual after any number of rejections is r_c / M, M its
// sum: rejecting a child takes p' to max(p' - q, 0) normalised, i.e. r_c / M to r_{c + M} / M'.  So a
// node's state is two scalars, and a rejection costs one pass over the node's two rows.
// One CTA per request walks the path; sums and comparisons are in 64 bits.
#include "msa_device.cuh"
#include "msa_internal.h"

namespace msa {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ double warp_sum_d(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

struct Smem {
    int parent[kTreeMaxNodes], tok[kTreeMaxNodes];
    float u[kTreeMaxNodes], p[kTreeMaxNodes], q[kTreeMaxNodes];   // at the node's token in its parent's rows
    int gone[kTreeMaxNodes];                                      // tokens taken out (no draft distribution)
    double part[kWarps];
    int found;
};

__device__ double residual(const float *__restrict__ p, const float *__restrict__ q, double c, const int *gone,
                           int n_gone, int t) {
    double r = double(p[t]);
    if (q) r -= c * double(q[t]);
    for (int i = 0; i < n_gone; ++i)
        if (gone[i] == t) r = 0.0;
    return r > 0.0 ? r : 0.0;
}

__global__ void __launch_bounds__(kThreads) k_verify_tree(
    const float *__restrict__ probs, const float *__restrict__ drafts, int vocab, const int32_t *__restrict__ tokens,
    const int32_t *__restrict__ node_off, const int32_t *__restrict__ parents, const float *__restrict__ u_accept,
    const float *__restrict__ u_next, int n_rows, int32_t *__restrict__ path, int32_t *__restrict__ n_acc,
    int32_t *__restrict__ next_token, int32_t *err) {
    __shared__ Smem sm;
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int row0;
    const int n = tree_rows_of(node_off, b, n_rows, err, tid == 0, &row0);
    if (n == 0) {
        if (tid == 0) {
            n_acc[b] = 0;
            next_token[b] = -1;
        }
        return;
    }
    if (tid < n) {
        const int par = parents[row0 + tid], tok = tokens[row0 + tid];
        const bool ok = tid > 0 && par >= 0 && par < tid && tok >= 0 && tok < vocab;
        if (tid == 0 ? par != -1 : !ok) raise_flag(err, MSA_FLAG_BOUNDS);
        sm.parent[tid] = ok ? par : -1;
        sm.tok[tid] = tok;
        if (ok) {
            sm.u[tid] = u_accept[row0 + tid];
            sm.p[tid] = probs[size_t(row0 + par) * vocab + tok];
            if (drafts) sm.q[tid] = drafts[size_t(row0 + par) * vocab + tok];
        }
        path[row0 + tid] = -1;
    }
    __syncthreads();
    // a contiguous range of the vocabulary per thread
    const int t0 = int((long long)tid * vocab / kThreads), t1 = int((long long)(tid + 1) * vocab / kThreads);
    auto block_sum = [&](double v) {
        v = warp_sum_d(v);
        __syncthreads();
        if (lane == 0) sm.part[warp] = v;
        __syncthreads();
        double s = 0.0;
        for (int w = 0; w < kWarps; ++w) s += sm.part[w];
        return s;
    };
    int at = 0, count = 0;
    double c, mass;
    int n_gone;
    const float *p, *q;
    for (;;) {
        if (tid == 0) path[row0 + count] = at;
        ++count;
        c = 0.0;
        mass = 1.0;
        n_gone = 0;
        p = probs + size_t(row0 + at) * vocab;
        q = drafts ? drafts + size_t(row0 + at) * vocab : nullptr;
        int next = -1;
        for (int x = at + 1; x < n && next < 0; ++x) {
            if (sm.parent[x] != at) continue;
            const double qx = q ? double(sm.q[x]) : 1.0;
            double r = double(sm.p[x]) - (q ? c * qx : 0.0);
            for (int i = 0; i < n_gone; ++i)
                if (sm.gone[i] == sm.tok[x]) r = 0.0;
            if (!(r > 0.0)) r = 0.0;
            if (double(sm.u[x]) * qx * mass < r) {
                next = x;
            } else if (q) {
                c += mass;
                double v = 0.0;
                for (int t = t0; t < t1; ++t) v += residual(p, q, c, nullptr, 0, t);
                mass = block_sum(v);
            } else {
                mass = fmax(mass - r, 0.0);   // rounding of p may leave less than nothing
                if (tid == 0) sm.gone[n_gone] = sm.tok[x];
                ++n_gone;
                __syncthreads();
            }
        }
        if (next < 0) break;
        at = next;
        __syncthreads();   // sm.gone is free again
    }
    // the next token from the residual, or from p where nothing is left of it
    double mine = 0.0, total = 0.0;
    for (int attempt = 0; attempt < 2; ++attempt) {
        if (attempt) q = nullptr, n_gone = 0;
        mine = 0.0;
        for (int t = t0; t < t1; ++t) mine += residual(p, q, c, sm.gone, n_gone, t);
        total = block_sum(mine);
        if (total > 0.0) break;
    }
    if (!(total > 0.0) || isinf(total)) {
        if (tid == 0) {
            raise_flag(err, MSA_FLAG_NAN);
            next_token[b] = -1;
            n_acc[b] = count;
        }
        return;
    }
    const double want = double(u_next[b]) * total;
    // exclusive prefix of this thread's range
    double incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    __syncthreads();
    if (lane == 31) sm.part[warp] = incl;
    if (tid == 0) sm.found = vocab;
    __syncthreads();
    double before = incl - mine;
    for (int w = 0; w < warp; ++w) before += sm.part[w];
    double run = before;
    int last = -1;
    for (int t = t0; t < t1; ++t) {
        const double r = residual(p, q, c, sm.gone, n_gone, t);
        run += r;
        if (r > 0.0) last = t;
        if (run > want) {
            atomicMin(&sm.found, t);
            break;
        }
    }
    __syncthreads();
    int tok = sm.found;
    __syncthreads();
    if (tok == vocab) {   // rounding left the last range short: the last token with mass
        if (tid == 0) sm.found = -1;
        __syncthreads();
        if (last >= 0) atomicMax(&sm.found, last);
        __syncthreads();
        tok = sm.found;
    }
    if (tid == 0) {
        next_token[b] = tok;
        n_acc[b] = count;
    }
}

}  // namespace

cudaError_t launch_verify_tree(const float *p, const float *q, int vocab, const int32_t *tokens,
                               const int32_t *node_off, const int32_t *parents, const float *u_accept,
                               const float *u_next, int n_rows, int n_req, int32_t *path, int32_t *n_acc,
                               int32_t *next_token, int32_t *err, cudaStream_t st) {
    k_verify_tree<<<unsigned(n_req), kThreads, 0, st>>>(p, q, vocab, tokens, node_off, parents, u_accept, u_next,
                                                        n_rows, path, n_acc, next_token, err);
    return cudaGetLastError();
}

}  // namespace msa
