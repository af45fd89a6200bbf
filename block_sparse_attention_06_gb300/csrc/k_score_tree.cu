// Block scores for the nodes of drafted trees.
//
// As the multi-token decode scan: s[i, g, j] = max_t q_idx[i, g] . k_idx[t, g] over the tokens of block j
// that node i may see, with the block's k-index read once for all nodes.  What differs is who is seen:
// every cached token (position < ctx), and of the drafted tokens the node's ancestors and itself, whose
// index keys come as dense rows and whose block is (ctx + depth) / 128.  Drafts therefore touch only
// the block that the context ends in and the one after it.
//   - one CTA per (request, page, 16 nodes); warp w scores KV group w (and w + 8);
//   - the warp stages its group's 128 x Di slice of the page in 32-token chunks (16-byte cp.async,
//     double-buffered, chunk columns XOR-swizzled so that ldmatrix reads them without bank conflicts);
//   - m16n8k16 bf16 MMAs with tokens as M and nodes as N; the max over tokens is taken on the fp32
//     accumulators.  A CTA of a block that drafts may touch then scores the drafted keys the same way.
#include "msa_device.cuh"
#include "msa_internal.h"

#include <algorithm>

namespace msa {
namespace {

constexpr int kWarps = 8;
constexpr int kChunkTok = 32;        // tokens per staged chunk
constexpr int kRows = 16;            // nodes of one CTA (two n-tiles of 8)

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t &r0, uint32_t &r1, uint32_t &r2, uint32_t &r3) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr));
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Position of the 16-byte chunk q of token row i in a staged chunk: rows of DI bf16, chunk index
// XOR-swizzled so that the 8 rows an ldmatrix phase reads fall in 8 distinct bank groups.
template <int DI>
__device__ __forceinline__ uint32_t stage_off(int i, int q) {
    if constexpr (DI == 64) return uint32_t(i * 128 + ((q ^ (i & 7)) << 4));
    else return uint32_t(i * 64 + ((q ^ ((i >> 1) & 3)) << 4));
}

template <int DI>
__global__ void __launch_bounds__(kWarps * 32) k_score_tree(
    const uint16_t *__restrict__ q_idx, const uint8_t *__restrict__ kidx, const uint8_t *__restrict__ kidx_new,
    const int32_t *__restrict__ block_table, const int32_t *__restrict__ ctx_lens,
    const int32_t *__restrict__ node_off, const uint64_t *__restrict__ anc, int n_rows, int n_pages, int G,
    int max_blocks, float *__restrict__ scores, int32_t *err) {
    constexpr int CH = DI / 8;                     // 16-byte chunks per token row
    constexpr int KS = DI / 16;                    // k-steps of 16
    constexpr int STAGE = kChunkTok * DI * 2;      // bytes of one staged chunk
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int draft_blk[kTreeMaxNodes];       // block of each drafted token
    const int b = blockIdx.x, j = blockIdx.y, n0 = blockIdx.z * kRows;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int row0;
    const int n = tree_rows_of(node_off, b, n_rows, err, tid == 0 && j == 0 && n0 == 0, &row0);
    const int T = min(kRows, n - n0);
    if (T <= 0) return;
    const int ctx = ctx_lens[b];
    if (ctx < 0) {
        if (tid == 0 && j == 0) raise_flag(err, MSA_FLAG_BOUNDS);
        return;
    }
    const int first = row0 + n0;
    const int n_cached = min(128, max(0, ctx - j * 128));   // cached tokens of this block
    const bool drafts = (j + 1) * 128 > ctx && j * 128 < ctx + n;
    if (n_cached == 0 && !drafts) {
        for (int i = tid; i < T * G; i += kWarps * 32)
            scores[(size_t(first + i / G) * G + (i % G)) * max_blocks + j] = -INFINITY;
        return;
    }
    int page = 0;
    if (n_cached > 0) {
        page = block_table[size_t(b) * max_blocks + j];
        if (page < 0 || page >= n_pages) {
            if (tid == 0) raise_flag(err, MSA_FLAG_BOUNDS);
            return;
        }
    }
    if (drafts && tid < n) draft_blk[tid] = (ctx + __popcll(anc[row0 + tid]) - 1) >> 7;
    __syncthreads();

    // this lane's accumulator columns: nodes nt * 8 + (lane & 3) * 2 + e
    uint64_t path[2][2];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = nt * 8 + (lane & 3) * 2 + e;
            path[nt][e] = drafts && i < T ? anc[first + i] : 0ull;
        }
    const int NT = (T + 7) >> 3;
    const uint32_t stage_s = smem_u32(smem + warp * 2 * STAGE);
    const int cached_chunks = (n_cached + kChunkTok - 1) / kChunkTok;
    const int chunks = cached_chunks + (drafts ? (n + kChunkTok - 1) / kChunkTok : 0);

    for (int g = warp; g < G; g += kWarps) {
        // q_idx fragments (B operand, "col": k = d, n = node): b0 = k 0..7 pair, b1 = k 8..15 pair
        uint32_t bq[2][KS][2];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const int i = nt * 8 + (lane >> 2);
                const int d = ks * 16 + (lane & 3) * 2;
                uint32_t v0 = 0, v1 = 0;
                if (i < T) {
                    const uint16_t *qp = q_idx + (size_t(first + i) * G + g) * DI;
                    v0 = *reinterpret_cast<const uint32_t *>(qp + d);
                    v1 = *reinterpret_cast<const uint32_t *>(qp + d + 8);
                }
                bq[nt][ks][0] = v0;
                bq[nt][ks][1] = v1;
            }
        // chunk c: 32 cached tokens of the page, or 32 drafted ones; rows past the end repeat the last one
        auto issue = [&](int c) {
            const uint32_t dst = stage_s + uint32_t((c & 1) * STAGE);
            const bool cached = c < cached_chunks;
            const int t0 = (cached ? c : c - cached_chunks) * kChunkTok;
            const int lim = cached ? 127 : n - 1;
            const uint8_t *src = (cached ? kidx + size_t(page) * 128 * G * DI * 2 : kidx_new + size_t(row0) * G * DI * 2) +
                                 size_t(g) * DI * 2;
#pragma unroll
            for (int k = 0; k < kChunkTok * CH / 32; ++k) {
                const int p = lane + 32 * k;
                const int i = p / CH, q = p % CH;
                cp_async_16(dst + stage_off<DI>(i, q), src + size_t(min(t0 + i, lim)) * G * DI * 2 + q * 16);
            }
            cp_async_commit();
        };
        float mx[2][2];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) mx[nt][0] = mx[nt][1] = -INFINITY;
        issue(0);
        if (chunks > 1) issue(1);
        else cp_async_commit();
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            cp_async_wait<1>();   // chunk c has landed (chunk c + 1 may be in flight)
            __syncwarp();
            const uint32_t buf = stage_s + uint32_t((c & 1) * STAGE);
            const bool cached = c < cached_chunks;
#pragma unroll
            for (int mt = 0; mt < kChunkTok / 16; ++mt) {
                float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    // A = 16 tokens x 16 index dims: matrices (rows 0-7 | 8-15) x (cols 0-7 | 8-15)
                    const int r = mt * 16 + (lane & 7) + ((lane >> 3) & 1) * 8;
                    const int q = ks * 2 + (lane >> 4);
                    uint32_t a0, a1, a2, a3;
                    ldsm_x4(buf + stage_off<DI>(r, q), a0, a1, a2, a3);
                    mma16816(acc[0], a0, a1, a2, a3, bq[0][ks][0], bq[0][ks][1]);
                    if (NT > 1) mma16816(acc[1], a0, a1, a2, a3, bq[1][ks][0], bq[1][ks][1]);
                }
                // accumulator: acc[nt][h * 2 + e] = token (lane >> 2) + 8 h, node nt * 8 + (lane & 3) * 2 + e
                const int tok0 = mt * 16 + (lane >> 2);
                if (cached) {
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                if (c * kChunkTok + tok0 + 8 * h < n_cached)
                                    mx[nt][e] = fmaxf(mx[nt][e], acc[nt][h * 2 + e]);
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int t = (c - cached_chunks) * kChunkTok + tok0 + 8 * h;
                        if (t >= n || draft_blk[t] != j) continue;
#pragma unroll
                        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                if (path[nt][e] >> t & 1) mx[nt][e] = fmaxf(mx[nt][e], acc[nt][h * 2 + e]);
                    }
                }
            }
            __syncwarp();
            if (c + 2 < chunks) issue(c + 2);
            else cp_async_commit();   // keep one group per chunk so that wait<1> stays exact
        }
        cp_async_wait<0>();
        // max over the 8 lanes that share the columns
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float v = mx[nt][e];
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                mx[nt][e] = v;
            }
        if (lane < 4) {
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = nt * 8 + lane * 2 + e;
                    if (i < T) scores[(size_t(first + i) * G + g) * max_blocks + j] = mx[nt][e];
                }
        }
        __syncwarp();   // the stage buffers are reused by the next group
    }
}

template <int DI>
cudaError_t launch_di(const void *q_idx, const void *kidx, const void *kidx_new, const int32_t *bt, const int32_t *ctx,
                      const int32_t *node_off, const uint64_t *anc, int n_rows, int n_req, int n_pages, const Shape &s,
                      float *scores, int32_t *err, cudaStream_t st) {
    const size_t smem = size_t(kWarps) * 2 * kChunkTok * DI * 2;
    cudaError_t e = cudaFuncSetAttribute(k_score_tree<DI>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    const int groups = (std::min(n_rows, kTreeMaxNodes) + kRows - 1) / kRows;
    const dim3 grid(static_cast<unsigned>(n_req), static_cast<unsigned>(s.max_blocks), static_cast<unsigned>(groups));
    k_score_tree<DI><<<grid, kWarps * 32, smem, st>>>(
        static_cast<const uint16_t *>(q_idx), static_cast<const uint8_t *>(kidx),
        static_cast<const uint8_t *>(kidx_new), bt, ctx, node_off, anc, n_rows, n_pages, s.G, s.max_blocks, scores,
        err);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_score_tree(const void *q_idx, const void *kidx, const void *kidx_new, const int32_t *block_table,
                              const int32_t *ctx_lens, const int32_t *node_off, const uint64_t *anc, int n_rows,
                              int n_req, int n_pages, const Shape &s, float *scores, int32_t *err, cudaStream_t st) {
    if (n_rows <= 0) return cudaSuccess;
    if (s.Di == 64)
        return launch_di<64>(q_idx, kidx, kidx_new, block_table, ctx_lens, node_off, anc, n_rows, n_req, n_pages, s,
                             scores, err, st);
    if (s.Di == 32)
        return launch_di<32>(q_idx, kidx, kidx_new, block_table, ctx_lens, node_off, anc, n_rows, n_req, n_pages, s,
                             scores, err, st);
    return cudaErrorNotSupported;
}

}  // namespace msa
