// Host-side launchers shared between the C-ABI layer and the kernel files.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "msa.h"

#include <atomic>
#include <utility>

namespace msa {

// Launch `kernel` on `st`; with pdl == true the launch carries programmatic
// stream serialisation, so it may overlap the tail of the previous kernel on the
// stream (the kernel must call pdl_wait() before reading that kernel's output).
template <typename... KArgs, typename... Args>
cudaError_t launch_kernel(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, bool pdl,
                          Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

struct Shape {
    int Hq, G, D, Di, topk, max_blocks, hpg;
    float sm_scale;
};

cudaError_t launch_score_decode(const void *q_idx, const void *kidx, const int32_t *block_table,
                                const int32_t *q_req, const int32_t *q_pos, int n_rows, int n_req,
                                int n_pages, const Shape &s, float *scores, int32_t *err,
                                cudaStream_t st);

// `bytes` (a multiple of 16) from page-locked host memory (its device mapping) to device memory.
cudaError_t launch_stage_from_host(const void *src, void *dst, size_t bytes, cudaStream_t st);
// Selected K/V pages from host memory into a device pool (zero-copy gather).
cudaError_t launch_offload_gather(const void *host_k, const void *host_v, const int32_t *page_table, int B,
                                  int n_host_pages, const Shape &s, void *pool_k, void *pool_v,
                                  int32_t *pool_page_table, int32_t *err, cudaStream_t st);
// Multi-token decode scoring: rows grouped by request (q_req non-decreasing, <= 16 rows each).
cudaError_t launch_score_decode_mt(const void *q_idx, const void *kidx, const int32_t *block_table,
                                   const int32_t *q_req, const int32_t *q_pos, int n_rows, int n_req, int n_pages,
                                   const Shape &s, float *scores, int32_t *err, cudaStream_t st);
cudaError_t launch_score_prefill(const void *q_idx, const void *kidx, const int32_t *block_table,
                                 const int32_t *q_req, const int32_t *q_pos, int n_rows, int n_req,
                                 int n_pages, const Shape &s, float *scores, uint64_t *lists, int32_t *err,
                                 cudaStream_t st);
// Prefill scoring with top-k fused: block chunks per row (candidate lists per (row, group, chunk)),
// candidates kept per list, and the merge of the lists into the selection.
int score_prefill_chunks(int max_blocks);
constexpr int kSelectListLen = 15;
// Target of the inversion's first pass (bit q of key k at bitmap[k * words + q / 32]);
// bitmap == nullptr means "do not mark".
struct InvMark {
    uint32_t *bitmap;
    size_t words;
    const int32_t *q_req;
    int n_req;
};
cudaError_t launch_topk_merge(const uint64_t *lists, const int32_t *q_pos, int n_rows, const Shape &s,
                              int n_chunks, int32_t *sel, const InvMark &mark, int32_t *err, cudaStream_t st);

cudaError_t launch_topk(const float *scores, const int32_t *q_pos, int n_rows, const Shape &s,
                        int32_t *sel, int32_t *err, cudaStream_t st);

cudaError_t launch_page_table(const int32_t *sel, const int32_t *block_table, const int32_t *seq_lens,
                              int B, int n_pages, const Shape &s, int32_t *pt, int32_t *row_len,
                              int32_t *err, cudaStream_t st);

size_t invert_workspace_bytes(int n_rows, int n_req, const Shape &s);
cudaError_t launch_invert(const int32_t *sel, const int32_t *q_req, int n_rows, int n_req,
                          const Shape &s, int32_t *blk_off, int32_t *blk_ent, int32_t *ent_pos, void *ws,
                          int32_t *err, cudaStream_t st);
// The inversion in two halves around a caller that marks the bitmap itself:
// invert_clear zeroes the bitmap in the inversion workspace and returns the mark
// target; launch_invert_finish counts, scans and emits from the marked bitmap.
InvMark invert_clear(const int32_t *q_req, int n_rows, int n_req, const Shape &s, void *ws, cudaStream_t st,
                     cudaError_t *e);
cudaError_t launch_invert_finish(const int32_t *sel, const int32_t *q_req, int n_rows, int n_req, const Shape &s,
                                 int32_t *blk_off, int32_t *blk_ent, int32_t *ent_pos, void *ws, int32_t *err,
                                 cudaStream_t st);

// Block-major prefill attention: a plan kernel writes the chunk work list into
// the workspace, then one persistent CTA per SM consumes it.
size_t prefill_workspace_bytes(int n_rows, int n_req, const Shape &s);
cudaError_t launch_attn_prefill(const void *q, const void *k_cache, const void *v_cache,
                                const int32_t *block_table, const int32_t *q_req,
                                const int32_t *q_pos, const int32_t *blk_off,
                                const int32_t *blk_ent, int n_rows, int n_req, int n_pages,
                                const Shape &s, void *o_part, float *lse_part, void *ws,
                                int32_t *err, cudaStream_t st);

cudaError_t launch_lse_merge(const void *o_part, const float *lse_part, const int32_t *sel,
                             const int32_t *ent_pos, int n_rows, const Shape &s, void *out, float *lse,
                             int32_t *err, cudaStream_t st);

// Decode workspace: segment partials (one per run of a row's pages inside one
// CTA's range, at the run's first slot), their lse, and one merge counter per
// (request, group) row.  The counters must be zero when the attention kernel
// starts; launch_attn_decode clears them itself unless counters_zeroed is set
// (the fused decode step clears them in its select kernel).
size_t decode_workspace_bytes(int B, const Shape &s);
int32_t *decode_ws_counters(void *ws, int B, const Shape &s);
cudaError_t launch_attn_decode(const void *q, const void *k_cache, const void *v_cache,
                               const int32_t *pt, const int32_t *row_len, int B, int n_pages,
                               const Shape &s, void *out, float *lse, void *ws, int32_t *err,
                               cudaStream_t st, bool counters_zeroed = false, bool pdl = false);

// Decode selection in one launch after the index scan: top-k per (request,
// group), page table and row lengths; also zeroes `counters` (B*G entries,
// may be null).  Launched with programmatic serialisation after the scan.
cudaError_t launch_decode_select(const float *scores, const int32_t *seq_lens, const int32_t *block_table,
                                 int B, int n_pages, const Shape &s, int32_t *sel, int32_t *pt,
                                 int32_t *row_len, int32_t *counters, int32_t *err, cudaStream_t st,
                                 bool pdl);

// Decode index scan whose rows are the B requests themselves (row b is request
// b at position seq_lens[b] - 1).
cudaError_t launch_score_decode_seq(const void *q_idx, const void *kidx, const int32_t *block_table,
                                    const int32_t *seq_lens, int B, int n_pages, const Shape &s,
                                    float *scores, int32_t *err, cudaStream_t st, bool pdl = false);

// Drafted trees (speculative decode): layout, scoring, attention, verification, commit.
constexpr int kTreeMaxNodes = 64;   // nodes per request (one bit each in a row's ancestor word)
cudaError_t launch_tree_rows(const int32_t *node_off, const int32_t *parents, const int32_t *ctx_lens, int n_rows,
                             int n_req, int max_blocks, int32_t *q_req, int32_t *q_pos, uint64_t *anc, int32_t *err,
                             cudaStream_t st);
cudaError_t launch_score_tree(const void *q_idx, const void *kidx, const void *kidx_new, const int32_t *block_table,
                              const int32_t *ctx_lens, const int32_t *node_off, const uint64_t *anc, int n_rows,
                              int n_req, int n_pages, const Shape &s, float *scores, int32_t *err, cudaStream_t st);
size_t tree_workspace_bytes(int n_rows, int n_req, const Shape &s);
cudaError_t launch_attn_tree(const void *q, const void *k_cache, const void *v_cache, const void *k_new,
                             const void *v_new, const int32_t *block_table, const int32_t *ctx_lens,
                             const int32_t *node_off, const uint64_t *anc, const int32_t *sel, int n_rows, int n_req,
                             int n_pages, const Shape &s, void *out, float *lse, void *ws, int32_t *err,
                             cudaStream_t st);
cudaError_t launch_verify_tree(const float *p, const float *q, int vocab, const int32_t *tokens,
                               const int32_t *node_off, const int32_t *parents, const float *u_accept,
                               const float *u_next, int n_rows, int n_req, int32_t *path, int32_t *n_acc,
                               int32_t *next_token, int32_t *err, cudaStream_t st);
cudaError_t launch_commit_tree(const void *k_new, const void *v_new, const void *kidx_new, int n_layers, void *k_cache,
                               void *v_cache, void *kidx_cache, const int32_t *block_table, const int32_t *ctx_lens,
                               const int32_t *node_off, const int32_t *path, const int32_t *n_acc, int n_rows,
                               int n_req, int n_pages, const Shape &s, int32_t *new_lens, int32_t *err,
                               cudaStream_t st);

// 8-bit caches of one layer: e4m3 codes [n_pages][G][128][width] and scale bytes [n_pages][G][128].
struct CacheQ8 {
    void *k, *k_scale, *v, *v_scale, *kidx, *kidx_scale;
};

// Rotary positions and the append of a layer's new rows: q, k, v, q_idx, k_idx (the last two may be absent);
// scale[0] says whether the caches are 8-bit.
struct RopeAppend {
    const void *src[5];
    long long stride[5];
    void *q_out, *q_idx_out;
    void *dst[3], *scale[3];
    const double *inv_freq, *inv_freq_idx;
    const int32_t *block_table, *q_req, *q_pos;
    int n_rows, n_req, n_pages, rot, rot_idx, interleaved;
    float gain;
    int32_t *err;
};
cudaError_t launch_rope_append(const RopeAppend &p, const Shape &s, cudaStream_t st);
// Blocks of 8-bit caches as bf16 pages; kidx may be null.
cudaError_t launch_cache_read(const CacheQ8 &c, const int32_t *bt_in, const int32_t *bt_out, const int32_t *lens,
                              int n_req, int n_pages, int n_pages_out, const Shape &s, void *k, void *v, void *kidx,
                              int32_t *err, cudaStream_t st);
// Decode index scan over 8-bit index keys: rows by (q_req, q_pos), or the requests at seq_lens - 1.
cudaError_t launch_score_q8(const void *q_idx, const CacheQ8 &c, const int32_t *block_table, const int32_t *q_req,
                            const int32_t *q_pos, const int32_t *seq_lens, int n_rows, int n_req, int n_pages,
                            const Shape &s, float *scores, int32_t *err, cudaStream_t st, bool pdl = false);
// Decode attention over 8-bit caches: the pages of a table, or a window and the first tokens.
cudaError_t launch_attn_decode_q8(const void *q, const CacheQ8 &c, const int32_t *page_table, const int32_t *row_len,
                                  int B, int n_pages, const Shape &s, void *out, float *lse, int32_t *err,
                                  cudaStream_t st, bool pdl = false);
cudaError_t launch_window_decode_q8(const void *q, const CacheQ8 &c, const int32_t *block_table, const int32_t *q_req,
                                    const int32_t *q_pos, int n_rows, int n_req, int n_pages, int window, int n_sink,
                                    const Shape &s, void *out, float *lse, int32_t *err, cudaStream_t st);
// The same window attention with runs of consecutive rows sharing their reads, on the tensor cores.
cudaError_t launch_window_prefill_q8(const void *q, const CacheQ8 &c, const int32_t *block_table, const int32_t *q_req,
                                     const int32_t *q_pos, int n_rows, int n_req, int n_pages, int window, int n_sink,
                                     const Shape &s, void *out, float *lse, int32_t *err, cudaStream_t st);

// Tensor-map creation through the driver entry point (no libcuda link dependency).
bool encode_tensor_map(void *map, int rank, const void *base, const uint64_t *dims,
                       const uint64_t *strides_bytes, const uint32_t *box, int swizzle_bytes,
                       const char **why);

int sm_count();

// The attributes of a kernel that takes `smem` bytes (and clusters of more than 8 CTAs), set at its first launch on
// a device; `done` is the kernel's own.
cudaError_t allow_once(std::atomic<uint64_t> &done, const void *kernel, size_t smem, bool large_clusters = false);

// One thread waits on an mbarrier that nothing arrives on (the device timeout path).
cudaError_t launch_selftest_timeout(int32_t *err, cudaStream_t st);

// Record the detail string that msa_last_error() returns on this thread.
void set_last_error(const char *msg);

}  // namespace msa
