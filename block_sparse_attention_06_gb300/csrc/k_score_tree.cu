// Block scores for the nodes of drafted trees, on the 5th-generation tensor cores.
//
// s[i, g, j] = max_t q_idx[i, g] . k_idx[t, g] over the tokens of block j that node i may see: every cached token
// (position < ctx), and of the drafted tokens the node's ancestors and itself, whose index keys come as dense
// rows and whose block is (ctx + depth) / 128.  Drafts touch only the block that the context ends in and the
// one after it.
//
// The scan reads the k-index once for all nodes of a request, and that read bounds it (61 MB per request of 60,000
// tokens at G = 8, Di = 64).  One persistent CTA per SM; the units (request, block, group), groups innermost, are
// cut into one contiguous range per CTA, so that a CTA keeps its request's queries in shared memory and streams
// whole pages.  With nodes as M (up to 64 of the 128 MMA rows; the rest is ignored) and the block's tokens as N,
// a node's score is a maximum over one TMEM lane.  Warp-level MMAs with tokens as M, as in the multi-token
// scan, hold 16 nodes at a time: four passes over the pages for 64 nodes.  8 x 60,000 tokens (492 MB): 84 us with 16
// nodes and 90 with 64, 5.9 and 5.5 TB/s; by warp-level MMAs 93 and 307.
// Warps:
//   4+5, 8+9, 12+13, 16+17  epilogue sets (a warp can read only the TMEM lane quarter of its index mod 4, and 64
//         nodes are two quarters), each with every fourth unit and a 128-column accumulator in TMEM;
//   0, 7, 10, 11  a producer for each set: 128-token tiles of the pages into the set's ring by TMA, drafted keys last;
//   1, 2, 3, 6  an MMA issuer for each set.  The waits, address arithmetic and commits of a tile cost one thread
//         1,000 to 1,500 cycles, more than the 720 that the pages' read leaves for it (one issuer: 140 us for 8 x
//         60,000 tokens; one producer: 106 us), so neither role is one thread;
//   14    the queries of a request (all groups), by TMA;
//   14, 15  write -inf to the blocks past the drafts.
// Every barrier has one waiting role, which waits for each of its phases in order: a role that could get a whole
// ring ahead of another on a shared barrier would take the parity of the phase before last for its own.
// Every wait is bounded.
#include "msa_device.cuh"
#include "msa_internal.h"

#include <algorithm>

namespace msa {
namespace {

constexpr int kThreads = 18 * 32;
constexpr int kSets = 4;
constexpr int kMaxDepth = 3;      // tiles of a set's ring
constexpr int kFillWarps = 2;
constexpr int kStage = 16 * 33;   // floats an epilogue warp stages: 16 / (groups of its set) blocks x 32 nodes, padded
constexpr int kSmemLimit = 232448 - 1024;   // of a CTA, less the statically declared part

struct Ctl {
    uint64_t q_full, q_free;
    uint64_t full[kSets * kMaxDepth], empty[kSets * kMaxDepth];
    uint64_t acc_full[kSets], acc_free[kSets];
    uint64_t drain;   // every issuer's last MMAs
    int wsum[kThreads / 32];
    int b0, v0;
    uint32_t tmem_base;
    int abort;
};

__device__ __forceinline__ long long range_begin(int c, long long n, int C) { return c * n / C; }

// A request as the scan sees it.
struct Req {
    int row0, n, ctx, nb;   // nb: blocks that hold cached or drafted tokens
    __device__ __forceinline__ void load(const int32_t *__restrict__ node_off, const int32_t *__restrict__ ctx_lens,
                                         int b, int n_rows, int max_blocks, int32_t *err, bool report) {
        n = tree_rows_of(node_off, b, n_rows, err, report, &row0);
        ctx = ctx_lens[b];
        if (ctx < 0) {
            if (report && n > 0) raise_flag(err, MSA_FLAG_BOUNDS);
            n = 0;
        }
        nb = n > 0 ? int(min((long long)max_blocks, ((long long)ctx + n + 127) >> 7)) : 0;
    }
};

// The units of a CTA's range, every STRIDE-th from the first-th on; every role walks them for itself.
template <int STRIDE>
struct Walk {
    const int32_t *node_off, *ctx_lens;
    int n_rows, max_blocks, G;
    long long left;          // units from the present one to the range's end, this one included
    int b, j, g;
    int request;             // requests of the range so far, less one
    bool begun;
    Req r;
    __device__ __forceinline__ void start(int b0, int v0) {
        b = b0;
        request = 0;
        begun = false;
        j = g = 0;
        if (left <= 0) return;
        r.load(node_off, ctx_lens, b, n_rows, max_blocks, nullptr, false);
        j = v0 / G;
        g = v0 - j * G;
    }
    __device__ __forceinline__ void move(int units) {
        left -= units;
        g += units;
        while (g >= G) {
            g -= G;
            if (++j == r.nb) {
                j = 0;
                ++request;
                do r.load(node_off, ctx_lens, ++b, n_rows, max_blocks, nullptr, false);
                while (r.nb == 0);
            }
        }
    }
    // On false the walk stands at the range's last unit (so `request` counts all of them).
    __device__ __forceinline__ bool next(int first = 0) {
        const int step = begun ? STRIDE : first;
        begun = true;
        if (left <= step) {
            if (left > 1) move(int(left) - 1);
            return false;
        }
        move(step);
        return true;
    }
    __device__ __forceinline__ int cached() const { return min(128, max(0, r.ctx - j * 128)); }
    __device__ __forceinline__ bool drafts() const { return (j + 1) * 128 > r.ctx; }   // j < nb: some may be here
};

template <int DI>
__global__ void __launch_bounds__(kThreads, 1) k_score_tree(
    const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
    const __grid_constant__ CUtensorMap dmap, const int32_t *__restrict__ block_table,
    const int32_t *__restrict__ ctx_lens, const int32_t *__restrict__ node_off, const uint64_t *__restrict__ anc,
    int n_rows, int n_req, int n_pages, int G, int max_blocks, int depth, float *__restrict__ scores,
    int32_t *err) {
    constexpr int TILE = 128 * DI * 2, QTILE = 64 * DI * 2;
    constexpr uint32_t kSw = DI == 64 ? 2u : 4u;           // descriptor swizzle: 128B / 64B
    constexpr uint32_t kSbo = 8u * DI * 2u;                // 8 rows of DI bf16
    constexpr uint32_t kIdesc = make_idesc_bf16(128, 128, 0, 0), kIdesc64 = make_idesc_bf16(128, 64, 0, 0);
    extern __shared__ uint8_t smem_raw[];
    __shared__ Ctl sm;
    uint8_t *const q_s = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *const ring = q_s + size_t(G + 1) * QTILE;     // an MMA reads 128 rows: one tile of slack
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        mbar_init(&sm.q_full, 1);
        mbar_init(&sm.q_free, kSets);
        for (int i = 0; i < kSets * depth; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], 1);
        }
        for (int s = 0; s < kSets; ++s) {
            mbar_init(&sm.acc_full[s], 1);
            mbar_init(&sm.acc_free[s], 2);
        }
        mbar_init(&sm.drain, kSets);
        sm.abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&sm.tmem_base, 128 * kSets);
        tmem_relinquish();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&qmap);
        tma_prefetch_desc(&kmap);
        tma_prefetch_desc(&dmap);
    }
    pdl_wait();
    pdl_trigger();
    // this CTA's range: a scan of the requests' units, a run of requests per thread
    const int b_lo = int((long long)tid * n_req / kThreads), b_hi = int((long long)(tid + 1) * n_req / kThreads);
    int mine = 0;
    for (int b = b_lo; b < b_hi; ++b) {
        Req r;
        r.load(node_off, ctx_lens, b, n_rows, max_blocks, err, blockIdx.x == 0);
        mine += r.nb * G;
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) sm.wsum[warp] = incl;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const int sums = lane < kThreads / 32 ? sm.wsum[lane] : 0;
    const int before = warp_sum_i(lane < warp ? sums : 0) + incl - mine;
    const long long total = warp_sum_i(sums);
    const int C = int(min((long long)gridDim.x, max(total, 1LL))), cta = blockIdx.x;   // no range is empty
    const long long x0 = cta < C ? range_begin(cta, total, C) : total;
    const long long x1 = cta < C ? range_begin(cta + 1, total, C) : total;
    if (x0 < x1 && x0 >= before && x0 < before + mine) {
        int b = b_lo, at = before;
        while (b + 1 < b_hi) {
            Req r;
            r.load(node_off, ctx_lens, b, n_rows, max_blocks, nullptr, false);
            if (x0 < at + r.nb * G) break;
            at += r.nb * G;
            ++b;
        }
        sm.b0 = b;
        sm.v0 = int(x0 - at);
    }
    __syncthreads();
    const uint32_t tmem = sm.tmem_base;
    const int b0 = x0 < x1 ? sm.b0 : 0, v0 = x0 < x1 ? sm.v0 : 0;

    if (warp == 0 || warp == 7 || warp == 10 || warp == 11) {
        // ------------------------------------------------------------ TMA producers (lane 0)
        if (lane == 0) {
            const int set = warp == 0 ? 0 : warp == 7 ? 1 : warp - 8;
            Walk<kSets> wk{node_off, ctx_lens, n_rows, max_blocks, G, x1 - x0};
            wk.start(b0, v0);
            int at = 0, loads = 0, b_of = -1, j_of = -1, page = 0, j_ahead = 0, ahead = 0;
            // The pages are read once, and evicted first they leave the block scores, whose 32-byte sectors fill up
            // over eight blocks, in L2 until they are whole (64 nodes: 98 us without).
            const uint64_t policy = l2_policy_evict_first();
            uint32_t phase = 1;   // of the slot's last reader, from the second round on
            auto page_of = [&](int j) -> int {
                return j * 128 < wk.r.ctx ? block_table[size_t(wk.b) * max_blocks + j] : 0;
            };
            // the ring's next slot, once its last reader is done with it
            auto claim = [&](uint32_t bytes) -> bool {
                if (loads >= depth && !mbar_wait(&sm.empty[set * depth + at], phase, err, &sm.abort)) return false;
                mbar_arrive_expect_tx(&sm.full[set * depth + at], bytes);
                return true;
            };
            auto advance = [&]() {
                ++loads;
                if (++at == depth) at = 0, phase ^= 1u;
            };
            while (wk.next(set)) {
                if (wk.b != b_of || wk.j != j_of) {
                    page = wk.b == b_of && wk.j == j_ahead ? ahead : page_of(wk.j);
                    b_of = wk.b;
                    j_of = wk.j;
                    if (page < 0 || page >= n_pages) {
                        raise_flag(err, MSA_FLAG_BOUNDS);
                        page = 0;   // a page that exists; the scores are unspecified
                    }
                    j_ahead = wk.j + max(1, kSets / G);   // the block of this set's next unit but G / 4, as a rule
                    if (j_ahead < wk.r.nb) ahead = page_of(j_ahead);
                }
                if (wk.cached() > 0) {
                    if (!claim(TILE)) break;
                    const int slot = set * depth + at;
                    tma_load_4d_hint(ring + size_t(slot) * TILE, &kmap, &sm.full[slot], 0, wk.g, 0, page, policy);
                    advance();
                }
                if (wk.drafts()) {
                    if (!claim(QTILE)) break;
                    const int slot = set * depth + at;
                    tma_load_3d(ring + size_t(slot) * TILE, &dmap, &sm.full[slot], 0, wk.g, wk.r.row0);
                    advance();
                }
            }
            if (sm.abort)   // the copies still in flight land before the CTA exits
                for (int n = max(0, loads - depth); n < loads; ++n)
                    mbar_wait(&sm.full[set * depth + n % depth], (n / depth) & 1, err, nullptr);
        }
    } else if (warp < 4 || warp == 6) {
        // ------------------------------------------------------------ MMA issuers (lane 0)
        if (lane == 0) {
            const int set = warp < 4 ? warp - 1 : 3;
            Walk<kSets> wk{node_off, ctx_lens, n_rows, max_blocks, G, x1 - x0};
            wk.start(b0, v0);
            int at = 0, tiles = 0, left_behind = 0;   // requests whose queries this issuer has done with
            uint32_t phase = 0;
            int q_of = -1;   // the request whose queries are here (waited for one by one: each issuer sees every phase)
            auto queries = [&](int request) -> bool {
                for (; q_of < request; ++q_of)
                    if (!mbar_wait(&sm.q_full, (q_of + 1) & 1, err, &sm.abort)) return false;
                return true;
            };
            // every issuer arrives once for each request of the range but the last, one phase at a time
            auto leave = [&]() -> bool {
                for (; left_behind < wk.request; ++left_behind) {
                    if (!queries(left_behind)) return false;
                    if (left_behind > 0 && !mbar_wait(&sm.q_free, (left_behind - 1) & 1, err, &sm.abort)) return false;
                    mma_commit(&sm.q_free);
                }
                return true;
            };
            bool ok = true;
            while (ok && wk.next(set)) {
                if (!(ok = leave())) break;
#pragma unroll 1
                for (int part = 0; part < 2; ++part) {   // cached tokens, drafted tokens
                    if (!(part ? wk.drafts() : wk.cached() > 0)) continue;
                    const int slot = set * depth + at;
                    if (!queries(wk.request) || !mbar_wait(&sm.full[slot], phase, err, &sm.abort) ||
                        (tiles > 0 && !mbar_wait(&sm.acc_free[set], (tiles - 1) & 1, err, &sm.abort))) {
                        ok = false;
                        break;
                    }
                    ++tiles;
                    tc_fence_after();
                    const uint32_t a = smem_u32(q_s + size_t(wk.g) * QTILE);
                    const uint32_t bb = smem_u32(ring + size_t(slot) * TILE);
#pragma unroll
                    for (int k = 0; k < DI / 16; ++k)
                        mma_bf16(tmem + uint32_t(set * 128), make_smem_desc(a + k * 32, 16, kSbo, kSw),
                                 make_smem_desc(bb + k * 32, 16, kSbo, kSw), part ? kIdesc64 : kIdesc, k > 0);
                    mma_commit(&sm.acc_full[set]);
                    mma_commit(&sm.empty[slot]);
                    if (++at == depth) at = 0, phase ^= 1u;
                }
            }
            if (ok) leave();
            mma_commit(&sm.drain);
            mbar_wait(&sm.drain, 0, err, nullptr);
        }
    } else if (warp >= 4 && (warp & 3) < 2) {
        // ------------------------------------------------------------ epilogue sets
        const int set = (warp >> 2) - 1, quad = warp & 3, i = quad * 32 + lane;   // node i
        const uint32_t t_s = tmem + (uint32_t(quad * 32) << 16) + uint32_t(set * 128);
        Walk<kSets> wk{node_off, ctx_lens, n_rows, max_blocks, G, x1 - x0};
        wk.start(b0, v0);
        const int j_start = wk.j, g_start = wk.g;
        const int span = G % kSets == 0 ? 16 / (G / kSets) : 0;   // blocks staged; 0: a set's groups change from block to block
        float *const stage = reinterpret_cast<float *>(ring + size_t(depth) * kSets * TILE) + (set * 2 + quad) * kStage;
        int tiles = 0, b_of = -1;
        unsigned long long path = 0, first = 0, second = 0;   // of this node; nodes by block: the context's last, the next
        bool ok = true;
        while (ok && wk.next(set)) {
            const Req &r = wk.r;
            if (wk.drafts() && b_of != wk.b) {
                b_of = wk.b;
                path = i < r.n ? anc[r.row0 + i] : 0ull;
                first = second = 0;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int m = h * 32 + lane;
                    const int blk = m < r.n ? (r.ctx + __popcll(anc[r.row0 + m]) - 1) >> 7 : -1;
                    first |= (unsigned long long)__ballot_sync(0xffffffffu, blk == r.ctx >> 7) << (32 * h);
                    second |= (unsigned long long)__ballot_sync(0xffffffffu, blk == (r.ctx >> 7) + 1) << (32 * h);
                }
            }
            const bool warp_live = quad * 32 < r.n;
            float best = -INFINITY;
#pragma unroll 1
            for (int part = 0; part < 2; ++part) {
                if (!(part ? wk.drafts() : wk.cached() > 0)) continue;
                if (!__all_sync(0xffffffffu, mbar_wait(&sm.acc_full[set], uint32_t(tiles & 1), err, &sm.abort))) {
                    ok = false;
                    break;
                }
                ++tiles;
                tc_fence_after();
                if (warp_live) {
                    const unsigned long long seen = path & (wk.j == r.ctx >> 7 ? first : second);
                    const int lim = part ? 64 : wk.cached();
#pragma unroll 1
                    for (int c0 = 0; c0 < lim; c0 += 64) {
                        uint32_t v[2][32];
                        tmem_ld32(t_s + uint32_t(c0), v[0]);
                        tmem_ld32(t_s + uint32_t(c0 + 32), v[1]);
                        tmem_ld_wait();
                        if (part || c0 + 64 > lim) {
                            const unsigned long long see =
                                part ? seen : lim - c0 >= 64 ? ~0ull : (1ull << (lim - c0)) - 1;
#pragma unroll
                            for (int e = 0; e < 64; ++e)
                                if (see >> e & 1) best = fmaxf(best, __uint_as_float(v[e >> 5][e & 31]));
                        } else {
                            float a[4] = {best, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                            for (int e = 0; e < 64; e += 8)
#pragma unroll
                                for (int x = 0; x < 4; ++x)
                                    a[x] = fmax3(a[x], __uint_as_float(v[e >> 5][(e & 31) + x]),
                                                 __uint_as_float(v[e >> 5][(e & 31) + 4 + x]));
                            best = fmaxf(fmax3(a[0], a[1], a[2]), a[3]);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.acc_free[set]);
            }
            if (!ok) break;
            if (!warp_live) continue;
            if (span == 0 || r.n <= 32) {
                if (i < r.n) scores[(size_t(r.row0 + i) * G + wk.g) * max_blocks + wk.j] = best;
                continue;
            }
            // A set has the same groups in every block: their scores are staged for `span` blocks and a row's go out in
            // one piece (one by one, each is a request of 32 bytes of its own to L2: 97 us against 90 for 64 nodes.
            // With few nodes the staging costs more than the requests: 86 us against 83 for 16).
            const int at = (wk.g / kSets) * span, in = wk.j & (span - 1);
            stage[(at + in) * 33 + lane] = best;
            if (in == span - 1 || wk.j == r.nb - 1 || wk.left <= G) {
                __syncwarp();
                // from the first block that this CTA has of this group
                const int j_first = wk.request > 0 ? 0 : j_start + (wk.g < g_start ? 1 : 0);
                const int jj = lane & (span - 1), j = wk.j - in + jj, x = lane / span, per = 32 / span;
                if (jj <= in && j >= j_first) {
                    float *dst = scores + (size_t(r.row0 + quad * 32 + x) * G + wk.g) * max_blocks + j;
                    const float *src = stage + (at + jj) * 33 + x;
                    const size_t step = size_t(per) * G * max_blocks;
                    const int rows = min(32, r.n - quad * 32);
#pragma unroll 4
                    for (int y = x; y < rows; y += per, dst += step, src += per) *dst = *src;
                }
                __syncwarp();
            }
        }
    } else {
        // ------------------------------------------------------------ queries (warp 14), -inf past the drafts
        if (warp == 14 && lane == 0) {
            Walk<1> wk{node_off, ctx_lens, n_rows, max_blocks, G, x1 - x0};
            wk.start(b0, v0);
            int requests = 0;
            if (x0 < x1)
                for (;; ++requests) {
                    if (requests > 0 && !mbar_wait(&sm.q_free, (requests - 1) & 1, err, &sm.abort)) break;
                    mbar_arrive_expect_tx(&sm.q_full, uint32_t(G) * QTILE);
                    for (int g = 0; g < G; ++g)
                        tma_load_3d(q_s + size_t(g) * QTILE, &qmap, &sm.q_full, 0, g, wk.r.row0);
                    const long long rest = 1LL * wk.r.nb * G - (1LL * wk.j * G + wk.g);   // units to the request's end
                    if (rest >= wk.left) {
                        ++requests;
                        break;
                    }
                    wk.move(int(rest));
                }
            if (requests > 0 && sm.abort) mbar_wait(&sm.q_full, (requests - 1) & 1, err, nullptr);
        }
        __syncwarp();
        if (warp >= 14) {
            const int fill = warp - 14;
            const int W = int(gridDim.x) * kFillWarps;
            int at = cta * kFillWarps + fill;   // (row, group) pairs of all requests, dealt to the warps in turn
            for (int b = 0; b < n_req; ++b) {
                Req r;
                r.load(node_off, ctx_lens, b, n_rows, max_blocks, nullptr, false);
                const int pairs = r.n * G;
                for (; at < pairs; at += W) {
                    float *row = scores + (size_t(r.row0) * G + at) * max_blocks;
                    for (int j = r.nb + lane; j < max_blocks; j += 32) row[j] = -INFINITY;
                }
                at -= pairs;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 128 * kSets);
}

template <int DI>
cudaError_t launch_di(const void *q_idx, const void *kidx, const void *kidx_new, const int32_t *bt, const int32_t *ctx,
                      const int32_t *node_off, const uint64_t *anc, int n_rows, int n_req, int n_pages, const Shape &s,
                      float *scores, int32_t *err, cudaStream_t st) {
    alignas(64) CUtensorMap qm, km, dm;
    const char *why = nullptr;
    {
        const uint64_t dims[3] = {uint64_t(DI), uint64_t(s.G), uint64_t(n_rows)};
        const uint64_t strides[2] = {uint64_t(DI) * 2, uint64_t(s.G) * DI * 2};
        const uint32_t box[3] = {uint32_t(DI), 1u, 64u};
        if (!encode_tensor_map(&qm, 3, q_idx, dims, strides, box, DI * 2, &why)) return cudaErrorInvalidValue;
        if (!encode_tensor_map(&dm, 3, kidx_new, dims, strides, box, DI * 2, &why)) return cudaErrorInvalidValue;
    }
    {
        const uint64_t dims[4] = {uint64_t(DI), uint64_t(s.G), 128ull, uint64_t(n_pages)};
        const uint64_t strides[3] = {uint64_t(DI) * 2, uint64_t(s.G) * DI * 2, 128ull * s.G * DI * 2};
        const uint32_t box[4] = {uint32_t(DI), 1u, 128u, 1u};
        if (!encode_tensor_map(&km, 4, kidx, dims, strides, box, DI * 2, &why)) return cudaErrorInvalidValue;
    }
    const size_t q_bytes = size_t(s.G + 1) * 64 * DI * 2, tile = 128 * DI * 2;
    const size_t stages = size_t(2 * kSets) * kStage * sizeof(float);
    const int depth = int(std::min<size_t>(kMaxDepth, (kSmemLimit - 1024 - q_bytes - stages) / (kSets * tile)));
    const size_t smem = 1024 + q_bytes + size_t(depth) * kSets * tile + stages;
    cudaError_t e = cudaFuncSetAttribute(k_score_tree<DI>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    return launch_kernel(k_score_tree<DI>, dim3(unsigned(sm_count())), dim3(kThreads), smem, st, true, qm, km, dm, bt,
                         ctx, node_off, anc, n_rows, n_req, n_pages, s.G, s.max_blocks, depth, scores, err);
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
