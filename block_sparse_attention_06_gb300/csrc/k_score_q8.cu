// Decode index scan over 8-bit index keys: score = max over a block's visible tokens of q_idx . kidx.
//
// A token and group is Di codes and a scale byte, half of the bf16 scan's bytes, and the scan is bound by
// them.  The dot products run on f16 MMAs (m16n8k16, tokens = M): a code is an f16 number, and q_idx is one times a
// power of two (msa_q8.cuh), so neither side is rounded.  All eight columns hold q_idx, so every lane of a quad has the
// results of its tokens; which lane goes on with a tile's tokens is dealt by turns.  Components are summed in the
// order that suits the loads: the four lanes of a quad take a quarter of the vector each.  (The 8-bit MMA of warps
// takes the codes as they are, but is three times as many instructions: it unpacks its operands itself, every time.)
//
// A unit is the slice of one block and group, one contiguous run of 128 Di codes and one of 128 scales.  One CTA per
// SM; each of its warps streams a contiguous range of the units that exist (row, then group, then block) through
// a ring of its own, filled by bulk copies that the warp itself issues as it frees a stage: some 200 KB are in flight
// per SM, no warp waits for another, and a range keeps q_idx in registers over the blocks of a (row, group).
//
// Measured: 8 x 60,000 tokens, G = 8, Di = 64 (250 MB) in 42 us, 0.88 of the copy rate (a CTA per page with loads into
// registers took 67); what is left is the start and the end of the stream.  One request of 1,500 tokens: 4.4 us, one
// launch and the chain q_pos, table, keys.
#include "msa_internal.h"
#include "msa_q8.cuh"

#include <algorithm>

namespace msa {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;

template <int DI>
struct Smem {
    static constexpr int NST = DI == 64 ? 3 : 6;          // stages per warp
    static constexpr int CODES = 128 * DI;
    alignas(128) uint8_t stage[kWarps][NST][CODES + 128];   // codes, then scales
    uint64_t full[kWarps][NST];
    long long sum[kWarps];
    int start_row[kWarps];
    long long start_off[kWarps];
};

// Rows as the scan sees them: by (q_req, q_pos), or the requests themselves at seq_lens - 1.
struct Rows {
    const int32_t *q_req, *q_pos, *seq_lens;
    int n_rows, n_req, max_blocks;
    __device__ __forceinline__ int pos(int r) const { return q_pos ? q_pos[r] : seq_lens[r] - 1; }
    __device__ __forceinline__ int req(int r) const { return q_req ? q_req[r] : r; }
    // candidate blocks of row r, 0 for a bad row
    __device__ __forceinline__ int blocks(int r) const {
        const int p = pos(r), q = req(r);
        return p < 0 || q < 0 || q >= n_req || (p >> 7) >= max_blocks ? 0 : (p >> 7) + 1;
    }
};

// A place in the order of units: block j of nb of group g of row r.
struct Cursor {
    int r, g, j, nb;
    __device__ __forceinline__ bool step(const Rows &rows, int G) {   // to the next unit; true where (r, g) changes
        if (++j < nb) return false;
        j = 0;
        if (++g == G) {
            g = 0;
            do ++r;
            while (r < rows.n_rows && (nb = rows.blocks(r)) == 0);
        }
        return true;
    }
};

// First of `total` units of range i of n_ranges.
__device__ __forceinline__ long long range_begin(long long total, long long n_ranges, long long i) {
    return total / n_ranges * i + total % n_ranges * i / n_ranges;
}

template <int DI>
__global__ void __launch_bounds__(kThreads, 1) k_score_q8(const uint16_t *__restrict__ q_idx,
                                                          const uint8_t *__restrict__ kidx,
                                                          const uint8_t *__restrict__ kscale,
                                                          const int32_t *__restrict__ block_table, const Rows rows, int G,
                                                          int n_pages, float *__restrict__ scores, int32_t *err) {
    using S = Smem<DI>;
    constexpr int NST = S::NST;
    constexpr int NW = DI / 16;      // words of a lane per token, MMAs per tile
    extern __shared__ uint8_t smem_raw[];
    S &sm = *reinterpret_cast<S *>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int MB = rows.max_blocks;
    if (lane == 0) {
        for (int i = 0; i < NST; ++i) mbar_init(&sm.full[warp][i], 1);
        fence_mbar_init();
    }
    __syncwarp();
    pdl_wait();
    pdl_trigger();

    // ---------------------------------------------------------------- the range
    const long long n_ranges = (long long)gridDim.x * kWarps, gw = (long long)blockIdx.x * kWarps + warp;
    Cursor in = {rows.n_rows, 0, 0, 0};  // of the next copy
    long long n;                         // units of this warp
    if (rows.n_rows <= 32) {             // a row per lane, every warp on its own
        const int nb = lane < rows.n_rows ? rows.blocks(lane) : 0;
        if (lane < rows.n_rows && nb == 0 && gw == 0) raise_flag(err, MSA_FLAG_BOUNDS);
        long long upto = nb;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        const long long total = __shfl_sync(0xffffffffu, upto, 31) * G;
        const long long x = range_begin(total, n_ranges, gw);
        n = range_begin(total, n_ranges, gw + 1) - x;
        const int r = __ffs(__ballot_sync(0xffffffffu, x < upto * G)) - 1;   // the row that holds it
        const long long off = x - __shfl_sync(0xffffffffu, upto - nb, r & 31) * G;
        const int rnb = __shfl_sync(0xffffffffu, nb, r & 31);
        if (n > 0) in = {r, int(off / rnb), int(off % rnb), rnb};
    } else {                             // a run of rows per thread
        const int per = (rows.n_rows + kThreads - 1) / kThreads;
        const int ra = min(tid * per, rows.n_rows), rz = min(ra + per, rows.n_rows);
        long long mine = 0;
        for (int r = ra; r < rz; ++r) {
            const int nb = rows.blocks(r);
            if (nb == 0 && blockIdx.x == 0) raise_flag(err, MSA_FLAG_BOUNDS);
            mine += nb;
        }
        long long upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        if (lane == 31) sm.sum[warp] = upto;
        __syncthreads();
        long long total = 0, before = upto - mine;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += sm.sum[w];
            total += sm.sum[w];
        }
        total *= G;
        for (int w = 0; w < kWarps; ++w) {   // whose first unit lies in this thread's rows
            const long long x = range_begin(total, n_ranges, (long long)blockIdx.x * kWarps + w);
            if (x >= before * G && x < (before + mine) * G) {
                long long off = x - before * G;
                int r = ra;
                for (;; ++r) {
                    const long long u = (long long)rows.blocks(r) * G;
                    if (off < u) break;
                    off -= u;
                }
                sm.start_row[w] = r;
                sm.start_off[w] = off;
            }
        }
        __syncthreads();
        n = range_begin(total, n_ranges, gw + 1) - range_begin(total, n_ranges, gw);
        if (n > 0) {
            in.r = sm.start_row[warp];
            in.nb = rows.blocks(in.r);
            in.g = int(sm.start_off[warp] / in.nb);
            in.j = int(sm.start_off[warp] - (long long)in.g * in.nb);
        }
    }

    // ---------------------------------------------------------------- the stream
    Cursor at = in;                      // of the unit at hand
    const uint64_t policy = l2_policy_evict_first();
    int pages = -1, pages_j = 0, pages_r = -1;   // lane l: the page of block pages_j + l of row pages_r
    int stage_page = -1;                 // lane l: the page in stage l, -1 for none
    auto issue = [&](int stage) {        // the copies of unit `in`
        if (pages_r != in.r || in.j < pages_j || in.j >= pages_j + 32) {
            pages_r = in.r;
            pages_j = in.j;
            pages = in.j + lane < in.nb ? block_table[size_t(rows.req(in.r)) * MB + in.j + lane] : -1;
        }
        int page = __shfl_sync(0xffffffffu, pages, in.j - pages_j);
        if (page < 0 || page >= n_pages) {
            if (lane == 0) raise_flag(err, MSA_FLAG_BOUNDS);
            page = -1;
        }
        if (lane == stage) stage_page = page;
        if (lane == 0 && page >= 0) {
            const size_t line = (size_t(page) * G + in.g) * 128;
            mbar_arrive_expect_tx(&sm.full[warp][stage], S::CODES + 128);
            bulk_load(sm.stage[warp][stage], kidx + line * DI, S::CODES, &sm.full[warp][stage], policy);
            bulk_load(sm.stage[warp][stage] + S::CODES, kscale + line, 128, &sm.full[warp][stage], policy);
        }
        in.step(rows, G);
    };
    for (int i = 0; i < NST && i < n; ++i) issue(i);

    // blocks past the rows' own: dealt over all warps
    for (long long i = gw; i < (long long)rows.n_rows * G; i += n_ranges) {
        const int nb = rows.blocks(int(i / G));
        for (int j = nb + lane; j < MB; j += 32) scores[i * MB + j] = -INFINITY;
    }

    const int rr = lane >> 2, c = lane & 3;
    uint32_t q[NW][2];                   // q_idx: four components per word of the codes
    float qs = 0.f;
    bool fresh = true;                   // q_idx is to be read
    int lim = 0, j0 = 0, stage = 0;
    float result = -INFINITY;            // lane l: the score of block j0 + l
    uint32_t used = 0u;                  // bit s: phase of stage s
    bool ok = true;
    for (long long i = 0; i < n; ++i) {
        if (fresh) {
            fresh = false;
            j0 = at.j;
            lim = rows.pos(at.r);
            // this lane's quarter of q_idx
            float x[DI / 4];
            const uint4 *qp = reinterpret_cast<const uint4 *>(q_idx + (size_t(at.r) * G + at.g) * DI + c * (DI / 4));
            uint32_t amax = 0u;
#pragma unroll
            for (int k = 0; k < DI / 32; ++k) {
                const uint4 w = __ldg(qp + k);
                const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    x[k * 8 + 2 * h] = bf16_lo(ww[h]);
                    x[k * 8 + 2 * h + 1] = bf16_hi(ww[h]);
                }
            }
#pragma unroll
            for (int k = 0; k < DI / 4; ++k) amax = max(amax, __float_as_uint(x[k]) & 0x7fffffffu);
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            const bool finite = amax < 0x7f800000u;
            const int e = finite ? f16_exponent(amax) : 0;
            const float inv = exp2i(-e);
            qs = finite ? exp2i(e) : __uint_as_float(0x7fffffffu);
#pragma unroll
            for (int k = 0; k < NW; ++k) {
                q[k][0] = pack_f16x2(x[4 * k] * inv, x[4 * k + 1] * inv);
                q[k][1] = pack_f16x2(x[4 * k + 2] * inv, x[4 * k + 3] * inv);
            }
        }
        float best = -INFINITY;
        if (__shfl_sync(0xffffffffu, stage_page, stage) >= 0) {
            if (!__all_sync(0xffffffffu, mbar_wait(&sm.full[warp][stage], (used >> stage) & 1u, err, nullptr))) {
                ok = false;
                break;
            }
            used ^= 1u << stage;
            const uint8_t *base = sm.stage[warp][stage];
            float s[4];                  // the dot products of this lane's tokens: tiles c and c + 4, rows rr and rr + 8
#pragma unroll
            for (int m = 0; m < 8; ++m) {
                uint32_t k0[NW], k1[NW];
                const uint8_t *p = base + (16 * m + rr) * DI + c * (DI / 4);
                if constexpr (DI == 64) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(p), y = *reinterpret_cast<const uint4 *>(p + 8 * DI);
                    k0[0] = x.x, k0[1] = x.y, k0[2] = x.z, k0[3] = x.w;
                    k1[0] = y.x, k1[1] = y.y, k1[2] = y.z, k1[3] = y.w;
                } else {
                    const uint2 x = *reinterpret_cast<const uint2 *>(p), y = *reinterpret_cast<const uint2 *>(p + 8 * DI);
                    k0[0] = x.x, k0[1] = x.y;
                    k1[0] = y.x, k1[1] = y.y;
                }
                float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < NW; ++k)
                    mma_f16(a, f16_of_low(k0[k]), f16_of_low(k1[k]), f16_of_high(k0[k]), f16_of_high(k1[k]), q[k][0],
                            q[k][1]);
                if ((m & 3) == c) {      // a select: every lane runs the MMAs
                    s[2 * (m >> 2)] = a[0];
                    s[2 * (m >> 2) + 1] = a[2];
                }
            }
            const int left = lim - at.j * 128;           // tokens t <= left are visible
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int t = 16 * (c + 4 * (k >> 1)) + 8 * (k & 1) + rr;
                const float v = s[k] * q8_scale(base[S::CODES + t]) * qs;
                if (t <= left) best = fmax_nan(best, v);
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) best = fmax_nan(best, __shfl_xor_sync(0xffffffffu, best, o));
        }
        if (lane == at.j - j0) result = best;
        __syncwarp();                    // the stage has been read
        if (i + NST < n) issue(stage);
        stage = stage + 1 == NST ? 0 : stage + 1;
        // whole lines of scores
        float *const out = scores + (size_t(at.r) * G + at.g) * MB + j0;
        const int have = at.j - j0 + 1;
        fresh = at.step(rows, G);
        if (fresh || have == 32 || i + 1 == n) {
            if (lane < have) out[lane] = result;
            j0 += 32;
        }
    }
    if (!ok) {                           // a copy that did not come: the others land before the CTA leaves
        for (int i = 0; i < NST; ++i)
            if (i != stage && __shfl_sync(0xffffffffu, stage_page, i) >= 0)
                mbar_wait(&sm.full[warp][i], (used >> i) & 1u, err, nullptr);
    }
}

template <int DI>
cudaError_t launch_t(const void *q_idx, const CacheQ8 &c, const int32_t *block_table, const Rows &rows, int G, int n_pages,
                     float *scores, int32_t *err, cudaStream_t st, bool pdl) {
    const size_t smem = sizeof(Smem<DI>) + 128;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_once(allowed, reinterpret_cast<const void *>(k_score_q8<DI>), smem);
    if (e != cudaSuccess) return e;
    const long long units = 1LL * rows.n_rows * rows.max_blocks * G;
    const int grid = int(std::min<long long>((units + kWarps - 1) / kWarps, sm_count()));
    return launch_kernel(k_score_q8<DI>, dim3(unsigned(grid)), dim3(kThreads), smem, st, pdl,
                         static_cast<const uint16_t *>(q_idx), static_cast<const uint8_t *>(c.kidx),
                         static_cast<const uint8_t *>(c.kidx_scale), block_table, rows, G, n_pages, scores, err);
}

}  // namespace

cudaError_t launch_score_q8(const void *q_idx, const CacheQ8 &c, const int32_t *block_table, const int32_t *q_req,
                            const int32_t *q_pos, const int32_t *seq_lens, int n_rows, int n_req, int n_pages,
                            const Shape &s, float *scores, int32_t *err, cudaStream_t st, bool pdl) {
    if (n_rows <= 0) return cudaSuccess;
    const Rows rows = {q_req, q_pos, seq_lens, n_rows, n_req, s.max_blocks};
    return s.Di == 64 ? launch_t<64>(q_idx, c, block_table, rows, s.G, n_pages, scores, err, st, pdl)
                      : launch_t<32>(q_idx, c, block_table, rows, s.G, n_pages, scores, err, st, pdl);
}

}  // namespace msa
