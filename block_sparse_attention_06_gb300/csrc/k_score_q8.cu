// Decode index scan over 8-bit index keys: score = max over a block's visible tokens of q_idx . kidx.
//
// A token and group is Di codes and a scale byte, half of the bf16 scan's bytes, and the scan is bound by
// them.  The dot products run on the 8-bit tensor cores (mma.sync m16n8k32, tokens = M): the codes go from
// global memory to the A operand as they are, and q_idx is the B operand in three e4m3 pieces whose sum is q_idx
// (msa_q8.cuh), so neither side is rounded.  hi and lo pieces fill the even and odd columns of the eight, so
// every lane of a quad holds the whole result of its tokens; which lane goes on with a tile's tokens is dealt by
// turns.  Components are summed in the order that suits the loads: the four lanes of a quad take a quarter
// of the vector each (16 or 8 consecutive bytes).
//
// One warp per (row, block, group): its slice is one contiguous run, read in half-tiles of 8 loads a lane.
#include "msa_internal.h"
#include "msa_q8.cuh"

namespace msa {
namespace {

constexpr int kWarps = 8;

template <int DI>
struct Words;   // the bytes that a lane reads of one token
template <>
struct Words<64> {
    uint4 w;
    __device__ __forceinline__ void load(const uint8_t *p) { w = ldg_stream_v4(p); }
    __device__ __forceinline__ uint32_t operator[](int i) const { return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w; }
};
template <>
struct Words<32> {
    uint2 w;
    __device__ __forceinline__ void load(const uint8_t *p) {
        asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(w.x), "=r"(w.y) : "l"(p));
    }
    __device__ __forceinline__ uint32_t operator[](int i) const { return i == 0 ? w.x : w.y; }
};

template <int DI>
__global__ void __launch_bounds__(kWarps * 32) k_score_q8(
    const uint16_t *__restrict__ q_idx, const uint8_t *__restrict__ kidx, const uint8_t *__restrict__ kscale,
    const int32_t *__restrict__ block_table, const int32_t *__restrict__ q_req, const int32_t *__restrict__ q_pos,
    const int32_t *__restrict__ seq_lens, int G, int n_req, int n_pages, int max_blocks, long long n_units,
    float *__restrict__ scores, int32_t *err) {
    constexpr int NW = DI / 16;      // words of a lane per token
    constexpr int KS = DI / 32;      // MMAs per tile and piece
    const int lane = threadIdx.x & 31;
    const long long unit = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);   // (row, block, group)
    pdl_wait();
    pdl_trigger();
    if (unit >= n_units) return;
    const int g = int(unit % G);
    const long long rb = unit / G;
    const int r = int(rb / max_blocks), j = int(rb - (long long)r * max_blocks);
    float *const out = scores + (size_t(r) * G + g) * max_blocks + j;

    const int p = q_pos ? q_pos[r] : seq_lens[r] - 1;
    const int req = q_req ? q_req[r] : r;
    int page = -1;
    bool bad = p < 0 || req < 0 || req >= n_req || (p >> 7) >= max_blocks;
    const bool candidate = !bad && j <= (p >> 7);
    if (candidate) {
        page = block_table[size_t(req) * max_blocks + j];
        bad = page < 0 || page >= n_pages;
    }
    if (!candidate || bad) {
        if (lane == 0) {
            *out = -INFINITY;
            if (bad && (candidate || j == 0)) raise_flag(err, MSA_FLAG_BOUNDS);
        }
        return;
    }

    const int rr = lane >> 2, c = lane & 3;
    const uint8_t *base = kidx + (size_t(page) * G + g) * 128 * DI + rr * DI + c * (DI / 4);
    const uint8_t *sbase = kscale + (size_t(page) * G + g) * 128 + rr;
    Words<DI> k[8];                  // tiles of 16 tokens: rows rr and rr + 8
#pragma unroll
    for (int i = 0; i < 8; ++i) k[i].load(base + i * 8 * DI);
    uint32_t sb[4];                  // scales of the tokens that this lane goes on with: tiles c and c + 4
#pragma unroll
    for (int i = 0; i < 4; ++i) sb[i] = __ldg(sbase + 16 * (c + 4 * (i >> 1)) + 8 * (i & 1));

    // this lane's quarter of q_idx in pieces
    float x[DI / 4];
    const uint4 *qp = reinterpret_cast<const uint4 *>(q_idx + (size_t(r) * G + g) * DI + c * (DI / 4));
    uint32_t amax = 0u;
#pragma unroll
    for (int i = 0; i < DI / 32; ++i) {
        const uint4 w = __ldg(qp + i);
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            x[i * 8 + 2 * h] = bf16_lo(ww[h]);
            x[i * 8 + 2 * h + 1] = bf16_hi(ww[h]);
        }
    }
#pragma unroll
    for (int i = 0; i < DI / 4; ++i) amax = max(amax, __float_as_uint(x[i]) & 0x7fffffffu);
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const bool finite = amax < 0x7f800000u;
    const int e = finite ? q8_exponent(amax) : 0;
    const float inv = exp2i(-e), qs = finite ? exp2i(e) : __uint_as_float(0x7fffffffu);
    uint32_t bh[NW], br[NW];         // columns: hi (even) or lo (odd); the rest (even) or nothing (odd)
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        float y[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) y[h] = x[4 * i + h] * inv;
        uint32_t hi, lo, re;
        q8_pieces(y, hi, lo, re);
        bh[i] = rr & 1 ? lo : hi;
        br[i] = rr & 1 ? 0u : re;
    }

    const int lim = p - j * 128;     // tokens t <= lim are visible
    float best = -INFINITY;
    float s[4];                      // the dot products of this lane's tokens
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            float a[4] = {0.f, 0.f, 0.f, 0.f}, b[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                mma_e4m3(a, k[2 * m][2 * ks], k[2 * m + 1][2 * ks], k[2 * m][2 * ks + 1], k[2 * m + 1][2 * ks + 1],
                         bh[2 * ks], bh[2 * ks + 1]);
                mma_e4m3(b, k[2 * m][2 * ks], k[2 * m + 1][2 * ks], k[2 * m][2 * ks + 1], k[2 * m + 1][2 * ks + 1],
                         br[2 * ks], br[2 * ks + 1]);
            }
            if (m == c) {            // a select: every lane runs the MMAs
                s[2 * hf] = a[0] + (a[1] * kQ8LoScale + b[0] * kQ8ReScale);
                s[2 * hf + 1] = a[2] + (a[3] * kQ8LoScale + b[2] * kQ8ReScale);
            }
        }
        if (hf == 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) k[i].load(base + (64 + i * 8) * DI);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = 16 * (c + 4 * (i >> 1)) + 8 * (i & 1) + rr;
        if (t <= lim) best = fmax_nan(best, s[i] * q8_scale(sb[i]) * qs);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) best = fmax_nan(best, __shfl_xor_sync(0xffffffffu, best, o));
    if (lane == 0) *out = best;
}

}  // namespace

cudaError_t launch_score_q8(const void *q_idx, const CacheQ8 &c, const int32_t *block_table, const int32_t *q_req,
                            const int32_t *q_pos, const int32_t *seq_lens, int n_rows, int n_req, int n_pages,
                            const Shape &s, float *scores, int32_t *err, cudaStream_t st, bool pdl) {
    const long long units = 1LL * n_rows * s.max_blocks * s.G;
    if (units <= 0) return cudaSuccess;
    const long long grid = (units + kWarps - 1) / kWarps;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    auto k = s.Di == 64 ? k_score_q8<64> : k_score_q8<32>;
    return launch_kernel(k, dim3(unsigned(grid)), dim3(kWarps * 32), 0, st, pdl, static_cast<const uint16_t *>(q_idx),
                         static_cast<const uint8_t *>(c.kidx), static_cast<const uint8_t *>(c.kidx_scale), block_table,
                         q_req, q_pos, seq_lens, s.G, n_req, n_pages, s.max_blocks, units, scores, err);
}

}  // namespace msa
