// 8-bit pages read back as bf16 pages: value = code * 2^(b - 127), a bf16 number already, so nothing is
// rounded.  The prefill kernels take bf16 pages; a chunk's context is read back once per layer and chunk.
//
// Pure streaming: 16 codes (16 bytes) per lane and load, 32 bytes per lane and store.  Lanes follow the
// output's order ([token][group][width]), so a warp stores whole lines; its loads are runs of `width` bytes.
// Measured: 68,192 tokens of G = 8, D = 128, Di = 64 (525 MB in all) in 82 us, 6.4 TB/s, 0.94 of the copy rate; four
// loads in flight and 16-byte stores took 113 us.  Three short requests: 3.7 us, one launch and two dependent loads.
#include "msa_internal.h"
#include "msa_q8.cuh"

namespace msa {
namespace {

constexpr int kThreads = 256;

struct Args {
    const uint8_t *code[3], *scale[3];
    uint8_t *out[3];
    const int32_t *bt_in, *bt_out, *lens;
    int n_pages, n_pages_out, max_blocks, G, width[3];
    int32_t *err;
};

__device__ __forceinline__ uint32_t bf16_pair(uint32_t codes, float s) {
    const float2 f = unpack_e4m3x2(codes);
    return pack_bf16x2(f.x * s, f.y * s);
}

__device__ __forceinline__ void st_global_v8(void *p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// EVEN: a token's chunks divide the CTA's threads, so a thread keeps its group and column and steps over tokens.
template <bool EVEN>
__global__ void __launch_bounds__(kThreads) k_cache_read(const __grid_constant__ Args a) {
    constexpr int U = 8;                 // loads in flight per lane
    const int b = blockIdx.x / a.max_blocks, j = blockIdx.x - b * a.max_blocks;
    const int which = blockIdx.y;
    const int to = a.bt_out[blockIdx.x];
    const int from = a.bt_in[blockIdx.x];
    const int n_tok = int(min(128LL, a.lens[b] - j * 128LL));   // 64 bits: a length may be any number
    if (to < 0 || n_tok <= 0) return;
    if (from < 0 || from >= a.n_pages || to >= a.n_pages_out) {
        if (threadIdx.x == 0 && which == 0) raise_flag(a.err, MSA_FLAG_BOUNDS);
        return;
    }
    const int width = a.width[which], cpv = width >> 4, per_tok = a.G * cpv;   // chunks of 16 per vector, per token
    const uint8_t *code = a.code[which] + size_t(from) * a.G * 128 * width;
    const uint8_t *scale = a.scale[which] + size_t(from) * a.G * 128;
    uint8_t *out = a.out[which] + size_t(to) * 128 * a.G * width * 2;
    const int n = n_tok * per_tok;
    const int t0 = threadIdx.x / per_tok, g0 = (threadIdx.x - t0 * per_tok) / cpv;
    const int c0 = threadIdx.x - t0 * per_tok - g0 * cpv, dt = kThreads / per_tok;
    for (int i0 = threadIdx.x, t1 = t0; i0 < n; i0 += U * kThreads, t1 += U * dt) {
        uint4 w[U];
        uint8_t s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * kThreads;
            if (i < n) {
                int t = t1 + u * dt, g = g0, c = c0;
                if constexpr (!EVEN) {
                    t = i / per_tok;
                    g = (i - t * per_tok) / cpv;
                    c = i - t * per_tok - g * cpv;
                }
                w[u] = ldg_stream_v4(code + (g * 128 + t) * width + c * 16);
                s[u] = __ldg(scale + g * 128 + t);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * kThreads;
            if (i < n) {
                const float f = q8_scale(s[u]);
                const uint32_t o[8] = {bf16_pair(w[u].x, f), bf16_pair(w[u].x >> 16, f), bf16_pair(w[u].y, f),
                                       bf16_pair(w[u].y >> 16, f), bf16_pair(w[u].z, f), bf16_pair(w[u].z >> 16, f),
                                       bf16_pair(w[u].w, f), bf16_pair(w[u].w >> 16, f)};
                st_global_v8(out + size_t(i) * 32, o);
            }
        }
    }
}

}  // namespace

cudaError_t launch_cache_read(const CacheQ8 &c, const int32_t *bt_in, const int32_t *bt_out, const int32_t *lens,
                              int n_req, int n_pages, int n_pages_out, const Shape &s, void *k, void *v, void *kidx,
                              int32_t *err, cudaStream_t st) {
    Args a = {};
    const void *code[3] = {c.k, c.v, c.kidx}, *scale[3] = {c.k_scale, c.v_scale, c.kidx_scale};
    void *out[3] = {k, v, kidx};
    for (int i = 0; i < 3; ++i) {
        a.code[i] = static_cast<const uint8_t *>(code[i]);
        a.scale[i] = static_cast<const uint8_t *>(scale[i]);
        a.out[i] = static_cast<uint8_t *>(out[i]);
        a.width[i] = i == 2 ? s.Di : s.D;
    }
    a.bt_in = bt_in;
    a.bt_out = bt_out;
    a.lens = lens;
    a.n_pages = n_pages;
    a.n_pages_out = n_pages_out;
    a.max_blocks = s.max_blocks;
    a.G = s.G;
    a.err = err;
    const bool even = kThreads % (s.G * (s.D / 16)) == 0 && (!kidx || kThreads % (s.G * (s.Di / 16)) == 0);
    const dim3 grid(unsigned(n_req) * unsigned(s.max_blocks), kidx ? 3u : 2u);
    return launch_kernel(even ? k_cache_read<true> : k_cache_read<false>, grid, dim3(kThreads), 0, st, false, a);
}

}  // namespace msa
