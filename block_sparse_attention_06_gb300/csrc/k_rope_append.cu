// Rotary positions and the append: one pass over the rows that a layer's projections give.
//
// A pair (a, b) of components turns by the angle pos * inv_freq[i]:
//   (a, b) -> gain * (a cos - b sin, b cos + a sin),
// pairs being components (i, i + rot/2) or (2i, 2i + 1), of the first `rot` components of q and k heads and
// the first `rot_idx` of the index vectors.  q and q_idx go to dense outputs, k, v and k_idx into the paged
// caches: as bf16, or as e4m3 rows with a scale (msa_q8.cuh), quantised from the fp32 rotation, so each value
// is rounded once.
//
// The angle of a far position loses its digits in fp32 (position 2^20 turns the first pair by 2^20 radians),
// so it is counted in turns in 64-bit fixed point: inv_freq / 2 pi, modulo one turn, as a fraction of 2^64;
// times the position, modulo 2^64, is the exact fraction of a turn.
//
// Memory-bound (16-byte loads and stores, every byte once).  A warp takes 32 chunks of 8 components of one
// section (q, k, v, q_idx or k_idx) at a time, in RPC rows at once, so RPC loads of a lane are in flight; a
// vector's lanes are neighbours, so half-split partners and the largest magnitude come by shuffles.
#include "msa_internal.h"
#include "msa_q8.cuh"

namespace msa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 64 + 32;   // of q and k (D <= 128), then of the index vectors (Di <= 64)

struct Args {
    const uint16_t *src[5];   // q, k, v, q_idx, k_idx
    long long stride[5];      // elements from row to row
    uint16_t *q_out, *q_idx_out;
    uint8_t *dst[3];          // k, v, k_idx caches (bf16 or codes)
    uint8_t *scale[3];        // their scales (8-bit caches)
    const double *inv_freq, *inv_freq_idx;
    const int32_t *block_table, *q_req, *q_pos;
    int n_rows, n_req, n_pages, max_blocks, Hq, G, D, Di, rot, rot_idx, interleaved, index;
    float gain;
    int32_t *err;
};

template <bool Q8, int RPC>
__global__ void __launch_bounds__(kThreads) k_rope_append(const __grid_constant__ Args a) {
    __shared__ __align__(16) float cos_s[RPC][kMaxPairs], sin_s[RPC][kMaxPairs];
    __shared__ int page_s[RPC], slot_s[RPC];   // page -1: nothing of the row is written
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row0 = blockIdx.x * RPC;

    if (tid < RPC) {
        const int r = row0 + tid;
        int page = -1, slot = 0;
        if (r < a.n_rows) {
            const int req = a.q_req[r], pos = a.q_pos[r];
            if (req != -1) {   // -1: a padding row
                if (req >= 0 && req < a.n_req && pos >= 0 && (pos >> 7) < a.max_blocks) {
                    page = a.block_table[size_t(req) * a.max_blocks + (pos >> 7)];
                    slot = pos & 127;
                }
                if (page < 0 || page >= a.n_pages) {
                    page = -1;
                    if (blockIdx.y == 0) raise_flag(a.err, MSA_FLAG_BOUNDS);
                }
            }
        }
        page_s[tid] = page;
        slot_s[tid] = slot;
    }
    const int half = a.rot >> 1, pairs = half + (a.index ? a.rot_idx >> 1 : 0);
    for (int i = tid; i < pairs; i += kThreads) {
        double f = (i < half ? a.inv_freq[i] : a.inv_freq_idx[i - half]) * 0.15915494309189534561;   // turns
        f -= floor(f);
        const unsigned long long turn = __double2ull_rz(f * 18446744073709551616.0);
#pragma unroll
        for (int k = 0; k < RPC; ++k) {
            const int r = row0 + k;
            const unsigned long long pos = r < a.n_rows ? (unsigned long long)(long long)a.q_pos[r] : 0ull;
            float s, c;
            sincospif(__ll2float_rn((long long)(turn * pos)) * 0x1p-63f, &s, &c);   // half turns in [-1, 1]
            const int at = i < half ? i : i - half + 64;
            cos_s[k][at] = c * a.gain;
            sin_s[k][at] = s * a.gain;
        }
    }
    __syncthreads();

    const int nq = a.Hq * a.D / 256, nk = (a.G * a.D + 255) / 256, ni = a.index ? (a.G * a.Di + 255) / 256 : 0;
    const int n_tasks = nq + 2 * nk + 2 * ni;
    for (int t = blockIdx.y * (kThreads / 32) + warp; t < n_tasks; t += gridDim.y * (kThreads / 32)) {
        // section: 0 q, 1 k, 2 v, 3 q_idx, 4 k_idx
        int sec, first;
        if (t < nq) sec = 0, first = 0;
        else if (t < nq + nk) sec = 1, first = nq;
        else if (t < nq + 2 * nk) sec = 2, first = nq + nk;
        else if (t < nq + 2 * nk + ni) sec = 3, first = nq + 2 * nk;
        else sec = 4, first = nq + 2 * nk + ni;
        const int width = sec >= 3 ? a.Di : a.D, heads = sec == 0 ? a.Hq : a.G;
        const int lpv = width >> 3;                          // lanes of one vector: 4, 8 or 16
        const int chunk = (t - first) * 32 + lane;           // of 8 components
        const bool in = chunk < heads * lpv;
        const int head = chunk / lpv, cpos = chunk - head * lpv;
        const int rot = sec == 2 ? 0 : sec >= 3 ? a.rot_idx : a.rot;
        const uint16_t *src = a.src[sec] + size_t(chunk) * 8;

        uint4 v[RPC];
#pragma unroll
        for (int k = 0; k < RPC; ++k) {
            v[k] = make_uint4(0u, 0u, 0u, 0u);
            if (in && page_s[k] >= 0)
                v[k] = ldg_stream_v4(src + (long long)(row0 + k) * a.stride[sec]);
        }
        // which lane holds the partners, and which cosines turn this chunk
        const int hc = rot >> 4;                             // chunks of half the rotated part
        const bool turned = cpos < 2 * hc;
        const bool upper = !a.interleaved && turned && cpos >= hc;
        const int partner = a.interleaved || !turned ? lane : upper ? lane - hc : lane + hc;
        const int at = (sec >= 3 ? 64 : 0) + (a.interleaved ? cpos * 4 : (upper ? cpos - hc : cpos) * 8);
#pragma unroll
        for (int k = 0; k < RPC; ++k) {
            float x[8] = {bf16_lo(v[k].x), bf16_hi(v[k].x), bf16_lo(v[k].y), bf16_hi(v[k].y),
                          bf16_lo(v[k].z), bf16_hi(v[k].z), bf16_lo(v[k].w), bf16_hi(v[k].w)};
            if (rot > 0) {   // uniform in the warp
                if (a.interleaved) {
                    if (turned) {
                        const float4 c = *reinterpret_cast<const float4 *>(&cos_s[k][at]);
                        const float4 s = *reinterpret_cast<const float4 *>(&sin_s[k][at]);
                        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float u = x[2 * i], w = x[2 * i + 1];
                            x[2 * i] = u * cc[i] - w * ss[i];
                            x[2 * i + 1] = w * cc[i] + u * ss[i];
                        }
                    }
                } else {
                    uint32_t p[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) p[i] = __shfl_sync(0xffffffffu, p[i], partner);
                    if (turned) {
                        const float sign = upper ? 1.f : -1.f;
#pragma unroll
                        for (int i = 0; i < 8; i += 4) {
                            const float4 c = *reinterpret_cast<const float4 *>(&cos_s[k][at + i]);
                            const float4 s = *reinterpret_cast<const float4 *>(&sin_s[k][at + i]);
                            x[i] = x[i] * c.x + sign * bf16_lo(p[i / 2]) * s.x;
                            x[i + 1] = x[i + 1] * c.y + sign * bf16_hi(p[i / 2]) * s.y;
                            x[i + 2] = x[i + 2] * c.z + sign * bf16_lo(p[i / 2 + 1]) * s.z;
                            x[i + 3] = x[i + 3] * c.w + sign * bf16_hi(p[i / 2 + 1]) * s.w;
                        }
                    }
                }
            }
            const int page = page_s[k], slot = slot_s[k];
            const bool live = in && page >= 0;
            const bool cached = sec == 1 || sec == 2 || sec == 4;
            if (Q8 && cached) {
                const int which = sec == 4 ? 2 : sec - 1;
                uint32_t amax = 0u;
#pragma unroll
                for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(x[i]) & 0x7fffffffu);
                for (int o = 1; o < lpv; o <<= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                const bool bad = amax >= 0x7f800000u;        // a NaN or an infinity among the components
                const int e = bad ? 0 : q8_exponent(amax);
                const float inv = exp2i(-e);
                uint2 code;
                code.x = pack_e4m3x2(x[0] * inv, x[1] * inv) | pack_e4m3x2(x[2] * inv, x[3] * inv) << 16;
                code.y = pack_e4m3x2(x[4] * inv, x[5] * inv) | pack_e4m3x2(x[6] * inv, x[7] * inv) << 16;
                if (bad) code = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
                if (live) {
                    const size_t line = (size_t(page) * a.G + head) * 128 + slot;
                    *reinterpret_cast<uint2 *>(a.dst[which] + line * width + cpos * 8) = code;
                    if (cpos == 0) {
                        a.scale[which][line] = bad ? uint8_t(255) : uint8_t(e + 127);
                        if (bad) raise_flag(a.err, MSA_FLAG_NAN);
                    }
                }
            } else if (live) {
                const uint4 w = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                           pack_bf16x2(x[6], x[7]));
                if (sec == 0) {
                    *reinterpret_cast<uint4 *>(a.q_out + size_t(row0 + k) * a.Hq * a.D + size_t(chunk) * 8) = w;
                } else if (sec == 3) {
                    *reinterpret_cast<uint4 *>(a.q_idx_out + size_t(row0 + k) * a.G * a.Di + size_t(chunk) * 8) = w;
                } else {
                    uint16_t *dst = reinterpret_cast<uint16_t *>(a.dst[sec == 4 ? 2 : sec - 1]);
                    *reinterpret_cast<uint4 *>(dst + ((size_t(page) * 128 + slot) * a.G + head) * width + cpos * 8) =
                        sec == 2 ? v[k] : w;
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_rope_append(const RopeAppend &p, const Shape &s, cudaStream_t st) {
    if (p.n_rows <= 0) return cudaSuccess;
    Args a = {};
    for (int i = 0; i < 5; ++i) {
        a.src[i] = static_cast<const uint16_t *>(p.src[i]);
        a.stride[i] = p.stride[i];
    }
    a.q_out = static_cast<uint16_t *>(p.q_out);
    a.q_idx_out = static_cast<uint16_t *>(p.q_idx_out);
    for (int i = 0; i < 3; ++i) {
        a.dst[i] = static_cast<uint8_t *>(p.dst[i]);
        a.scale[i] = static_cast<uint8_t *>(p.scale[i]);
    }
    a.inv_freq = p.inv_freq;
    a.inv_freq_idx = p.inv_freq_idx;
    a.block_table = p.block_table;
    a.q_req = p.q_req;
    a.q_pos = p.q_pos;
    a.n_rows = p.n_rows;
    a.n_req = p.n_req;
    a.n_pages = p.n_pages;
    a.max_blocks = s.max_blocks;
    a.Hq = s.Hq;
    a.G = s.G;
    a.D = s.D;
    a.Di = s.Di;
    a.rot = p.rot;
    a.rot_idx = p.rot_idx;
    a.interleaved = p.interleaved;
    a.index = p.src[3] != nullptr;
    a.gain = p.gain;
    a.err = p.err;
    // Few rows: one row per CTA and one task per warp, for latency.  Many: four rows per CTA share the
    // fractions of a turn and keep four loads per lane in flight.
    const int tasks = s.Hq * s.D / 256 + 2 * ((s.G * s.D + 255) / 256) + (a.index ? 2 * ((s.G * s.Di + 255) / 256) : 0);
    const bool few = p.n_rows < 4 * sm_count();
    const dim3 grid(unsigned(few ? p.n_rows : (p.n_rows + 3) / 4), unsigned(few ? (tasks + 7) / 8 : 1));
    const bool q8 = p.scale[0] != nullptr;
    void (*k)(Args) = q8 ? (few ? k_rope_append<true, 1> : k_rope_append<true, 4>)
                         : (few ? k_rope_append<false, 1> : k_rope_append<false, 4>);
    return launch_kernel(k, grid, dim3(kThreads), 0, st, false, a);
}

}  // namespace msa
