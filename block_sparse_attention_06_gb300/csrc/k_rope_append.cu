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
// times the position, modulo 2^64, is the fraction of a turn with the error of inv_freq / 2 pi in 64-bit floating point
// and 2^-64 of a turn per position alone.  Cosine and sine are worked out from it to 2^-28 of themselves and rounded
// once: codes are rounded from what they turn, and an error more would move what lies next to a border.
//
// Every byte is moved once, by 16-byte loads and stores.  A warp takes 32 chunks of 8 components of one
// section (q, k, v, q_idx or k_idx) at a time, in RPC rows at once, so RPC loads of a lane are in flight; a
// vector's lanes are neighbours, so half-split partners and the largest magnitude come by shuffles.
//
// Measured (Hq = 64, G = 8, D = 128, Di = 64).  8,192 rows into bf16 caches: 66 us, 5.6 TB/s, 0.82 of the copy rate;
// into 8-bit caches: 77 us, 4.5 TB/s, 0.67: some 150 instructions per 512 bytes keep 0.62 of the issue slots
// busy, and a warp's loads wait for its arithmetic.  8 rows: 2.9 us, the latency of one launch and one
// load after the table's.  (With sincospif of the angle in fp32 65 and 75 us; its last bits move codes that lie next to a
// border.)  Two or eight rows per CTA, loads ahead of the task at hand, and CTAs that go on over batches of rows were
// slower or no faster.
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

// (y0, y1) = (y0, y1) (c0, c1) + (p0, p1) (s0, s1), two fp32 lanes per instruction.
__device__ __forceinline__ void turn2(float &y0, float &y1, float p0, float p1, float c0, float c1, float s0, float s1) {
    asm("{\n\t.reg .b64 y, p, c, s;\n\tmov.b64 y, {%0, %1};\n\tmov.b64 p, {%2, %3};\n\tmov.b64 c, {%4, %5};\n\t"
        "mov.b64 s, {%6, %7};\n\tmul.rn.f32x2 y, y, c;\n\tfma.rn.f32x2 y, p, s, y;\n\tmov.b64 {%0, %1}, y;\n\t}"
        : "+f"(y0), "+f"(y1)
        : "f"(p0), "f"(p1), "f"(c0), "f"(c1), "f"(s0), "f"(s1));
}

// gain * (cos, sin) of turn / 2^64 turns, rounded once but for 2^-28 of themselves (0.8 and 0.7 x 2^-28 at most of two
// million angles; 3.2 x 2^-28 without the error of z in z q, and one cosine in thirty near an eighth of a turn then was not
// the nearest fp32 number, where one in a hundred is not): the nearest quarter turn is taken off, and the Taylor series of
// the angle that is left (at most pi/4) run with the errors of their leading terms carried along.
__device__ __forceinline__ float2 cos_sin(unsigned long long turn, float gain) {
    const uint32_t quarters = uint32_t((turn + (1ull << 61)) >> 62);
    const long long left = (long long)(turn - ((unsigned long long)quarters << 62));   // 2^-63 half turns
    const float r = __ll2float_rn(left), r_lo = __ll2float_rn(left - (long long)r);
    constexpr float kPi = 3.14159274f, kPiLo = -8.74227766e-8f, kSixth = -0.166666672f, kSixthLo = 4.96705377e-9f;
    const float x = r * 0x1p-63f, t = x * kPi, te = fmaf(x, kPi, -t) + fmaf(x, kPiLo, r_lo * 0x1p-63f * kPi);   // angle
    const float z = t * t, ze = fmaf(t, t, -z) + 2.f * t * te;                                                  // squared
    // 1 - z/2 + z q, q = z (1/4! - z/6! + z^2/8! - z^3/10!); the error of z turns both by ze (2 q - 1/2)
    const float q = z * fmaf(z, fmaf(z, fmaf(z, -2.75573192e-7f, 2.48015873e-5f), -1.38888889e-3f), 4.16666667e-2f);
    const float ch = fmaf(-0.5f, z, 1.f), ct = fmaf(z, q, fmaf(ze, fmaf(2.f, q, -0.5f), fmaf(-0.5f, z, 1.f - ch)));
    const float c = ch + ct, c_lo = (ch - c) + ct;
    // t - t z/3! + t z^2 (1/5! - z/7! + z^2/9! - z^3/11!)
    const float v = t * z, ve = fmaf(t, z, -v) + fmaf(te, z, t * ze);
    const float p = v * kSixth, pe = fmaf(v, kSixth, -p) + fmaf(v, kSixthLo, ve * kSixth);
    const float w = fmaf(z, fmaf(z, fmaf(z, -2.50521084e-8f, 2.75573192e-6f), -1.98412698e-4f), 8.33333333e-3f);
    const float sh = t + p, st = fmaf(v * z, w, ((t - sh) + p) + (te + pe));
    const float s = sh + st, s_lo = (sh - s) + st;
    const bool odd = quarters & 1u;
    const float g = quarters & 2u ? -gain : gain;
    const float c1 = odd ? -s : c, c1_lo = odd ? -s_lo : c_lo, s1 = odd ? c : s, s1_lo = odd ? c_lo : s_lo;
    return make_float2(fmaf(c1, g, c1_lo * g), fmaf(s1, g, s1_lo * g));
}

template <bool Q8, int RPC>
__global__ void __launch_bounds__(kThreads, 4) k_rope_append(const __grid_constant__ Args a) {
    __shared__ __align__(16) float cos_s[RPC][kMaxPairs], sin_s[RPC][kMaxPairs];
    __shared__ int page_s[RPC], slot_s[RPC];   // page -1: nothing of the row is written
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row0 = blockIdx.x * RPC;

    const int nq = a.Hq * a.D / 256, nk = (a.G * a.D + 255) / 256, ni = a.index ? (a.G * a.Di + 255) / 256 : 0;
    const int n_tasks = nq + 2 * nk + 2 * ni;
    struct Task {
        int sec, chunk, width, heads;    // section: 0 q, 1 k, 2 v, 3 q_idx, 4 k_idx; the lane's chunk in it
    };
    auto task = [&](int t) {
        Task x;
        int first;
        if (t < nq) x.sec = 0, first = 0;
        else if (t < nq + nk) x.sec = 1, first = nq;
        else if (t < nq + 2 * nk) x.sec = 2, first = nq + nk;
        else if (t < nq + 2 * nk + ni) x.sec = 3, first = nq + 2 * nk;
        else x.sec = 4, first = nq + 2 * nk + ni;
        x.chunk = (t - first) * 32 + lane;
        x.width = x.sec >= 3 ? a.Di : a.D;
        x.heads = x.sec == 0 ? a.Hq : a.G;
        return x;
    };
    auto load = [&](const Task &x, uint4 (&v)[RPC]) {
        const bool in = x.chunk < x.heads * (x.width >> 3);
        const uint16_t *src = a.src[x.sec] + size_t(x.chunk) * 8 + (long long)row0 * a.stride[x.sec];
#pragma unroll
        for (int k = 0; k < RPC; ++k) {
            v[k] = make_uint4(0u, 0u, 0u, 0u);
            if (in && row0 + k < a.n_rows) v[k] = ldg_stream_v4(src + k * a.stride[x.sec]);
        }
    };
    uint4 v[RPC];
    int t = blockIdx.y * (kThreads / 32) + warp;
    Task x = {};
    if (t < n_tasks) {                   // on their way while the angles are worked out
        x = task(t);
        load(x, v);
    }

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
        // Half-split pairs come eight to a chunk: the first four of all chunks, then the second four, so that the lanes of
        // a vector read neighbouring 16 bytes.
        const bool idx = i >= half;
        const int j = idx ? i - half : i, quarter = (idx ? a.rot_idx : a.rot) >> 2;
        const int at = (idx ? 64 : 0) + (a.interleaved ? j : (j >> 2 & 1) * quarter + (j >> 3) * 4 + (j & 3));
#pragma unroll
        for (int k = 0; k < RPC; ++k) {
            const int r = row0 + k;
            const unsigned long long pos = r < a.n_rows ? (unsigned long long)(long long)a.q_pos[r] : 0ull;
            const float2 y = cos_sin(turn * pos, a.gain);
            cos_s[k][at] = y.x;
            sin_s[k][at] = y.y;
        }
    }
    __syncthreads();

    while (t < n_tasks) {
        const int sec = x.sec, chunk = x.chunk;
        const int lv = __ffs(x.width) - 4, lpv = 1 << lv;    // lanes of one vector: 4, 8 or 16
        const bool in = chunk < x.heads << lv;
        const int head = chunk >> lv, cpos = chunk & (lpv - 1);
        const int rot = sec == 2 ? 0 : sec >= 3 ? a.rot_idx : a.rot;
        const bool cached = sec == 1 || sec == 2 || sec == 4;
        const int which = sec == 4 ? 2 : sec - 1;            // of the caches
        // which lane holds the partners, and which cosines turn this chunk
        const int hc = rot >> 4;                             // chunks of half the rotated part
        const bool turned = cpos < 2 * hc;
        const bool upper = !a.interleaved && turned && cpos >= hc;
        const int partner = a.interleaved || !turned ? lane : upper ? lane - hc : lane + hc;
        const uint32_t flip = upper ? 0u : 0x80008000u;      // (a, b) -> (a cos - b sin, b cos + a sin)
        const int at = (sec >= 3 ? 64 : 0) + (upper ? cpos - hc : cpos) * 4;
#pragma unroll
        for (int k = 0; k < RPC; ++k) {
            const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
            float y[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                y[2 * i] = bf16_lo(w[i]);
                y[2 * i + 1] = bf16_hi(w[i]);
            }
            if (rot > 0) {   // uniform in the warp
                if (a.interleaved) {
                    if (turned) {
                        const float4 c = *reinterpret_cast<const float4 *>(&cos_s[k][at]);
                        const float4 s = *reinterpret_cast<const float4 *>(&sin_s[k][at]);
                        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float u = y[2 * i], z = y[2 * i + 1];
                            y[2 * i] = u * cc[i] - z * ss[i];
                            y[2 * i + 1] = z * cc[i] + u * ss[i];
                        }
                    }
                } else {
                    uint32_t p[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) p[i] = __shfl_sync(0xffffffffu, w[i], partner) ^ flip;
                    if (turned) {
#pragma unroll
                        for (int i = 0; i < 4; i += 2) {
                            const float4 c = *reinterpret_cast<const float4 *>(&cos_s[k][at + (i >> 1) * (rot >> 2)]);
                            const float4 s = *reinterpret_cast<const float4 *>(&sin_s[k][at + (i >> 1) * (rot >> 2)]);
                            turn2(y[2 * i], y[2 * i + 1], bf16_lo(p[i]), bf16_hi(p[i]), c.x, c.y, s.x, s.y);
                            turn2(y[2 * i + 2], y[2 * i + 3], bf16_lo(p[i + 1]), bf16_hi(p[i + 1]), c.z, c.w, s.z, s.w);
                        }
                    }
                }
            }
            const int page = page_s[k], slot = slot_s[k];
            const bool live = in && page >= 0;
            if (Q8 && cached) {
                uint32_t amax = 0u;
#pragma unroll
                for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(y[i]) & 0x7fffffffu);
                for (int o = 1; o < lpv; o <<= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                const bool bad = amax >= 0x7f800000u;        // a NaN or an infinity among the components
                const int e = bad ? 0 : q8_exponent(amax);
                const float inv = exp2i(-e);
                uint2 code;
                code.x = pack_e4m3x2(y[0] * inv, y[1] * inv) | pack_e4m3x2(y[2] * inv, y[3] * inv) << 16;
                code.y = pack_e4m3x2(y[4] * inv, y[5] * inv) | pack_e4m3x2(y[6] * inv, y[7] * inv) << 16;
                if (bad) code = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
                if (live) {
                    const size_t line = (size_t(page) * a.G + head) * 128 + slot;
                    *reinterpret_cast<uint2 *>(a.dst[which] + line * x.width + cpos * 8) = code;
                    if (cpos == 0) {
                        a.scale[which][line] = bad ? uint8_t(255) : uint8_t(e + 127);
                        if (bad) raise_flag(a.err, MSA_FLAG_NAN);
                    }
                }
            } else if (live) {
                uint4 o = v[k];                              // what does not turn goes on as it is
                if (turned)
                    o = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                                   pack_bf16x2(y[6], y[7]));
                uint16_t *dst;
                if (sec == 0) dst = a.q_out + size_t(row0 + k) * a.Hq * a.D + size_t(chunk) * 8;
                else if (sec == 3) dst = a.q_idx_out + size_t(row0 + k) * a.G * a.Di + size_t(chunk) * 8;
                else
                    dst = reinterpret_cast<uint16_t *>(a.dst[which]) +
                          ((size_t(page) * 128 + slot) * a.G + head) * x.width + cpos * 8;
                *reinterpret_cast<uint4 *>(dst) = o;
            }
        }
        t += gridDim.y * (kThreads / 32);
        if (t < n_tasks) {
            x = task(t);
            load(x, v);
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
    // fractions of a turn and keep four loads per lane in flight.  Both, in us, bf16 / 8-bit: 8 rows
    // 2.6 and 9.1 / 2.9 and 11.1; 304 rows 7.5 and 11.4 / 8.0 and 13.5; 500 rows 11.9 and 12.3 / 12.1 and 13.9; 608 rows
    // 14.4 and 12.7 / 14.7 and 14.4; 2,048 rows 44 and 21 / 46 and 24.
    const int tasks = s.Hq * s.D / 256 + 2 * ((s.G * s.D + 255) / 256) + (a.index ? 2 * ((s.G * s.Di + 255) / 256) : 0);
    const bool few = 2LL * p.n_rows < 7LL * sm_count();
    const dim3 grid(unsigned(few ? p.n_rows : (p.n_rows + 3) / 4), unsigned(few ? (tasks + 7) / 8 : 1));
    const bool q8 = p.scale[0] != nullptr;
    void (*k)(Args) = q8 ? (few ? k_rope_append<true, 1> : k_rope_append<true, 4>)
                         : (few ? k_rope_append<false, 1> : k_rope_append<false, 4>);
    return launch_kernel(k, grid, dim3(kThreads), 0, st, false, a);
}

}  // namespace msa
