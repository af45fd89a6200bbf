// Decode attention over 8-bit caches: the pages of a row's selected blocks, or a window and the first tokens.
//
// A row is one query token of one KV group; its Hq/G heads attend the row's visible tokens,
//   s_t = sm_scale * q . k_t,   out = sum_t softmax(s)_t v_t,   lse = log sum_t exp(s_t).
//
// What bounds it is the read of K and V (one byte per component, and two scale bytes per token), and with
// few rows the latency of a chain: table, K, softmax, join.  So:
//   - a unit is 32 tokens of one page, and one warp takes a unit on its own, from global memory straight into
//     MMA operands, with its own running maximum and sum: no shared memory, no barrier until the row's end.  K
//     and V of a unit are loaded together, K of the next one while this one's softmax and P V run.
//   - a row's units are dealt to the warps of a cluster of CTAs (more CTAs where there are few rows), whose
//     partials are joined through distributed shared memory, always in the same order: no workspace, no atomics.
//
// S^T = K q^T runs on the 8-bit tensor cores (m16n8k32, tokens = M, heads = N): K's codes are the A operand as
// they are, q is three e4m3 pieces that sum to it (msa_q8.cuh); the token's scale and the head's factor multiply
// the fp32 result.  O^T = V^T P^T runs on bf16 MMAs (m16n8k16, components = M): a code seeeemmm becomes the
// bf16 number s0000eeeemmm0000 = code * 2^-120 by shifts and masks (subnormal codes included, and no code gives
// a NaN or an infinity, so tokens that a row does not see cannot reach it), and P carries the token's scale
// relative to the largest that the warp has seen: P_t = p_t 2^(e_t - E + 100), so O is held times 2^(-20 - E) and
// scales of any size fit, with 100 binades between the largest and what is lost.  P is rounded to bf16, once.
//
// Layout.  In a unit lane (r, c) = (lane / 4, lane % 4) reads tokens 4r .. 4r+3 of K (its quad covers the row,
// a quarter each) and tokens 8c .. 8c+7 of V (D/8 components each): whole lines per load.  The C fragment of S^T
// then has the tokens 4r+i, i = 0 .. 3; packed over two heads and transposed by movmatrix it is the B fragment of
// P V for tokens 8c+i and 8c+4+i, which are two of the lane's eight.
#include "msa_internal.h"
#include "msa_q8.cuh"

#include <algorithm>

namespace msa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kUnit = 32;            // tokens

__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void mma_bf16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// Codes in bytes 0 and 2, or 1 and 3, of w as two bf16 numbers code * 2^-120.
__device__ __forceinline__ uint32_t bf16_even(uint32_t w) { return ((w << 4) & 0x07f007f0u) | ((w << 8) & 0x80008000u); }
__device__ __forceinline__ uint32_t bf16_odd(uint32_t w) { return ((w >> 4) & 0x07f007f0u) | (w & 0x80008000u); }

// 2^d for d <= 0, 0 below 2^-126.
__device__ __forceinline__ float pow2_down(int d) { return __uint_as_float(uint32_t(max(d + 127, 0)) << 23); }

// out = (x 2^20) 2^E for x = O 2^(-20 - E) / l, with E as a scale byte.
__device__ __forceinline__ float unscaled(float x, int e) { return x * 0x1p20f * q8_scale(uint32_t(e)); }

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ uint32_t cluster_map(uint32_t smem, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem), "r"(rank));
    return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}

struct Args {
    const uint16_t *q;
    const uint8_t *k, *k_scale, *v, *v_scale;
    const int32_t *page_table, *row_len;             // pages of the selected blocks
    const int32_t *block_table, *q_req, *q_pos;      // window
    int window, n_sink;
    int G, topk, n_req, n_pages, max_blocks, cluster;
    float sm_scale;
    uint16_t *out;
    float *lse;
    int32_t *err;
};

// What a row attends, in units.
template <bool WINDOW>
struct Row {
    int units;
    int len;                  // selected pages: tokens of the row
    int lo, hi, a, n_a;       // window: tokens [lo, hi) and the first a, of which n_a units
    const int32_t *table;

    // First token of unit u in its page's numbering is `t_in`; tokens v0 .. v1-1 of the unit are visible.
    // Returns the page, -1 where there is nothing to read.
    __device__ __forceinline__ int unit(int u, int n_pages, int *t_in, int *v0, int *v1, int32_t *err) const {
        int page;
        if constexpr (WINDOW) {
            const int base = u < n_a ? u * kUnit : (lo / kUnit + (u - n_a)) * kUnit;
            *v0 = u < n_a ? 0 : lo - base;
            *v1 = (u < n_a ? a : hi) - base;
            page = table[base >> 7];
            *t_in = base & 127;
            if (page < 0 || page >= n_pages) {
                raise_flag(err, MSA_FLAG_BOUNDS);
                return -1;
            }
        } else {
            *v0 = 0;
            *v1 = len - u * kUnit;
            page = table[u >> 2];
            *t_in = (u & 3) * kUnit;
            if (page >= n_pages) raise_flag(err, MSA_FLAG_BOUNDS);
            if (page < 0 || page >= n_pages) return -1;
        }
        return page;
    }
};

template <int D>
struct Smem {
    alignas(16) float o[kWarps][8][D + 4];
    float m[kWarps][8], l[kWarps][8];
    int e[kWarps];
    alignas(16) float po[8][D];       // of the CTA, read by the cluster
    float pm[8], pl[8];
    int pe;
};

template <int D, int HPG, bool WINDOW>
__global__ void __launch_bounds__(kThreads, 3) k_attn_q8(const __grid_constant__ Args a) {
    constexpr int KW = D / 16;       // words of K a lane reads per token
    constexpr int VW = D / 32;       // words of V a lane reads per token
    constexpr int KS = D / 32;       // k32 steps of S
    constexpr int MT = D / 16;       // m16 tiles of O
    __shared__ Smem<D> sm;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 2, c = lane & 3;
    const int row = blockIdx.x / a.cluster, rank = blockIdx.x - row * a.cluster;
    const int b = row / a.G, g = row - b * a.G;
    pdl_wait();
    pdl_trigger();

    Row<WINDOW> rw;
    if constexpr (WINDOW) {
        const int req = a.q_req[b], p = a.q_pos[b];
        if (req == -1) return;       // a padding row: the whole cluster leaves
        const bool ok = req >= 0 && req < a.n_req && p >= 0 && (p >> 7) < a.max_blocks;
        if (!ok && tid == 0 && rank == 0) raise_flag(a.err, MSA_FLAG_BOUNDS);
        rw.lo = max(0, p - (a.window - 1));
        rw.hi = p + 1;
        rw.a = min(a.n_sink, rw.lo);
        rw.n_a = (rw.a + kUnit - 1) / kUnit;
        rw.units = ok ? rw.n_a + p / kUnit - rw.lo / kUnit + 1 : 0;
        rw.table = a.block_table + size_t(ok ? req : 0) * a.max_blocks;
    } else {
        rw.len = min(a.row_len[row], a.topk * 128);
        rw.units = max(0, (rw.len + kUnit - 1) / kUnit);
        rw.table = a.page_table + size_t(row) * a.topk;
    }

    uint32_t kw[4][KW], vw[8][VW];   // codes of the unit at hand (K: of the next one from the softmax on)
    uint32_t ksb, vsb;               // scale bytes of tokens 4r .. 4r+3
    auto load_k = [&](int page, int t_in) {
        const size_t line = (size_t(page) * a.G + g) * 128 + t_in;
        const uint8_t *kp = a.k + (line + 4 * r) * D + c * (D / 4);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int w = 0; w < KW; w += 4) {
                const uint4 x = ldg_stream_v4(kp + i * D + w * 4);
                kw[i][w] = x.x;
                kw[i][w + 1] = x.y;
                kw[i][w + 2] = x.z;
                kw[i][w + 3] = x.w;
            }
        ksb = __ldg(reinterpret_cast<const uint32_t *>(a.k_scale + line) + r);
    };
    auto load_v = [&](int page, int t_in) {
        const size_t line = (size_t(page) * a.G + g) * 128 + t_in;
        const uint8_t *vp = a.v + (line + 8 * c) * D + r * (D / 8);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (VW == 4) {
                const uint4 x = ldg_stream_v4(vp + i * D);
                vw[i][0] = x.x;
                vw[i][1] = x.y;
                vw[i][2] = x.z;
                vw[i][3] = x.w;
            } else {
                asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
                             : "=r"(vw[i][0]), "=r"(vw[i][1]) : "l"(vp + i * D));
            }
        }
        vsb = __ldg(reinterpret_cast<const uint32_t *>(a.v_scale + line) + r);
    };

    const int step = a.cluster * kWarps;
    int u = rank * kWarps + warp;
    int t_in = 0, v0 = 0, v1 = 0, page = -1;
    if (u < rw.units) {
        page = rw.unit(u, a.n_pages, &t_in, &v0, &v1, a.err);
        if (page >= 0) {
            load_k(page, t_in);
            load_v(page, t_in);
        }
    }

    // q of head r in pieces (a quarter of the components per lane), and the factor of heads 2c, 2c + 1
    uint32_t qh[KW], ql[KW], qr[KW];
    float hq0, hq1;
    {
        float x[D / 4];
        const int head = g * HPG + (r < HPG ? r : 0);
        const uint4 *qp = reinterpret_cast<const uint4 *>(a.q + (size_t(b) * a.G * HPG + head) * D + c * (D / 4));
        uint32_t amax = 0u;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const uint4 w = __ldg(qp + i);
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                x[i * 8 + 2 * h] = bf16_lo(ww[h]);
                x[i * 8 + 2 * h + 1] = bf16_hi(ww[h]);
            }
        }
#pragma unroll
        for (int i = 0; i < D / 4; ++i) amax = max(amax, __float_as_uint(x[i]) & 0x7fffffffu);
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const bool finite = amax < 0x7f800000u;
        const int e = finite ? q8_exponent(amax) : 0;
        const float inv = exp2i(-e);
#pragma unroll
        for (int i = 0; i < KW; ++i) {
            float y[4];
#pragma unroll
            for (int h = 0; h < 4; ++h) y[h] = x[4 * i + h] * inv;
            q8_pieces(y, qh[i], ql[i], qr[i]);
        }
        const float hq = finite ? a.sm_scale * kLog2e * exp2i(e) : __uint_as_float(0x7fffffffu);
        hq0 = __shfl_sync(0xffffffffu, hq, 8 * c);
        hq1 = __shfl_sync(0xffffffffu, hq, 8 * c + 4);
    }

    float o[MT][4];
#pragma unroll
    for (int t = 0; t < MT; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;   // heads 2c, 2c + 1; l over this lane's tokens
    int emax = 0;                    // largest scale byte of V so far (255 aside): E + 127

    for (; u < rw.units; u += step) {
        int page_n = -1, t_n = 0, v0_n = 0, v1_n = 0;
        if (u + step < rw.units) page_n = rw.unit(u + step, a.n_pages, &t_n, &v0_n, &v1_n, a.err);
        if (page < 0) {              // nothing to read: only the next unit's loads
            if (page_n >= 0) {
                load_k(page_n, t_n);
                load_v(page_n, t_n);
            }
        } else {
            float s[4][2];           // logits in log2 units: token 4r + i, head 2c + h
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
                float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f}, z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    const uint32_t a0 = kw[2 * mt][2 * ks], a1 = kw[2 * mt + 1][2 * ks];
                    const uint32_t a2 = kw[2 * mt][2 * ks + 1], a3 = kw[2 * mt + 1][2 * ks + 1];
                    mma_e4m3(x, a0, a1, a2, a3, qh[2 * ks], qh[2 * ks + 1]);
                    mma_e4m3(y, a0, a1, a2, a3, ql[2 * ks], ql[2 * ks + 1]);
                    mma_e4m3(z, a0, a1, a2, a3, qr[2 * ks], qr[2 * ks + 1]);
                }
#pragma unroll
                for (int h = 0; h < 4; ++h)
                    s[2 * mt + (h >> 1)][h & 1] = x[h] + (y[h] * kQ8LoScale + z[h] * kQ8ReScale);
            }
            const uint32_t kb = ksb, vb = vsb;
            if (page_n >= 0) load_k(page_n, t_n);
            const bool whole = v0 <= 0 && v1 >= kUnit;
            float mx0 = -INFINITY, mx1 = -INFINITY;
            int eb[4];               // scale bytes of V (-1: not visible)
            int etop = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float ks = q8_scale((kb >> (8 * i)) & 255u);
                eb[i] = int((vb >> (8 * i)) & 255u);
                s[i][0] = s[i][0] * ks * hq0;
                s[i][1] = s[i][1] * ks * hq1;
                if (!whole && (4 * r + i < v0 || 4 * r + i >= v1)) {
                    s[i][0] = s[i][1] = -INFINITY;
                    eb[i] = -1;
                }
                etop = max(etop, eb[i] == 255 ? 0 : eb[i]);
                mx0 = fmaxf(mx0, s[i][0]);
                mx1 = fmaxf(mx1, s[i][1]);
            }
            etop = __reduce_max_sync(0xffffffffu, etop);
            if (etop > emax) {       // uniform in the warp
                const float al = pow2_down(emax - etop);
                emax = etop;
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    o[t][0] *= al;
                    o[t][1] *= al;
                    o[t][2] *= al;
                    o[t][3] *= al;
                }
            }
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) {
                mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, x));
                mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, x));
            }
            if (__any_sync(0xffffffffu, mx0 > m0 || mx1 > m1)) {
                const float n0 = fmaxf(m0, mx0), n1 = fmaxf(m1, mx1);
                const float al0 = n0 == -INFINITY ? 1.f : fast_exp2(m0 - n0);
                const float al1 = n1 == -INFINITY ? 1.f : fast_exp2(m1 - n1);
                m0 = n0;
                m1 = n1;
                l0 *= al0;
                l1 *= al1;
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    o[t][0] *= al0;
                    o[t][1] *= al1;
                    o[t][2] *= al0;
                    o[t][3] *= al1;
                }
            }
            const float r0 = m0 == -INFINITY ? 0.f : m0, r1 = m1 == -INFINITY ? 0.f : m1;
            uint32_t pt[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float p0 = fast_exp2(s[i][0] - r0), p1 = fast_exp2(s[i][1] - r1);
                l0 += p0;
                l1 += p1;
                // 2^(e - E + 100): 0 for tokens that are not visible, NaN for a NaN row
                const int x = max(eb[i] - emax + 227, 0) << 23;
                const float f = eb[i] < 0 ? 0.f : __uint_as_float(eb[i] == 255 ? 0x7fffffffu : uint32_t(x));
                pt[i] = transpose8(pack_bf16x2(p0 * f, p1 * f));
            }
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    const uint32_t sel = t & 1 ? 0x7632u : 0x5410u;
                    const uint32_t x = __byte_perm(vw[2 * kk][t >> 1], vw[2 * kk + 4][t >> 1], sel);
                    const uint32_t y = __byte_perm(vw[2 * kk + 1][t >> 1], vw[2 * kk + 5][t >> 1], sel);
                    mma_bf16_16816(o[t], bf16_even(x), bf16_odd(x), bf16_even(y), bf16_odd(y), pt[2 * kk],
                                   pt[2 * kk + 1]);
                }
            if (page_n >= 0) load_v(page_n, t_n);
        }
        page = page_n;
        t_in = t_n;
        v0 = v0_n;
        v1 = v1_n;
    }

    // ---------------------------------------------------------------- join: warps, then CTAs
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, x);
        l1 += __shfl_xor_sync(0xffffffffu, l1, x);
    }
    if (r == 0) {
        sm.m[warp][2 * c] = m0;
        sm.m[warp][2 * c + 1] = m1;
        sm.l[warp][2 * c] = l0;
        sm.l[warp][2 * c + 1] = l1;
        if (lane == 0) sm.e[warp] = emax;
    }
#pragma unroll
    for (int t = 0; t < MT; t += 2) {
        const int d = r * (D / 8) + 2 * t;
        *reinterpret_cast<float4 *>(&sm.o[warp][2 * c][d]) = make_float4(o[t][0], o[t][2], o[t + 1][0], o[t + 1][2]);
        *reinterpret_cast<float4 *>(&sm.o[warp][2 * c + 1][d]) = make_float4(o[t][1], o[t][3], o[t + 1][1], o[t + 1][3]);
    }
    __syncthreads();
    constexpr int PAIRS = HPG * D / 2;
    const size_t head0 = size_t(b) * a.G * HPG + size_t(g) * HPG;
    int ecta = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) ecta = max(ecta, sm.e[i]);
    // a pair of output components from the sums over all partials
    auto finish = [&](int h, int d, float top, float l, float x, float y, int e) {
        const float inv = l == 0.f ? 0.f : 1.0f / l;
        *reinterpret_cast<uint32_t *>(a.out + (head0 + h) * D + d) = pack_bf16x2(unscaled(x * inv, e), unscaled(y * inv, e));
        if (d == 0) a.lse[head0 + h] = l == 0.f ? -INFINITY : (top + log2f(l)) * kLn2;
    };
    for (int i = tid; i < PAIRS; i += kThreads) {
        const int h = i / (D / 2), d = (i - h * (D / 2)) * 2;
        float top = -INFINITY;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) top = fmaxf(top, sm.m[k][h]);
        const float ref = top == -INFINITY ? 0.f : top;
        float l = 0.f, x = 0.f, y = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            const float w = fast_exp2(sm.m[k][h] - ref), wo = w * pow2_down(sm.e[k] - ecta);
            l += w * sm.l[k][h];
            x += wo * sm.o[k][h][d];
            y += wo * sm.o[k][h][d + 1];
        }
        if (a.cluster == 1) {
            finish(h, d, top, l, x, y, ecta);
        } else {
            *reinterpret_cast<float2 *>(&sm.po[h][d]) = make_float2(x, y);
            if (d == 0) {
                sm.pm[h] = top;
                sm.pl[h] = l;
            }
        }
    }
    if (a.cluster == 1) return;
    if (tid == 0) sm.pe = ecta;
    cluster_arrive();
    cluster_wait();
    const uint32_t pe = smem_u32(&sm.pe);
    int ec = 0;
    for (int k = 0; k < a.cluster; ++k) ec = max(ec, __float_as_int(ld_cluster(cluster_map(pe, k))));
    const int share = PAIRS / a.cluster;   // a power of two, at least 8
    for (int i = tid; i < share; i += kThreads) {
        const int j = rank * share + i;
        const int h = j / (D / 2), d = (j - h * (D / 2)) * 2;
        const uint32_t pm = smem_u32(&sm.pm[h]), pl = smem_u32(&sm.pl[h]), po = smem_u32(&sm.po[h][d]);
        float top = -INFINITY;
        for (int k = 0; k < a.cluster; ++k) top = fmaxf(top, ld_cluster(cluster_map(pm, k)));
        const float ref = top == -INFINITY ? 0.f : top;
        float l = 0.f, x = 0.f, y = 0.f;
        for (int k = 0; k < a.cluster; ++k) {
            const float w = fast_exp2(ld_cluster(cluster_map(pm, k)) - ref);
            const float wo = w * pow2_down(__float_as_int(ld_cluster(cluster_map(pe, k))) - ec);
            const float2 v = ld_cluster2(cluster_map(po, k));
            l += w * ld_cluster(cluster_map(pl, k));
            x += wo * v.x;
            y += wo * v.y;
        }
        finish(h, d, top, l, x, y, ec);
    }
    cluster_arrive();                // no CTA leaves while another reads its partials
    cluster_wait();
}

template <int D, int HPG, bool WINDOW>
cudaError_t launch_t(Args a, long long rows, int units, cudaStream_t st, bool pdl) {
    // Enough CTAs to have three on every SM, as long as every warp of the cluster has a unit.
    const long long want = 3LL * sm_count();
    int cs = 1;
    while (cs < 16 && rows * cs * 2 <= want && cs * 2 * kWarps <= units) cs *= 2;
    a.cluster = cs;
    if (rows * cs > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    auto k = k_attn_q8<D, HPG, WINDOW>;
    if (cs > 8) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(rows * cs));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(cs);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k, a);
}

template <bool WINDOW>
cudaError_t launch_any(const Args &a, const Shape &s, long long rows, int units, cudaStream_t st, bool pdl) {
#define MSA_AQ_CASE(DD, HH) \
    if (s.D == DD && s.hpg == HH) return launch_t<DD, HH, WINDOW>(a, rows, units, st, pdl);
    MSA_AQ_CASE(128, 8) MSA_AQ_CASE(128, 4) MSA_AQ_CASE(64, 8) MSA_AQ_CASE(64, 4)
#undef MSA_AQ_CASE
    return cudaErrorNotSupported;
}

Args common(const void *q, const CacheQ8 &c, int n_pages, const Shape &s, void *out, float *lse, int32_t *err) {
    Args a = {};
    a.q = static_cast<const uint16_t *>(q);
    a.k = static_cast<const uint8_t *>(c.k);
    a.k_scale = static_cast<const uint8_t *>(c.k_scale);
    a.v = static_cast<const uint8_t *>(c.v);
    a.v_scale = static_cast<const uint8_t *>(c.v_scale);
    a.G = s.G;
    a.topk = s.topk;
    a.n_pages = n_pages;
    a.max_blocks = s.max_blocks;
    a.sm_scale = s.sm_scale;
    a.out = static_cast<uint16_t *>(out);
    a.lse = lse;
    a.err = err;
    return a;
}

}  // namespace

cudaError_t launch_attn_decode_q8(const void *q, const CacheQ8 &c, const int32_t *page_table, const int32_t *row_len,
                                  int B, int n_pages, const Shape &s, void *out, float *lse, int32_t *err,
                                  cudaStream_t st, bool pdl) {
    Args a = common(q, c, n_pages, s, out, lse, err);
    a.page_table = page_table;
    a.row_len = row_len;
    return launch_any<false>(a, s, 1LL * B * s.G, s.topk * 4, st, pdl);
}

cudaError_t launch_window_decode_q8(const void *q, const CacheQ8 &c, const int32_t *block_table, const int32_t *q_req,
                                    const int32_t *q_pos, int n_rows, int n_req, int n_pages, int window, int n_sink,
                                    const Shape &s, void *out, float *lse, int32_t *err, cudaStream_t st) {
    Args a = common(q, c, n_pages, s, out, lse, err);
    a.block_table = block_table;
    a.q_req = q_req;
    a.q_pos = q_pos;
    a.n_req = n_req;
    a.window = window;
    a.n_sink = n_sink;
    const long long most = std::min<long long>(s.max_blocks * 4LL, window / kUnit + 2LL + n_sink / kUnit);
    return launch_any<true>(a, s, 1LL * n_rows * s.G, int(most), st, false);
}

}  // namespace msa
