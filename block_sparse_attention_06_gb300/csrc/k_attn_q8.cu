// Decode attention over 8-bit caches: the pages of a row's selected blocks, or a window and the first tokens.
//
// A row is one query token of one KV group; its Hq/G heads attend the row's visible tokens,
//   s_t = sm_scale * q . k_t,   out = sum_t softmax(s)_t v_t,   lse = log sum_t exp(s_t).
//
// What bounds it is the read of K and V (one byte per component, and two scale bytes per token), and with
// few rows the latency of a chain: table, K, softmax, join.  So:
//   - a unit is 32 tokens of one page, and each warp streams its units through a buffer of its own in shared memory by
//     asynchronous copies, with its own running sums: no barrier between warps until the row's end.  The next K is
//     copied as soon as this one is in the MMAs, the next V as soon as this one is, so one buffer for each is
//     enough and sixteen warps fit an SM (eight with two buffers each took 50 us where these take 47);
//   - a row's units are dealt to the warps of a cluster of CTAs (more CTAs where there are few rows).  At the end
//     every warp writes its partial into the shared memory of the CTAs that own a share of the row's output; one
//     cluster barrier, and each CTA joins its share, always in the same order: no workspace, no atomics.
//
// Both contractions run on f16 MMAs (m16n8k16, heads = N): a code is an f16 number.
//   S^T = K q^T (tokens = M): q is f16 times a power of two (msa_q8.cuh), so nothing is rounded; the token's scale and
//   the head's factor multiply the fp32 result.
//   O^T = V^T P^T (components = M): P carries the token's scale, P_t = 2^(x_t - rx + 12) with x_t = (s_t - rs) + e_t,
//   and is rounded to f16, 2^-12 of itself or 2^-37 of the largest, whichever is more; the weights 2^(s_t - rs) are
//   summed in fp32.  rs is raised where a weight would pass 2^60, rx where P would pass 2^15.9, which is rare: a unit
//   costs no shuffle for them.  (x counts from rs, so logits of any size lose nothing to the exponent.)  A row of zeros in
//   V, whose scale of 1 says nothing of its size, is kept out of rx: beside it values of 2^-40 came back as 0.
// What a row does not see cannot reach it: its P is 0, and its bytes of V are cleared (a code may be a NaN).
// (The 8-bit MMA of warps takes codes as they are, but is no faster: it unpacks its operands itself, every time, and
// needs P and q in pieces.)
//
// Measured (Hq = 64, G = 8, D = 128).  8 requests x 16 blocks (33 MB): 12.5 to 13.0 us against 5.0 at the copy rate; the
// chain is a launch, two table loads, four units per warp at some 2,000 cycles and the join.  32 requests, window of 4,096
// (257 MB): 48 us against 38; 256 clusters of one CTA on 152 SMs leave a third of the SMs one row where the others have
// two.  (1 % less without a look at rows of zeros.)  First kernel, with 8-bit MMAs: 17.5 and 94.
//
// Layout.  A unit's K and V are 32 rows of D bytes, swizzled by the copy (128- or 64-byte pattern).  Lane (r, c) =
// (lane / 4, lane % 4) reads a quarter of K's rows 8i + r, i = 0 .. 3, and an eighth of V's rows 8i + 2c and 8i + 2c + 1:
// with the swizzle both take distinct banks (D = 128).  The C fragment of S^T then has the tokens 8i + r; P packed over
// two heads and transposed by movmatrix is the B fragment of P V for tokens 8i + 2c and 8i + 2c + 1.
#include "msa_internal.h"
#include "msa_q8.cuh"

#include <algorithm>

namespace msa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kUnit = 32;            // tokens
constexpr float kShift = 12.f;       // P is at most 2^12 where its reference was set ...
constexpr float kRaiseP = 3.9f;      // ... and its reference is raised where it would pass 2^15.9 (f16 ends below 2^16)
constexpr float kRaiseL = 60.f;      // a weight may pass its reference by 2^60

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ uint32_t cluster_map(uint32_t smem, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem), "r"(rank));
    return r;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void st_cluster4(uint32_t addr, float x, float y, float z, float w) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(x), "f"(y), "f"(z), "f"(w) : "memory");
}

// 4-byte global -> shared copy.
__device__ __forceinline__ void cp_async_4(uint32_t smem_dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_dst), "l"(src) : "memory");
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

constexpr int kMaxCluster = 16;

template <int D, int HPG>
struct Smem {
    alignas(1024) uint8_t kv[kWarps][2][kUnit * D];   // a warp's unit: K, V
    alignas(16) uint8_t scale[kWarps][2][kUnit];
    // this CTA's share of the partials of all warps of the cluster (its HPG * D / cluster components), and their
    // references and sums
    alignas(16) float part[kWarps * HPG * D];
    float rx[kMaxCluster * kWarps][8], rs[kMaxCluster * kWarps][8], l[kMaxCluster * kWarps][8];
    float factor[8];
};

// Byte offset of 16-byte column `ch` of row t of a unit.
template <int D>
__device__ __forceinline__ uint32_t unit_off(int t, int ch) {
    return uint32_t(t * D + ((D == 128 ? ch ^ (t & 7) : ch ^ ((t >> 1) & 3)) << 4));
}

template <int D, int HPG, bool WINDOW>
__global__ void __launch_bounds__(kThreads, 2)
    k_attn_q8(const __grid_constant__ Args a) {
    using S = Smem<D, HPG>;
    constexpr int KW = D / 16;       // words of K a lane reads per token
    constexpr int VW = D / 32;       // words of V a lane reads per token
    constexpr int MT = D / 16;       // m16 tiles of O
    extern __shared__ uint8_t smem_raw[];
    S &sm = *reinterpret_cast<S *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
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

    cluster_arrive();                // waited for before this CTA writes into the others: they have started by then

    // This warp's units: first, first + step, ...  Lane l looks up the l-th of 32 at a time.
    const int step = a.cluster * kWarps, first = rank * kWarps + warp;
    const int n = first < rw.units ? (rw.units - first + step - 1) / step : 0;
    int u_page = -1, u_at = 0;       // the page, and t_in | v0 << 8 | v1 << 16 (v0, v1 in 0 .. 32)
    auto look_up = [&](int i0) {
        u_page = -1;
        if (i0 + lane < n) {
            int t_in, v0, v1;
            u_page = rw.unit(first + (i0 + lane) * step, a.n_pages, &t_in, &v0, &v1, a.err);
            u_at = t_in | max(v0, 0) << 8 | min(max(v1, 0), kUnit) << 16;
        }
    };
    constexpr int CPR = D / 16;                          // 16-byte columns of a row
    auto line_of = [&](int page, int at) { return (size_t(page) * a.G + g) * 128 + (at & 127); };
    auto copy = [&](uint32_t dst, const uint8_t *src) {
#pragma unroll
        for (int k = 0; k < CPR; ++k)
            cp_async_16(dst + unit_off<D>((lane + 32 * k) / CPR, lane % CPR), src + lane * 16 + k * 512);
    };
    const uint8_t *const ku = sm.kv[warp][0], *const vu = sm.kv[warp][1];
    // unit i, its page and place; K and both scales are one group of copies, V the next one
    auto begin = [&](int i, int *page, int *at) {
        *page = -1;
        if (i < n) {
            if ((i & 31) == 0) look_up(i);
            *page = __shfl_sync(0xffffffffu, u_page, i & 31);
            *at = __shfl_sync(0xffffffffu, u_at, i & 31);
            if (*page >= 0) {
                const size_t line = line_of(*page, *at);
                copy(smem_u32(ku), a.k + line * D);
                if (lane < 16)
                    cp_async_4(smem_u32(sm.scale[warp][lane >> 3]) + (lane & 7) * 4,
                               (lane < 8 ? a.k_scale : a.v_scale) + line + (lane & 7) * 4);
            }
        }
        cp_async_commit();
    };
    auto begin_v = [&](int page, int at) {
        if (page >= 0) copy(smem_u32(vu), a.v + line_of(page, at) * D);
        cp_async_commit();
    };
    int page, at = 0;                // of the unit at hand
    begin(0, &page, &at);
    begin_v(page, at);

    // q of head r (a quarter of the components per lane), and the factor of heads 2c, 2c + 1
    uint32_t q[KW][2];
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
        const int e = finite ? f16_exponent(amax) : 0;
        const float inv = exp2i(-e);
#pragma unroll
        for (int i = 0; i < KW; ++i) {
            q[i][0] = pack_f16x2(x[4 * i] * inv, x[4 * i + 1] * inv);
            q[i][1] = pack_f16x2(x[4 * i + 2] * inv, x[4 * i + 3] * inv);
        }
        const float hq = finite ? a.sm_scale * kLog2e * exp2i(e) : __uint_as_float(0x7fffffffu);
        hq0 = __shfl_sync(0xffffffffu, hq, 8 * c);
        hq1 = __shfl_sync(0xffffffffu, hq, 8 * c + 4);
    }

    float o[MT][4];
#pragma unroll
    for (int t = 0; t < MT; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
    // heads 2c, 2c + 1: references of P and of the weights, the weights' sum over this lane's tokens
    float rx[2] = {-INFINITY, -INFINITY}, rs[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    for (int i = 0; i < n; ++i) {
        cp_async_wait<1>();
        __syncwarp();                // every lane's part of K and the scales is there
        const bool have = page >= 0;
        const int v0 = at >> 8 & 255, v1 = at >> 16;     // visible tokens
        float s[4][2], x[4][2];      // logits in log2 units, and x (see above): token 8k + r, head 2c + h
        float ve;                    // the exponent of V's scale, -inf where the token is not visible, NaN for a NaN row
        if (have) {
            // scales: of token `lane` here, of tokens 8k + r by shuffles
            const uint32_t vb = sm.scale[warp][1][lane];
            const bool seen = lane >= v0 && lane < v1;
            const float kf = q8_scale(sm.scale[warp][0][lane]);
            ve = !seen ? -INFINITY : vb == 255u ? __uint_as_float(0x7fffffffu) : float(int(vb) - 127);
            const float base[2] = {rs[0] == -INFINITY ? 0.f : rs[0], rs[1] == -INFINITY ? 0.f : rs[1]};
            float y[2][2][4];        // four chains of MMAs: their latency counts
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int k = 0; k < 4; ++k) y[mt][0][k] = y[mt][1][k] = 0.f;
#pragma unroll
            for (int j = 0; j < KW; j += 4) {
                uint32_t kw[2][2][4];
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(
                            ku + unit_off<D>(16 * mt + 8 * k + r, c * (KW / 4) + j / 4));
                        kw[mt][k][0] = x.x;
                        kw[mt][k][1] = x.y;
                        kw[mt][k][2] = x.z;
                        kw[mt][k][3] = x.w;
                    }
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
                        mma_f16(y[mt][k & 1], f16_of_low(kw[mt][0][k]), f16_of_low(kw[mt][1][k]),
                                f16_of_high(kw[mt][0][k]), f16_of_high(kw[mt][1][k]), q[j + k][0], q[j + k][1]);
            }
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float f = __shfl_sync(0xffffffffu, kf, 16 * mt + 8 * k + r);
                    const float e = __shfl_sync(0xffffffffu, ve, 16 * mt + 8 * k + r);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int i = 2 * k + h;
                        float v = (y[mt][0][i] + y[mt][1][i]) * f * (h ? hq1 : hq0);
                        if (e == -INFINITY) v = -INFINITY;           // not visible, whatever K holds
                        s[2 * mt + k][h] = v;
                        x[2 * mt + k][h] = (v - base[h]) + e;
                    }
                }
        }
        __syncwarp();                // K and the scales have been read
        int next = -1, next_at = 0;
        begin(i + 1, &next, &next_at);
        if (have) {
            bool raise = false;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float mx = fmaxf(fmaxf(x[0][h], x[1][h]), fmaxf(x[2][h], x[3][h]));
                const float ms = fmaxf(fmaxf(s[0][h], s[1][h]), fmaxf(s[2][h], s[3][h]));
                raise |= mx > rx[h] + kRaiseP || ms > rs[h] + kRaiseL;
            }
            if (__any_sync(0xffffffffu, raise)) {
                // A row of zeros in V (its scale is 1) adds nothing and must not set P's reference: values far below 1 beside
                // it would be lost.  Where a token's scale is 1, V's rows are looked at, token `lane`'s by each lane.
                if (__any_sync(0xffffffffu, ve == 0.f)) {
                    cp_async_wait<1>();
                    __syncwarp();
                    uint32_t any = 0u;
#pragma unroll
                    for (int k = 0; k < CPR; ++k) {
                        const uint4 y = *reinterpret_cast<const uint4 *>(vu + unit_off<D>(lane, k));
                        any |= y.x | y.y | y.z | y.w;
                    }
                    if (ve == 0.f && (any & 0x7f7f7f7fu) == 0u) ve = -INFINITY;
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float ms = fmaxf(fmaxf(s[0][h], s[1][h]), fmaxf(s[2][h], s[3][h]));
#pragma unroll
                    for (int k = 4; k < 32; k <<= 1) ms = fmaxf(ms, __shfl_xor_sync(0xffffffffu, ms, k));
                    ms = fmaxf(ms, rs[h]);
                    const float down = rs[h] == -INFINITY ? 0.f : ms - rs[h];   // by which what counts from rs falls
                    rs[h] = ms;
                    l[h] *= fast_exp2(-down);
                    float mx = -INFINITY;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float e = __shfl_sync(0xffffffffu, ve, 8 * k + r);
                        x[k][h] = (s[k][h] - (ms == -INFINITY ? 0.f : ms)) + e;
                        mx = fmaxf(mx, x[k][h]);
                    }
#pragma unroll
                    for (int k = 4; k < 32; k <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
                    const float old = rx[h] - down;
                    mx = fmaxf(mx, old);
                    const float ax = mx == -INFINITY ? 1.f : fast_exp2(old - mx);
                    rx[h] = mx;
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        o[t][h] *= ax;
                        o[t][2 + h] *= ax;
                    }
                }
            }
            uint32_t pt[4];          // P of tokens 8k + 2c, 8k + 2c + 1 and head r
            {
                const float bx0 = rx[0] == -INFINITY ? 0.f : rx[0] - kShift, bx1 = rx[1] == -INFINITY ? 0.f : rx[1] - kShift;
                const float bs0 = rs[0] == -INFINITY ? 0.f : rs[0], bs1 = rs[1] == -INFINITY ? 0.f : rs[1];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    l[0] += fast_exp2(s[k][0] - bs0);
                    l[1] += fast_exp2(s[k][1] - bs1);
                    pt[k] = transpose8(pack_f16x2(fast_exp2(x[k][0] - bx0), fast_exp2(x[k][1] - bx1)));
                }
            }
            cp_async_wait<1>();      // all but the next unit's K
            __syncwarp();
            uint32_t vw[8][VW];      // tokens 8 (k / 2) + 2c + k % 2
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int t = 8 * (k >> 1) + 2 * c + (k & 1);
                if constexpr (VW == 4) {
                    const uint4 y = *reinterpret_cast<const uint4 *>(vu + unit_off<D>(t, r));
                    vw[k][0] = y.x;
                    vw[k][1] = y.y;
                    vw[k][2] = y.z;
                    vw[k][3] = y.w;
                } else {
                    const uint2 y = *reinterpret_cast<const uint2 *>(vu + unit_off<D>(t, r >> 1) + (r & 1) * 8);
                    vw[k][0] = y.x;
                    vw[k][1] = y.y;
                }
            }
            if (v0 > 0 || v1 < kUnit) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int t = 8 * (k >> 1) + 2 * c + (k & 1);
                    if (t < v0 || t >= v1) {
#pragma unroll
                        for (int j = 0; j < VW; ++j) vw[k][j] = 0u;
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < VW; ++j) {
                uint32_t av[4][4];   // components 4j .. 4j + 3 of the four pairs of tokens
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t t0 = __byte_perm(vw[2 * k][j], vw[2 * k + 1][j], 0x5140);
                    const uint32_t t1 = __byte_perm(vw[2 * k][j], vw[2 * k + 1][j], 0x7362);
                    av[k][0] = f16_of_low(t0);
                    av[k][1] = f16_of_high(t0);
                    av[k][2] = f16_of_low(t1);
                    av[k][3] = f16_of_high(t1);
                }
#pragma unroll
                for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        mma_f16(o[2 * j + k], av[2 * kk][2 * k], av[2 * kk][2 * k + 1], av[2 * kk + 1][2 * k],
                                av[2 * kk + 1][2 * k + 1], pt[2 * kk], pt[2 * kk + 1]);
            }
        }
        __syncwarp();                // V has been read
        begin_v(next, next_at);
        page = next;
        at = next_at;
    }
    cp_async_wait<0>();

    // ---------------------------------------------------------------- join
#pragma unroll
    for (int k = 4; k < 32; k <<= 1) {
        l[0] += __shfl_xor_sync(0xffffffffu, l[0], k);
        l[1] += __shfl_xor_sync(0xffffffffu, l[1], k);
    }
    cluster_wait();
    // The row's HPG * D components are shared out in equal runs; a lane's D / 8 of a head fall to one CTA.
    const int share = HPG * D / a.cluster, wid = rank * kWarps + warp;
    const uint32_t part = smem_u32(sm.part) + uint32_t(wid * share) * 4u;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int e = (2 * c + h) * D + r * (D / 8);
        if (2 * c + h < HPG) {
            const uint32_t dst = cluster_map(part + uint32_t(e % share) * 4u, e / share);
#pragma unroll
            for (int t = 0; t < MT; t += 2)
                st_cluster4(dst + t * 8, o[t][h], o[t][2 + h], o[t + 1][h], o[t + 1][2 + h]);
        }
    }
    for (int k = r; k < a.cluster; k += 8) {             // lanes of r take the CTAs in turn
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            st_cluster(cluster_map(smem_u32(&sm.rx[wid][2 * c + h]), k), rx[h]);
            st_cluster(cluster_map(smem_u32(&sm.rs[wid][2 * c + h]), k), rs[h]);
            st_cluster(cluster_map(smem_u32(&sm.l[wid][2 * c + h]), k), l[h]);
        }
    }
    cluster_arrive();
    cluster_wait();
    const size_t head0 = size_t(b) * a.G * HPG + size_t(g) * HPG;
    const int n_part = a.cluster * kWarps;
    auto weight = [](float ref, float top) { return top == -INFINITY ? 0.f : fast_exp2(ref - top); };
    // a head's largest references, and the partials' weights in place of theirs: a warp per head
    if (warp < HPG) {
        float ts = -INFINITY, tx = -INFINITY;            // the largest rs: what every partial is brought to
        for (int k = lane; k < n_part; k += 32) ts = fmaxf(ts, sm.rs[k][warp]);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) ts = fmaxf(ts, __shfl_xor_sync(0xffffffffu, ts, o));
        auto rx_of = [&](int k) {
            return sm.rs[k][warp] == -INFINITY ? -INFINITY : sm.rx[k][warp] + (sm.rs[k][warp] - ts);
        };
        for (int k = lane; k < n_part; k += 32) tx = fmaxf(tx, rx_of(k));
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) tx = fmaxf(tx, __shfl_xor_sync(0xffffffffu, tx, o));
        float sum = 0.f;
        for (int k = lane; k < n_part; k += 32) {
            sum += weight(sm.rs[k][warp], ts) * sm.l[k][warp];
            sm.rx[k][warp] = weight(rx_of(k), tx);
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) {
            sm.factor[warp] = sum == 0.f ? 0.f : weight(tx - kShift, 0.f) / sum;
            if (rank == warp * D / share) a.lse[head0 + warp] = sum == 0.f ? -INFINITY : (ts + log2f(sum)) * kLn2;
        }
    }
    __syncthreads();
    for (int i = tid * 2; i < share; i += kThreads * 2) {
        const int e = rank * share + i, h = e / D, d = e - h * D;
        float x = 0.f, y = 0.f;
        for (int k = 0; k < n_part; ++k) {
            const float wx = sm.rx[k][h];
            const float2 v = *reinterpret_cast<const float2 *>(&sm.part[k * share + i]);
            x += wx * v.x;
            y += wx * v.y;
        }
        const float f = sm.factor[h];
        *reinterpret_cast<uint32_t *>(a.out + (head0 + h) * D + d) = pack_bf16x2(x * f, y * f);
    }
}

template <int D, int HPG, bool WINDOW>
cudaError_t launch_t(Args a, long long rows, int units, cudaStream_t st, bool pdl) {
    // A CTA per SM, as long as every warp of the cluster has a unit; clusters of 8 and 16 for few rows alone, since they
    // wait for SMs of one GPC, and 16 where every warp has two units.  Clusters of 1, 2, 4, 8 and 16 CTAs, in us (*: what
    // this takes).  16 blocks, 64 rows: 16.8, *12.5, 14.5, 26.5, 68; 11 blocks, D = 64, 24 rows: 9.6, 7.5, *7.0, 8.4, 19.4;
    // window of 4,096, 256 rows: *47, 54, 62, 107, 278; 16 rows: 2, 4, 8, 16: 17.5, *12.8, 14.5, 26; 8 rows: 17.0, 12.3,
    // *10.7, 15.5; 2 rows: 17.0, 12.3, *10.7, 11.8; window of 1,024, 8 rows: 9.4, *8.6, 8.8, 14.6; dense, 60,000 tokens, 8
    // rows: 158, 84, *47, 46; 2 rows: 158, 83, 47, *30.  (Taken before rows of zeros were looked for, which adds 1 %.)
    // The host does not know the rows' lengths: the rule takes them for full, and short rows in a table for long ones,
    // or under a window past their length, get clusters whose warps have nothing to do (8 CTAs: 10.7 us, 2: 8.6).
    const long long sms = sm_count();
    int cs = 1;
    while (cs < kMaxCluster && rows * cs * 2 <= (cs < 4 ? sms : sms / 2) && cs * (cs < 8 ? 2 : 4) * kWarps <= units) cs *= 2;
    a.cluster = cs;
    if (rows * cs > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    auto k = k_attn_q8<D, HPG, WINDOW>;
    const size_t smem = sizeof(Smem<D, HPG>) + 1024;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_once(allowed, reinterpret_cast<const void *>(k), smem, true);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(rows * cs));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
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
