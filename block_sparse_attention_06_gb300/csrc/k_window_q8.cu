// Window attention of a chunk's rows over 8-bit caches, on the 5th-generation tensor cores.
//
// Row r (position p of its request) attends the tokens t <= p with t > p - window or t < n_sink.  A tile is
// 128/HPG consecutive rows times the HPG heads of one KV group = the 128 rows of an MMA's M; an item is two such
// tiles (A, B) per CTA of one group, whose rows need nearly the same pages, and its steps are those pages:
//   S = Q K^T  (128 x 128 x D),  P = 2^((S - ref) scale),  O += P V  (128 x D x 128),  l += row sums of P.
// ref is a row's reference, raised only where a logit passes it by 2^24 (P and the sums are bf16 and fp32, whose
// precision does not depend on size), so O is next to never rescaled; out = O / l, lse = ref scale + log l.
//
// K and V come as codes and scales; eight warps turn a page into bf16 tiles in shared memory, exactly (a code
// becomes code * 2^-120 by shifts and masks, one multiplication by a power of two gives the value), so the MMAs
// round nothing of the cache; P is rounded to bf16 (2^-9 of itself), as V is in a bf16 cache.  A row of V that is NaN is
// written as zeros and the rows that see it are made NaN at the end: what a row does not see cannot reach it, whatever
// its bits.
//
// With heads of 128 two CTAs (a cluster) share an item: each converts half of a page, K by tokens and V by columns,
// and the MMAs of M = 256 read both halves.  (8,192 rows, window of 4,096, Hq = 64, G = 8: 1.03 ms, against 1.20 with
// single CTAs, whose converters take twice the issue slots.  Heads of 64 use single CTAs: half of V's columns would be
// half as wide as the operand's swizzle.)
//
// What bounds it: the chain S, softmax, P V of a tile.  TMEM holds two S and two O (512 columns with heads of 128), so
// two tiles take turns.  S of a page comes in halves of 64 tokens: P takes half of S's columns, so the first half of the
// next S goes into the other half as soon as P is there, before P V, and its softmax runs under P V.  A step of
// both tiles takes about 4,000 cycles, of which the tensor cores work 2,048; issue slots are busy 0.60 of the time, memory
// next to never.  Measured: 8,192 rows at 60,000, window of 4,096, 4 first tokens: 0.98 ms, 0.59 of the measured bf16 rate
// counting the visible tokens.  What brought it there from 1.53 ms: arrivals without a release over the cluster (1.61
// -> 1.41), a softmax of one pass (1.41 -> 1.17; the maximum first, or a vote for every 32 columns, breaks the code into
// short pieces), MMAs from a warp that stays together (1.17 -> 1.04), S by halves (1.05 -> 1.00), no branch per converted
// token (1.00 -> 0.98).  One thread per row and eight warps need half the instructions of two threads per row and sixteen.
//
// One CTA per SM, 20 warps, persistent over items:
//   warp 0     planner: for each item the pages that any of its rows sees, in a ring of step descriptors;
//   warp 1     MMA issuer and TMEM owner: per tile, once P of step s-1 is there, the first half of S(s), P V of s-1, the
//              second half of S(s) (a pair's first CTA for both);
//   warp 2     Q loader (TMA, one box per tile and 64 columns);   warp 3  idle;
//   warps 4-7, 8-11   softmax of tiles A and B, one row per thread; each also writes its tile's results;
//   warps 12-19  converters: the next page's codes wait in registers while this one's are written.
// TMEM: S_A | S_B | O_A | O_B (128 + 128 + D + D columns); P is written over S.
// Every wait is bounded; a timeout raises MSA_FLAG_TIMEOUT and every role drains.
#include "msa_internal.h"
#include "msa_q8.cuh"

#include <algorithm>
#include <type_traits>

namespace msa {
namespace {

constexpr int kThreads = 640;
constexpr int kRing = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// log2 units by which a logit may pass its row's reference: with V below 2^74 the sums stay in fp32
constexpr float kRaise = 24.f;

constexpr int kFirst = 1, kLast = 2, kEnd = 4, kNan = 8, kWhole = 16;   // kWhole: every row sees every token

struct alignas(16) Step {
    int32_t flags;
    int32_t page;          // physical page
    int32_t base;          // position of its first token
    int32_t req;
    uint32_t nan_v[4];     // tokens whose V row is NaN (kNan)
    int32_t row0, g;       // the item: its first row, its group
};

template <int D, bool PAIR>
struct Smem {
    static constexpr int TILE = 128 * D * 2 / (PAIR ? 2 : 1);   // a CTA's part of a page's K or V
    alignas(1024) uint8_t q[2][128 * D * 2];
    alignas(1024) uint8_t k[2][TILE];
    alignas(1024) uint8_t v[2][TILE];
    Step step[kRing];
    uint64_t desc_full[kRing], desc_empty[kRing];
    uint64_t q_tma[2], q_full[2], q_empty[2];
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
    uint64_t s_full[2][2], p_full[2], o_full[2];   // per tile; S by halves of a page
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    int empty;             // set where some head of a row has no weights
};

struct Args {
    const uint16_t *q;
    const uint8_t *k, *k_scale, *v, *v_scale;
    const int32_t *block_table, *q_req, *q_pos;
    int n_rows, n_req, n_pages, max_blocks, Hq, G, window, n_sink, n_items;
    float sm_scale;
    uint16_t *out;
    float *lse;
    int32_t *err;
};

// A head of a row (both in the whole call's numbering) for which no weight was counted, though the row sees a token, is
// NaN where its q is not finite: such logits are NaN or infinite, and their sum is NaN unless they all are -inf.
template <int D>
__device__ __forceinline__ void poison_empty(const Args &a, int row, int h) {
    if (row >= a.n_rows) return;
    const int req = a.q_req[row], pos = a.q_pos[row];
    const size_t head = size_t(row) * a.Hq + h;
    if (req < 0 || req >= a.n_req || pos < 0 || (pos >> 7) >= a.max_blocks || a.lse[head] != -INFINITY) return;
    bool finite = true, saw = false;
    for (int i = 0; i < D; ++i) finite &= (a.q[head * D + i] & 0x7f80u) != 0x7f80u;
    for (int j = a.n_sink > 0 ? 0 : max(0, pos - (a.window - 1)) >> 7; !finite && !saw && j <= pos >> 7; ++j) {
        const int page = a.block_table[size_t(req) * a.max_blocks + j];
        saw = (j * 128 + 127 > pos - a.window || j * 128 < a.n_sink) && page >= 0 && page < a.n_pages;
    }
    if (!saw) return;
    for (int i = 0; i < D; ++i) a.out[head * D + i] = 0x7fffu;
    a.lse[head] = __uint_as_float(0x7fffffffu);
}

// Two fp32 lanes per instruction; b2 and c2 hold one value in both halves.
__device__ __forceinline__ uint64_t dup2(float x) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(x));
    return r;
}
// d = (a + b) c
__device__ __forceinline__ void add_mul2(float &d0, float &d1, float a0, float a1, uint64_t b2, uint64_t c2) {
    asm("{\n\t.reg .b64 x, d;\n\tmov.b64 x, {%2, %3};\n\tadd.rn.f32x2 d, x, %4;\n\tmul.rn.f32x2 d, d, %5;\n\t"
        "mov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "l"(b2), "l"(c2));
}
__device__ __forceinline__ void fadd2_acc(uint64_t &acc2, float a0, float a1) {
    asm("{\n\t.reg .b64 x;\n\tmov.b64 x, {%1, %2};\n\tadd.rn.f32x2 %0, %0, x;\n\t}" : "+l"(acc2) : "f"(a0), "f"(a1));
}
__device__ __forceinline__ float sum2(uint64_t acc2) {
    float a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(acc2));
    return a + b;
}

// The lowest n bits set, n clamped to [0, 32].
__device__ __forceinline__ uint32_t ones_below(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }

// D/16 MMAs of S = Q K^T, both operands K-major with the 128-byte swizzle: a k-step of 16 columns is 32 bytes
// further in a sub-tile of 64 columns; with heads of 128, Q's two sub-tiles are 16 KB apart and those of a CTA's half of K
// 8 KB.  One asm block, so that the issuing thread spends as few issue slots as it can.
template <int D, bool PAIR>
__device__ __forceinline__ void mma_s(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t el) {
    static_assert(PAIR == (D == 128), "heads of 128 take pairs, heads of 64 single CTAs");
    if constexpr (PAIR) {
        asm volatile(
            "{\n\t.reg .pred e, f, t;\n\t.reg .b64 a1, a2, a3, a4, a5, a6, a7, b1, b2, b3, b4, b5, b6, b7;\n\t"
            "setp.ne.b32 e, %4, 0;\n\tsetp.ne.b32 f, %3, %3;\n\tsetp.eq.b32 t, %3, %3;\n\t"
            "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\tadd.s64 a4, %1, 1024;\n\t"
            "add.s64 a5, %1, 1026;\n\tadd.s64 a6, %1, 1028;\n\tadd.s64 a7, %1, 1030;\n\t"
            "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\tadd.s64 b4, %2, 512;\n\t"
            "add.s64 b5, %2, 514;\n\tadd.s64 b6, %2, 516;\n\tadd.s64 b7, %2, 518;\n\t"
            "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, f;\n\t"
            "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a1, b1, %3, t;\n\t"
            "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a2, b2, %3, t;\n\t"
            "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a3, b3, %3, t;\n\t"
            "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a4, b4, %3, t;\n\t"
            "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a5, b5, %3, t;\n\t"
            "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a6, b6, %3, t;\n\t"
            "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a7, b7, %3, t;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(el)
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred e, f, t;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
            "setp.ne.b32 e, %4, 0;\n\tsetp.ne.b32 f, %3, %3;\n\tsetp.eq.b32 t, %3, %3;\n\t"
            "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
            "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, f;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(el)
            : "memory");
    }
}

// Eight MMAs of O (+)= P V: P in TMEM (bf16 pairs, 8 columns per 16 tokens), V MN-major, 16 tokens 2 KB apart.
template <bool PAIR>
__device__ __forceinline__ void mma_pv(uint32_t d, uint32_t p, uint64_t v, uint32_t idesc, uint32_t accumulate,
                                       uint32_t el) {
    if constexpr (PAIR) {
        asm volatile(
            "{\n\t.reg .pred e, f, t;\n\t.reg .b64 b1, b2, b3, b4, b5, b6, b7;\n\t.reg .b32 a1, a2, a3, a4, a5, a6, a7;\n\t"
            "setp.ne.b32 e, %5, 0;\n\tsetp.ne.b32 f, %4, 0;\n\tsetp.eq.b32 t, %4, %4;\n\t"
            "add.s32 a1, %1, 8;\n\tadd.s32 a2, %1, 16;\n\tadd.s32 a3, %1, 24;\n\tadd.s32 a4, %1, 32;\n\t"
            "add.s32 a5, %1, 40;\n\tadd.s32 a6, %1, 48;\n\tadd.s32 a7, %1, 56;\n\t"
            "add.s64 b1, %2, 128;\n\tadd.s64 b2, %2, 256;\n\tadd.s64 b3, %2, 384;\n\tadd.s64 b4, %2, 512;\n\t"
            "add.s64 b5, %2, 640;\n\tadd.s64 b6, %2, 768;\n\tadd.s64 b7, %2, 896;\n\t"
            "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, f;\n\t"
            "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [a1], b1, %3, t;\n\t"
            "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [a2], b2, %3, t;\n\t"
            "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [a3], b3, %3, t;\n\t"
            "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [a4], b4, %3, t;\n\t"
            "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [a5], b5, %3, t;\n\t"
            "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [a6], b6, %3, t;\n\t"
            "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [a7], b7, %3, t;\n\t}" ::"r"(d),
            "r"(p), "l"(v), "r"(idesc), "r"(accumulate), "r"(el)
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred e, f, t;\n\t.reg .b64 b1, b2, b3, b4, b5, b6, b7;\n\t.reg .b32 a1, a2, a3, a4, a5, a6, a7;\n\t"
            "setp.ne.b32 e, %5, 0;\n\tsetp.ne.b32 f, %4, 0;\n\tsetp.eq.b32 t, %4, %4;\n\t"
            "add.s32 a1, %1, 8;\n\tadd.s32 a2, %1, 16;\n\tadd.s32 a3, %1, 24;\n\tadd.s32 a4, %1, 32;\n\t"
            "add.s32 a5, %1, 40;\n\tadd.s32 a6, %1, 48;\n\tadd.s32 a7, %1, 56;\n\t"
            "add.s64 b1, %2, 128;\n\tadd.s64 b2, %2, 256;\n\tadd.s64 b3, %2, 384;\n\tadd.s64 b4, %2, 512;\n\t"
            "add.s64 b5, %2, 640;\n\tadd.s64 b6, %2, 768;\n\tadd.s64 b7, %2, 896;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, f;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a4], b4, %3, t;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a5], b5, %3, t;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a6], b6, %3, t;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a7], b7, %3, t;\n\t}" ::"r"(d),
            "r"(p), "l"(v), "r"(idesc), "r"(accumulate), "r"(el)
            : "memory");
    }
}

// A pair of CTAs: MMAs of M = 256 over both SMs, issued by the first CTA.  Barriers that the issuer waits on are the
// first CTA's; its commits arrive in both CTAs.  What these arrivals hand over is read by the tensor cores alone: the
// fences before them (of tcgen05, of the async proxy) order it, and a release over the cluster, which would hold
// the softmax warps up for 1500 cycles per step, is not needed.
template <bool PAIR>
__device__ __forceinline__ void commit(uint64_t *bar, uint32_t el) {
    if constexpr (PAIR)
        asm volatile("{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %2, 0;\n\t"
                     "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                     "\n\t}" ::"r"(smem_u32(bar)), "h"(uint16_t(3)), "r"(el) : "memory");
    else
        asm volatile("{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
                     "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
                         smem_u32(bar)), "r"(el) : "memory");
}

// 1 in one lane of the warp.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e;
}

template <bool PAIR>
__device__ __forceinline__ void arrive_first(uint64_t *bar) {
    if constexpr (PAIR)
        asm volatile("{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %0, 0;\n\t"
                     "mbarrier.arrive.shared::cluster.b64 _, [r];\n\t}" ::"r"(smem_u32(bar)) : "memory");
    else
        mbar_arrive(bar);
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Infinities as the largest number of their sign.
__device__ __forceinline__ uint32_t finite_bf16x2(uint32_t a) {
    uint32_t r;
    asm("{\n\t.reg .b32 x;\n\tmin.bf16x2 x, %1, %2;\n\tmax.bf16x2 %0, x, %3;\n\t}"
        : "=r"(r) : "r"(a), "r"(0x7f7f7f7fu), "r"(0xff7fff7fu));
    return r;
}

// 16 codes as 16 bf16 numbers code * 2^-120 * f (f: a bf16 number in both halves).
__device__ __forceinline__ void convert16(const uint4 &w, uint32_t f, uint32_t (&o)[8]) {
    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // codes 0, 1 and 2, 3 side by side: bytes 0 and 2, then 1 and 3, of a word in the order 0, 2, 1, 3
        const uint32_t x = __byte_perm(ww[i], 0u, 0x3120);
        o[2 * i] = mul_bf16x2(((x << 4) & 0x07f007f0u) | ((x << 8) & 0x80008000u), f);
        o[2 * i + 1] = mul_bf16x2(((x >> 4) & 0x07f007f0u) | (x & 0x80008000u), f);
    }
}

// 32 lanes x 16 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
template <int D, int HPG, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    k_window_q8(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap qmap) {
    constexpr int EPT = 128 / HPG;       // rows per tile
    constexpr int NSUB = D / 64;         // 64-column sub-tiles
    constexpr int CT = PAIR ? 2 : 1;     // CTAs that work on an item
    constexpr uint32_t kIdescS = make_idesc_bf16(CT * 128, 64, 0, 0);
    constexpr uint32_t kIdescO = make_idesc_bf16(CT * 128, D, 0, 1);
    using S = Smem<D, PAIR>;
    extern __shared__ uint8_t smem_raw[];
    S &sm = *reinterpret_cast<S *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int rank = PAIR ? blockIdx.x & 1 : 0;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int32_t *const err = a.err;

    if (tid == 0) {
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&sm.desc_full[i], 32);
            mbar_init(&sm.desc_empty[i], 18);   // issuer, Q loader, 8 softmax warps, 8 converter warps
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.q_tma[i], 1);
            mbar_init(&sm.q_full[i], CT);
            mbar_init(&sm.q_empty[i], 1);
            mbar_init(&sm.k_full[i], 8 * CT);
            mbar_init(&sm.k_empty[i], 1);
            mbar_init(&sm.v_full[i], 8 * CT);
            mbar_init(&sm.v_empty[i], 1);
            mbar_init(&sm.s_full[i][0], 1);
            mbar_init(&sm.s_full[i][1], 1);
            mbar_init(&sm.p_full[i], 4 * CT);
            mbar_init(&sm.o_full[i], 1);
        }
        mbar_init(&sm.drain, 1);
        sm.abort = sm.empty = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        if constexpr (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem_base)),
                         "r"(512) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            tmem_alloc(&sm.tmem_base, 512);
            tmem_relinquish();
        }
    }
    if (warp == 2 && lane == 0) tma_prefetch_desc(&qmap);
    tc_fence_before();
    if constexpr (PAIR) cluster_sync();  // the other CTA's barriers are there too
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    const volatile Step *const steps = sm.step;

    if (warp == 0) {
        // ------------------------------------------------------------ planner
        int s = 0;                       // steps published
        bool ok = true, pending = false;
        Step st = {};                    // the step in hand: published with the next one, when its scales are here
        uint32_t vs = 0u;                // its V scales, four tokens a lane
        auto publish = [&](int more) {
            const int slot = s % kRing;
            if (s >= kRing) {
                bool w = true;
                if (lane == 0) w = mbar_wait(&sm.desc_empty[slot], ((s / kRing) - 1) & 1, err, &sm.abort);
                if (!__shfl_sync(0xffffffffu, w, 0)) {
                    ok = false;
                    return;
                }
            }
            uint32_t nib = 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) nib |= ((vs >> (8 * i)) & 255u) == 255u ? 1u << i : 0u;
            const bool nan = __any_sync(0xffffffffu, nib != 0u);
            if (nan) {
                uint32_t m = nib << (4 * (lane & 7));
                m |= __shfl_xor_sync(0xffffffffu, m, 1);
                m |= __shfl_xor_sync(0xffffffffu, m, 2);
                m |= __shfl_xor_sync(0xffffffffu, m, 4);
                if ((lane & 7) == 0) sm.step[slot].nan_v[lane >> 3] = m;
            }
            if (lane == 0) {
                Step &d = sm.step[slot];
                d.flags = st.flags | more | (nan ? kNan : 0);
                d.page = st.page;
                d.base = st.base;
                d.req = st.req;
                d.row0 = st.row0;
                d.g = st.g;
            }
            mbar_arrive(&sm.desc_full[slot]);
            ++s;
        };
        for (int item = blockIdx.x / CT; ok && item < a.n_items; item += gridDim.x / CT) {
            const int set = item / a.G, g = item - set * a.G;
            const int row0 = set * 2 * CT * EPT, mine0 = row0 + rank * 2 * EPT;
            // the item's rows (both CTAs of a pair plan the same steps), 2 CT EPT / 32 a lane
            constexpr int RPL = 2 * CT * EPT / 32;
            int rq[RPL], rp[RPL];
#pragma unroll
            for (int i = 0; i < RPL; ++i) {
                const int r = row0 + i * 32 + lane;
                rq[i] = r < a.n_rows ? a.q_req[r] : -1;
                rp[i] = r < a.n_rows ? a.q_pos[r] : 0;
                if (rq[i] != -1 && (rq[i] < 0 || rq[i] >= a.n_req || rp[i] < 0 || (rp[i] >> 7) >= a.max_blocks)) {
                    if (g == 0) raise_flag(err, MSA_FLAG_BOUNDS);
                    rq[i] = -2;              // sees nothing: no page is whole beside it, and it gets 0 and -inf
                }
            }
            int rq0[RPL];
#pragma unroll
            for (int i = 0; i < RPL; ++i) rq0[i] = rq[i];
            int flags = kFirst;
            auto next_req = [&]() {      // the lowest request that is left, -1 for none
                int m = 0x7fffffff;
#pragma unroll
                for (int i = 0; i < RPL; ++i) m = min(m, rq[i] < 0 ? 0x7fffffff : rq[i]);
                m = __reduce_min_sync(0xffffffffu, m);
                return m == 0x7fffffff ? -1 : m;
            };
            for (int req = next_req(); ok && req >= 0;) {
                int pmin = 0x7fffffff, pmax = -1;
#pragma unroll
                for (int i = 0; i < RPL; ++i)
                    if (rq[i] == req) {
                        pmin = min(pmin, rp[i]);
                        pmax = max(pmax, rp[i]);
                    }
                pmin = __reduce_min_sync(0xffffffffu, pmin);
                pmax = __reduce_max_sync(0xffffffffu, pmax);
                bool alone = true;           // no row of another request
#pragma unroll
                for (int i = 0; i < RPL; ++i) alone &= rq0[i] == -1 || rq0[i] == req;
                alone = __all_sync(0xffffffffu, alone);
                const int32_t *table = a.block_table + size_t(req) * a.max_blocks;
                const int sink = min(a.n_sink, pmax + 1);
                const int n_sp = (sink + 127) >> 7;                       // blocks with tokens that stay visible
                const int lo = max(n_sp, max(0, pmin - (a.window - 1)) >> 7);
                const int n_w = max(0, (pmax >> 7) - lo + 1);
                for (int x0 = 0; ok && x0 < n_sp + n_w; x0 += 32) {       // 32 blocks at a time, one a lane
                    const int x = x0 + lane;
                    const int j = x < n_sp ? x : lo + (x - n_sp);
                    const bool in = x < n_sp + n_w;
                    int page = in ? table[j] : -1;
                    bool need = false;                                    // does any row of the request see a token of it?
#pragma unroll
                    for (int i = 0; i < RPL; ++i)
                        for (int l = 0; l < 32; ++l) {
                            const int q = __shfl_sync(0xffffffffu, rq[i], l), p = __shfl_sync(0xffffffffu, rp[i], l);
                            need |= q == req && j * 128 <= p &&
                                    (j * 128 + 127 > p - a.window || j * 128 < a.n_sink);
                        }
                    need = need && in;
                    if (need && (page < 0 || page >= a.n_pages)) {
                        raise_flag(err, MSA_FLAG_BOUNDS);
                        need = false;
                    }
                    uint32_t left = __ballot_sync(0xffffffffu, need);
                    while (ok && left) {
                        const int l = __ffs(left) - 1;
                        left &= left - 1u;
                        const int pg = __shfl_sync(0xffffffffu, page, l), jj = __shfl_sync(0xffffffffu, j, l);
                        const uint32_t vn = __ldg(
                            reinterpret_cast<const uint32_t *>(a.v_scale + (size_t(pg) * a.G + g) * 128) + lane);
                        if (pending) publish(0);
                        const bool whole = alone && jj * 128 + 127 <= pmin &&
                                           (jj * 128 > pmax - a.window || jj * 128 + 128 <= a.n_sink);
                        st.flags = flags | (whole ? kWhole : 0);
                        st.page = pg;
                        st.base = jj * 128;
                        st.req = req;
                        st.row0 = mine0;
                        st.g = g;
                        vs = vn;
                        flags = 0;
                        pending = true;
                    }
                }
#pragma unroll
                for (int i = 0; i < RPL; ++i)
                    if (rq[i] == req) rq[i] = -1;
                req = next_req();
            }
            if (ok && pending) {
                publish(kLast);
                pending = false;
            }
            if (ok && flags == kFirst) {   // no row of the item sees a page that exists: zeros
                for (int i = lane; i < 2 * EPT * HPG; i += 32) {
                    const int r = mine0 + i / HPG;
                    if (r >= a.n_rows || a.q_req[r] == -1) continue;
                    const size_t h = size_t(r) * a.Hq + g * HPG + i % HPG;
                    for (int d = 0; d < D; d += 8)
                        *reinterpret_cast<uint4 *>(a.out + h * D + d) = make_uint4(0u, 0u, 0u, 0u);
                    a.lse[h] = -INFINITY;
                }
            }
        }
        if (ok) {
            st.flags = kEnd;
            vs = 0u;
            publish(0);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        // The warp stays together, and one lane's MMAs are predicated: descriptors then are uniform registers.
        const uint32_t el = elect_one();
        const uint64_t qd0 = make_smem_desc(smem_u32(sm.q[0]), 16, 1024, 2);
        const uint64_t qd1 = make_smem_desc(smem_u32(sm.q[1]), 16, 1024, 2);
        const uint64_t kd0 = make_smem_desc(smem_u32(sm.k[0]), 16, 1024, 2);
        const uint64_t vd0 = make_smem_desc(smem_u32(sm.v[0]), 16384, 1024, 2);
        constexpr uint64_t kNext = Smem<D, PAIR>::TILE >> 4;      // from a descriptor to the other stage's
        auto wait = [&](uint64_t *bar, int parity) {
            return bool(__all_sync(0xffffffffu, mbar_wait(bar, uint32_t(parity), err, &sm.abort)));
        };
        constexpr uint64_t kHalf = (PAIR ? 4096 : 8192) >> 4;     // from K's first 64 tokens to the others
        // P V of tile x at step s; `first`: overwrite O
        auto issue_pv = [&](int x, int s, bool first) -> bool {
            if (x == 0 && !wait(&sm.v_full[s & 1], (s >> 1) & 1)) return false;
            tc_fence_after();
            mma_pv<PAIR>(tmem + 256u + uint32_t(x * D), tmem + uint32_t(x * 128 + (s & 1) * 64),
                         vd0 + uint64_t(s & 1) * kNext, kIdescO, first ? 0u : 1u, el);
            return true;
        };
        int items = 0;               // whose Q has been waited for
        bool before = false;         // the step before was its item's first
        for (int s = 0;; ++s) {
            const int slot = s % kRing;
            if (!wait(&sm.desc_full[slot], (s / kRing) & 1)) break;
            const int flags = steps[slot].flags;
            const bool first = __any_sync(0xffffffffu, flags & kFirst), last = __any_sync(0xffffffffu, flags & kLast);
            const bool end = __any_sync(0xffffffffu, flags & kEnd);
            if (lane == 0) mbar_arrive(&sm.desc_empty[slot]);
            if (end) break;
            if (rank != 0) continue;     // the first CTA issues for both
            if (!wait(&sm.k_full[s & 1], (s >> 1) & 1)) break;
            const uint64_t kd = kd0 + uint64_t(s & 1) * kNext;
            bool ok = true;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                // P of the step before is there, so all of its S has been read: the half that P is not in is free
                ok = first ? wait(&sm.q_full[x], items & 1) : wait(&sm.p_full[x], (s - 1) & 1);
                if (!ok) break;
                tc_fence_after();
                mma_s<D, PAIR>(tmem + uint32_t(x * 128 + (s & 1) * 64), x ? qd1 : qd0, kd, kIdescS, el);
                commit<PAIR>(&sm.s_full[x][0], el);
                if (!first) {
                    ok = issue_pv(x, s - 1, before);
                    if (!ok) break;
                    if (x == 1) commit<PAIR>(&sm.v_empty[(s - 1) & 1], el);
                }
                mma_s<D, PAIR>(tmem + uint32_t(x * 128 + 64 - (s & 1) * 64), x ? qd1 : qd0, kd + kHalf, kIdescS, el);
                commit<PAIR>(&sm.s_full[x][1], el);
                if (x == 1) commit<PAIR>(&sm.k_empty[s & 1], el);
                if (last) commit<PAIR>(&sm.q_empty[x], el);
            }
            if (!ok) break;
            items += first;
            before = first;
            if (last) {              // the item's results wait for it, and the next item's Q is still on its way
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    ok = wait(&sm.p_full[x], s & 1) && issue_pv(x, s, first);
                    if (!ok) break;
                    commit<PAIR>(&sm.o_full[x], el);
                    if (x == 1) commit<PAIR>(&sm.v_empty[s & 1], el);
                }
                if (!ok) break;
            }
        }
        if (rank == 0) {
            if constexpr (PAIR)
                asm volatile("{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
                             "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
                                 smem_u32(&sm.drain)), "r"(el) : "memory");
            else
                commit<false>(&sm.drain, el);
            mbar_wait(&sm.drain, 0, err, nullptr);
        }
    } else if (warp == 2) {
        // ------------------------------------------------------------ Q loader (lane 0)
        if (lane == 0) {
            int items = 0, loaded[2] = {0, 0};
            for (int s = 0;; ++s) {
                const int slot = s % kRing;
                if (!mbar_wait(&sm.desc_full[slot], (s / kRing) & 1, err, &sm.abort)) break;
                const int flags = steps[slot].flags, row0 = steps[slot].row0, g = steps[slot].g;
                mbar_arrive(&sm.desc_empty[slot]);
                if (flags & kEnd) break;
                if (!(flags & kFirst)) continue;
                bool ok = true;
                for (int x = 0; ok && x < 2; ++x) {
                    if (items > 0 && !mbar_wait(&sm.q_empty[x], (items - 1) & 1, err, &sm.abort)) {
                        ok = false;
                        break;
                    }
                    uint64_t *bar = PAIR ? &sm.q_tma[x] : &sm.q_full[x];
                    mbar_arrive_expect_tx(bar, 128 * D * 2);
#pragma unroll
                    for (int i = 0; i < NSUB; ++i)   // rows past the last read as zeros
                        tma_load_3d(sm.q[x] + i * 16384, &qmap, bar, i * 64, g * HPG, row0 + x * EPT);
                    loaded[x] = items + 1;
                }
                if (!ok) break;
                if constexpr (PAIR) {
                    for (int x = 0; ok && x < 2; ++x) {
                        ok = mbar_wait(&sm.q_tma[x], items & 1, err, &sm.abort);
                        if (ok) arrive_first<PAIR>(&sm.q_full[x]);
                    }
                    if (!ok) break;
                }
                ++items;
            }
            if (sm.abort)                // copies in flight land before the CTA exits
                for (int x = 0; x < 2; ++x)
                    if (loaded[x] > 0) mbar_wait(PAIR ? &sm.q_tma[x] : &sm.q_full[x], (loaded[x] - 1) & 1, err, nullptr);
        }
    } else if (warp >= 12) {
        // ------------------------------------------------------------ converters
        // A thread takes a few consecutive tokens, 16 codes of each (its lane's column).  The upper four lanes of a
        // quarter warp take them in the order 1, 0, 3, 2: the swizzle then puts the eight stores of a quarter warp into
        // eight different 16-byte columns.  A pair of CTAs shares a page: each converts half of K's tokens and half of
        // V's columns, which is what the MMAs of pairs read of it.
        const int w = warp - 12;
        const int swap = (lane >> 2) & 1;
        constexpr int KL = D / 16, KT = KL / 2 / CT;         // K: lanes per token, tokens per thread
        constexpr int VL = D / 16 / CT, VT = D / 32 / CT;    // V
        static_assert(KT == 2 && VT == 2, "the scales of a thread's tokens are one 16-bit load");
        using Lane = struct {
            int col, tok0, row;                              // 16 codes of the tile's tokens tok0 .., the page's row ..
            uint32_t at;                                     // their sub-tile of 64 columns
            int ch;                                          // their first 16-byte chunk in it
            size_t off;                                      // bytes from the page's first row
        };
        auto lane_of = [&](int lanes, int toks, bool split, int col_first, uint32_t sub_bytes) {
            Lane x;
            x.col = lane % lanes;
            x.tok0 = (w * (32 / lanes) + lane / lanes) * toks;
            x.at = uint32_t(x.col >> 2) * sub_bytes;
            x.ch = (x.col & 3) * 2;
            x.row = split ? (x.tok0 & 31) + rank * 32 + (x.tok0 >> 5) * 64 : x.tok0;   // half of either half page
            x.off = size_t(x.row) * D + col_first + x.col * 16;
            return x;
        };
        const Lane kl = lane_of(KL, KT, PAIR, 0, PAIR ? 8192u : 16384u);
        const Lane vl = lane_of(VL, VT, false, PAIR ? rank * 64 : 0, 16384u);
        // codes c[i] of token tok0 + (i ^ swap); returns the scale bytes in that order
        auto load = [&](const uint8_t *codes, const uint8_t *scales, size_t page_line, const Lane &x, auto &c) {
            constexpr int T = sizeof(c) / sizeof(uint4);
            const uint8_t *p = codes + page_line * D + x.off;
#pragma unroll
            for (int i = 0; i < T; ++i) c[i] = __ldg(reinterpret_cast<const uint4 *>(p + (i ^ swap) * D));
            const uint8_t *sp = scales + page_line + x.row;
            const uint32_t sc = __ldg(reinterpret_cast<const uint16_t *>(sp));
            return swap ? __byte_perm(sc, 0u, 0x4401) : sc;
        };
        auto store = [&](uint8_t *tile, const Lane &x, const auto &c, uint32_t sc, bool values) {
            constexpr int T = sizeof(c) / sizeof(uint4);
            const uint32_t base = smem_u32(tile) + x.at;
            auto put = [&](int t, const uint32_t (&o)[8]) {
                const uint32_t p0 = base + uint32_t(t * 128) + uint32_t((x.ch ^ (t & 7)) << 4);
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(p0), "r"(o[0]), "r"(o[1]), "r"(o[2]),
                             "r"(o[3]) : "memory");
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(p0 ^ 16u), "r"(o[4]), "r"(o[5]), "r"(o[6]),
                             "r"(o[7]) : "memory");
            };
            if (__all_sync(0xffffffffu, (sc & 0x8080u) == 0u)) {   // no scale above 1, no NaN row: 2^(120 + e)
#pragma unroll
                for (int i = 0; i < T; ++i) {
                    uint32_t o[8];
                    convert16(c[i], ((sc >> (8 * i) & 255u) + 120u) * 0x00800080u, o);
                    put(x.tok0 + (i ^ swap), o);
                }
            } else {                     // rolled: short, beside the code that always runs
#pragma unroll 1
                for (int i = 0; i < T; ++i) {
                    // 2^120 and then 2^e where e > 0; a NaN row: of K NaN, so the logits of the rows that see it are; of
                    // V zeros (see above)
                    const uint32_t b = (sc >> (8 * i)) & 255u;
                    const uint32_t f = b == 255u ? (values ? 0u : 0x7fff7fffu) : (min(b, 127u) + 120u) * 0x00800080u;
                    const uint32_t up = b == 255u ? 0x3f803f80u : max(b, 127u) * 0x00800080u;
                    uint4 w = c[0];
#pragma unroll
                    for (int k = 1; k < T; ++k)
                        if (i == k) w = c[k];
                    uint32_t o[8];
                    convert16(w, f, o);
#pragma unroll
                    for (int k = 0; k < 8; ++k) o[k] = mul_bf16x2(o[k], up);
                    if (values) {    // finite under any scale: P is 0 for a row that does not see it
#pragma unroll
                        for (int k = 0; k < 8; ++k) o[k] = finite_bf16x2(o[k]);
                    }
                    put(x.tok0 + (i ^ swap), o);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
        };
        // the next step's descriptor; false at the end
        int sd = 0, page = 0, g = 0;
        auto desc = [&]() -> bool {
            const int slot = sd % kRing;
            if (!__all_sync(0xffffffffu, mbar_wait(&sm.desc_full[slot], (sd / kRing) & 1, err, &sm.abort))) return false;
            const int flags = steps[slot].flags;
            page = steps[slot].page;
            g = steps[slot].g;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.desc_empty[slot]);
            ++sd;
            return !(flags & kEnd);
        };
        uint4 kc[KT], vc[VT];
        uint32_t ks = 0u, vs = 0u;
        auto load_k = [&]() { ks = load(a.k, a.k_scale, (size_t(page) * a.G + g) * 128, kl, kc); };
        auto load_v = [&]() { vs = load(a.v, a.v_scale, (size_t(page) * a.G + g) * 128, vl, vc); };
        bool more = desc();              // there is a step that is not written yet
        if (more) {
            load_k();
            load_v();
        }
        for (int s = 0; more; ++s) {
            const int b = s & 1;
            if (s >= 2 && !__all_sync(0xffffffffu, mbar_wait(&sm.k_empty[b], ((s >> 1) - 1) & 1, err, &sm.abort))) break;
            store(sm.k[b], kl, kc, ks, false);
            if (lane == 0) arrive_first<PAIR>(&sm.k_full[b]);
            more = desc();
            if (more) load_k();
            if (s >= 2 && !__all_sync(0xffffffffu, mbar_wait(&sm.v_empty[b], ((s >> 1) - 1) & 1, err, &sm.abort))) break;
            store(sm.v[b], vl, vc, vs, true);
            if (lane == 0) arrive_first<PAIR>(&sm.v_full[b]);
            if (more) load_v();
        }
    } else if (warp >= 4) {
        // ------------------------------------------------------------ softmax (warps 4-7: A, 8-11: B)
        const int x = (warp - 4) >> 2;
        const int quad = warp & 3;                          // TMEM lanes this warp may access
        const int trow = quad * 32 + lane;
        const int e = trow / HPG, h = trow - e * HPG;
        const uint32_t t_s = tmem + (uint32_t(quad * 32) << 16) + uint32_t(x * 128);
        const uint32_t t_o = tmem + (uint32_t(quad * 32) << 16) + 256u + uint32_t(x * D);
        const float scale = a.sm_scale * kLog2e;
        const uint64_t scale2 = dup2(scale);
        int row = -1, req = -1, pos = -1, g = 0;            // of this thread, in the item at hand
        int items = 0;                   // done
        float ref = -INFINITY, l = 0.f;
        bool poison = false;
        for (int s = 0;; ++s) {
            const int slot = s % kRing;
            bool ok = __all_sync(0xffffffffu, mbar_wait(&sm.desc_full[slot], (s / kRing) & 1, err, &sm.abort));
            const int4 d = *reinterpret_cast<const int4 *>(&sm.step[slot]);
            const int flags = d.x;
            uint32_t nan_v[4] = {0u, 0u, 0u, 0u};
            if (flags & kNan) {
#pragma unroll
                for (int i = 0; i < 4; ++i) nan_v[i] = steps[slot].nan_v[i];
            }
            if (flags & kFirst) {
                row = steps[slot].row0 + x * EPT + e;
                g = steps[slot].g;
                req = row < a.n_rows ? a.q_req[row] : -1;
                pos = row < a.n_rows ? a.q_pos[row] : 0;
                if (pos < 0 || (pos >> 7) >= a.max_blocks) {   // outside the table: sees nothing (nor does a bad request)
                    req = req == -1 ? -1 : -2;
                    pos = 0;
                }
                ref = -INFINITY;
                l = 0.f;
                poison = false;
            }
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(&sm.desc_empty[slot]);
            if (!ok || (flags & kEnd)) break;
            // Tokens c of the page with c <= hi and (c >= lo or c < sk) are visible: bit c % 32 of word c / 32.  Rows of
            // a tile are near one another, so where the page as a whole is not, most words are all ones or all zeros
            // in the whole warp.
            uint32_t see[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
            if (!(flags & kWhole)) {
                const int hi = req == d.w ? pos - d.z : -1;
                const int lo = pos - (a.window - 1) - d.z, sk = a.n_sink - d.z;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    see[k] = ones_below(hi + 1 - 32 * k) & (~ones_below(lo - 32 * k) | ones_below(sk - 32 * k));
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) poison |= (nan_v[k] & see[k]) != 0u;
            // S of the page's halves comes into the halves of the tile's columns, the first one into that which P of the
            // step before does not take; P goes over the first one.
            const uint32_t t_p = t_s + uint32_t((s & 1) * 64);
            auto wait_s = [&](int hb) {
                ok &= bool(__all_sync(0xffffffffu, mbar_wait(&sm.s_full[x][hb], s & 1, err, &sm.abort)));
                tc_fence_after();
            };
            // One pass over each half of the row: weights by the reference so far, and the maximum beside them.  Where a
            // logit passes the reference too far (S of the half is still there), the reference is raised and the half
            // weighed again.  The code between two votes has no branches: with one per 32 columns a step took 1.4 times
            // as long.
            auto weigh = [&](int hb, uint32_t bits0, uint32_t bits1, auto masked) {
                const uint32_t t = t_s + uint32_t(((s & 1) ^ hb) * 64);
                wait_s(hb);
                for (;;) {
                    const uint64_t nref2 = dup2(ref == -INFINITY ? 0.f : -ref);
                    uint64_t acc2[4] = {0, 0, 0, 0};
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    uint32_t v[2][16], w[2][16];
                    tmem_ld16(t, v[0]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t (&c)[16] = v[k & 1];
                        tmem_ld_wait();
                        if (k < 3) tmem_ld16(t + uint32_t(16 * k + 16), v[(k + 1) & 1]);
                        if constexpr (decltype(masked)::value) {
                            const uint32_t bits = k < 2 ? bits0 : bits1;
#pragma unroll
                            for (int i = 0; i < 16; ++i) c[i] = bits >> (16 * (k & 1) + i) & 1u ? c[i] : 0xff800000u;
                        }
#pragma unroll
                        for (int i = 0; i < 16; i += 8)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                mx[j] = fmax3(mx[j], __uint_as_float(c[i + j]), __uint_as_float(c[i + 4 + j]));
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            float xa, xb;
                            add_mul2(xa, xb, __uint_as_float(c[2 * i]), __uint_as_float(c[2 * i + 1]), nref2, scale2);
                            const float pa = fast_exp2(xa), pb = fast_exp2(xb);
                            w[k >> 1][8 * (k & 1) + i] = pack_bf16x2(pa, pb);
                            fadd2_acc(acc2[i & 3], pa, pb);
                        }
                    }
                    const float m = fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]);
                    const bool raise = (m - ref) * scale > kRaise;   // false for rows that see nothing
                    if (!__any_sync(0xffffffffu, raise)) {
                        tmem_st16(t_p + uint32_t(32 * hb), w[0]);
                        tmem_st16(t_p + uint32_t(32 * hb + 16), w[1]);
                        l += (sum2(acc2[0]) + sum2(acc2[1])) + (sum2(acc2[2]) + sum2(acc2[3]));
                        return;
                    }
                    // by a whole number of binades, so that what was summed with the old reference is brought to the
                    // new one by a power of two: exactly, the first half's P (bf16) included
                    const float up = raise && ref != -INFINITY ? ceilf((m - ref) * scale) : 0.f;
                    const float al = up < 126.f ? __int_as_float((127 - int(up)) << 23) : 0.f;
                    ref = !raise ? ref : up > 0.f && up < 126.f ? ref + up / scale : m;
                    l *= al;
                    const uint32_t al2 = pack_bf16x2(al, al);
                    tmem_st_wait();
#pragma unroll 1
                    for (int i = 0; i < 32 * hb; i += 16) {
                        uint32_t o[16];
                        tmem_ld16(t_p + uint32_t(i), o);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] = mul_bf16x2(o[j], al2);
                        tmem_st16(t_p + uint32_t(i), o);
                    }
                    if (!(flags & kFirst)) {   // S of the second half comes behind the P V before it: O is complete then
                        wait_s(1);
#pragma unroll 1
                        for (int i = 0; i < D; i += 16) {
                            uint32_t o[16];
                            tmem_ld16(t_o + uint32_t(i), o);
                            tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * al);
                            tmem_st16(t_o + uint32_t(i), o);
                        }
                    }
                }
            };
            if (flags & kWhole) {
#pragma unroll 1
                for (int hb = 0; hb < 2; ++hb) weigh(hb, 0u, 0u, std::false_type());
            } else {
#pragma unroll 1
                for (int hb = 0; hb < 2; ++hb) weigh(hb, hb ? see[2] : see[0], hb ? see[3] : see[1], std::true_type());
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (ok && lane == 0) arrive_first<PAIR>(&sm.p_full[x]);
            if (flags & kLast) {
                ok = __all_sync(0xffffffffu, mbar_wait(&sm.o_full[x], items & 1, err, &sm.abort)) && ok;
                ++items;
                tc_fence_after();
                const bool live = ok && row < a.n_rows && req != -1;
                const size_t head = live ? size_t(row) * a.Hq + g * HPG + h : 0;
                const float inv = poison ? __uint_as_float(0x7fffffffu) : l == 0.f ? 0.f : 1.0f / l;
                uint16_t *o_out = a.out + head * D;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    tmem_ld32(t_o + uint32_t(c), o);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        uint4 w;
                        w.x = pack_bf16x2(__uint_as_float(o[i]) * inv, __uint_as_float(o[i + 1]) * inv);
                        w.y = pack_bf16x2(__uint_as_float(o[i + 2]) * inv, __uint_as_float(o[i + 3]) * inv);
                        w.z = pack_bf16x2(__uint_as_float(o[i + 4]) * inv, __uint_as_float(o[i + 5]) * inv);
                        w.w = pack_bf16x2(__uint_as_float(o[i + 6]) * inv, __uint_as_float(o[i + 7]) * inv);
                        if (live) *reinterpret_cast<uint4 *>(o_out + c + i) = w;
                    }
                }
                if (live && l == 0.f) sm.empty = 1;
                if (live) a.lse[head] = l == 0.f ? -INFINITY : (ref * scale + log2f(l)) * kLn2;
                tc_fence_before();
            }
            if (!ok) break;
        }
    }

    tc_fence_before();
    if constexpr (PAIR) cluster_sync();  // neither CTA leaves while the other's MMAs or arrivals may reach it
    else __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        if constexpr (PAIR)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
        else
            tmem_dealloc(tmem, 512);
    }
    // Heads without weights got 0 and -inf.  Those whose q is not finite are made NaN here, behind all roles: looked for in
    // the epilogue, they took 2 % of the kernel's time.
    if (sm.empty && !sm.abort) {
        for (int item = blockIdx.x / CT; item < a.n_items; item += gridDim.x / CT) {
            const int set = item / a.G, g = item - set * a.G;
            for (int i = tid; i < 2 * EPT * HPG; i += kThreads)
                poison_empty<D>(a, (set * CT + rank) * 2 * EPT + i / HPG, g * HPG + i % HPG);
        }
    }
}

template <int D, int HPG, bool PAIR>
cudaError_t launch_t(const void *q, Args a, const Shape &s, cudaStream_t st) {
    alignas(64) CUtensorMap qm;
    const char *why = nullptr;
    const uint64_t dims[3] = {uint64_t(D), uint64_t(s.Hq), uint64_t(a.n_rows)};
    const uint64_t strides[2] = {uint64_t(D) * 2, uint64_t(s.Hq) * D * 2};
    const uint32_t box[3] = {64u, uint32_t(HPG), uint32_t(128 / HPG)};
    if (!encode_tensor_map(&qm, 3, q, dims, strides, box, 128, &why)) return cudaErrorInvalidValue;
    constexpr int CT = PAIR ? 2 : 1, kRows = 2 * CT * 128 / HPG;
    const long long items = ((a.n_rows + kRows - 1LL) / kRows) * s.G;
    if (items > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    a.n_items = int(items);
    const size_t smem = sizeof(Smem<D, PAIR>) + 1024;
    auto k = k_window_q8<D, HPG, PAIR>;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_once(allowed, reinterpret_cast<const void *>(k), smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(std::min<long long>(items, sm_count() / CT) * CT));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CT;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, a, qm);
}

}  // namespace

cudaError_t launch_window_prefill_q8(const void *q, const CacheQ8 &c, const int32_t *block_table, const int32_t *q_req,
                                     const int32_t *q_pos, int n_rows, int n_req, int n_pages, int window, int n_sink,
                                     const Shape &s, void *out, float *lse, int32_t *err, cudaStream_t st) {
    Args a = {};
    a.q = static_cast<const uint16_t *>(q);
    a.k = static_cast<const uint8_t *>(c.k);
    a.k_scale = static_cast<const uint8_t *>(c.k_scale);
    a.v = static_cast<const uint8_t *>(c.v);
    a.v_scale = static_cast<const uint8_t *>(c.v_scale);
    a.block_table = block_table;
    a.q_req = q_req;
    a.q_pos = q_pos;
    a.n_rows = n_rows;
    a.n_req = n_req;
    a.n_pages = n_pages;
    a.max_blocks = s.max_blocks;
    a.Hq = s.Hq;
    a.G = s.G;
    a.window = window;
    a.n_sink = n_sink;
    a.sm_scale = s.sm_scale;
    a.out = static_cast<uint16_t *>(out);
    a.lse = lse;
    a.err = err;
#define MSA_WQ_CASE(DD, HH) \
    if (s.D == DD && s.hpg == HH) return launch_t<DD, HH, DD == 128>(q, a, s, st);
    MSA_WQ_CASE(128, 8) MSA_WQ_CASE(128, 4) MSA_WQ_CASE(64, 8) MSA_WQ_CASE(64, 4)
#undef MSA_WQ_CASE
    return cudaErrorNotSupported;
}

}  // namespace msa
