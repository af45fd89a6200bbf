// Sparse attention of drafted trees over the paged cache, on the 5th-generation tensor cores.
//
// Row (node i, head h) of group g attends, with one softmax, the cached tokens of the blocks that node i selected
// and those of its ancestors (and itself) whose block it selected:
//   o = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m),  s_t = sm_scale * q . k_t,  m = max_t s_t.
//
// The nodes of a tree agree on many blocks, so the work goes by the union of their selections: each (request,
// group, up to 256 / HPG nodes) is a tile, its items are the selected blocks (each with the word of the nodes that
// selected it) and one item for the drafted tokens, and each item's K and V are read once for all nodes of the
// tile.  With up to 128 rows in a tile that read bounds the loop (8 x 60,000 tokens of 16 nodes: 174 MB in 26 us,
// 6.6 TB/s; 48 us with the plan, the first loads, the last output and the join).  With two halves of 128 rows it
// is the chain S, softmax, P V of each half, 1.7 us for a unit, that bounds it (64 nodes: 499 MB, 140 us in all;
// the same time with every page in L2).
//
// k_tree_plan, one CTA per (request, group): the union through a bitmap over blocks in shared memory, ranked by
// popcounts, hence the same whatever order its threads run in.  With HPG = 8 and more than 16 nodes the nodes' order
// matters: a tile reads what any of its nodes selected, and its 128-row halves skip the items that none of theirs did.
// Two orders are counted, items and units of halves together, and the cheaper one is taken: the tree's own, and one by
// the least hash of a node's blocks that not most nodes have, which is the same for two nodes the more likely the
// more of their blocks they share.  8 x 60,000 tokens, 64 nodes: windows of 7 blocks that nodes far apart share, 256 us
// in the tree's own order and 137 hashed; children that keep all but one of their parent's blocks, 122 and 155 in a
// chain, 130 and 151 with parents among the four nodes before, 138 and 138 with four children a node in breadth order
// (counting both costs 2 us).  A tile's items are then merged so that the halves take turns (143 us, and 147 without).
//
// k_attn_tree, one persistent CTA per SM: the items of all tiles, in order, are cut into one range per CTA, so one
// long tile is spread over many SMs and many short ones share them.  Leaving one tile for the next costs a CTA
// about the time of kTileCost items (its output, and no attention meanwhile), so each tile counts for so many
// items more where the ranges are cut (one, where a range is a few items and latency counts).  The part of a tile
// inside a range is a segment; it keeps one online softmax.  A tile cut by a range's end leaves partials
// (unnormalised O, max and sum, in 32 bits: in 16 they would cost a rounding more) in the workspace, and
// k_tree_join joins them in the order of the ranges: a kernel of its own, because one CTA reading all partials of
// a tile took longer than the attention itself (13 partials of 40 rows: 20 us of 35).  Warps:
//   0      K/V producer: TMA boxes of 64 columns x 128 tokens (128B swizzle) into a ring for each;
//   1      MMA issuer: S = Q K^T into the TMEM buffer of a softmax group, then, one unit later, O += P V with
//          P in TMEM (over S) and V as an MN-major shared-memory operand (an issuer for each was no faster, and
//          its warp is worth more to the check of V: 16 nodes, 57 us against 52);
//   4-7, 8-11  two softmax groups, one thread per row.  With up to 128 rows in the tile they take alternate
//          items, each with an O of its own, joined at the segment's end; with more, each has half the
//          rows.  P = 2^(s - m) for a reference m that is the row's first maximum (rounded up to a whole
//          power of two) until a logit passes it by 2^40: P, sums and O are floating point of 8 exponent bits
//          throughout, so a reference below the true maximum costs no precision, S is read once, and O, in
//          TMEM, is next to never rescaled (by a power of two then, exactly).  P is rounded to bf16, as the
//          operand of the MMA: half a step, 2^-8 of each weight, as large as the rounding of the output;
//   2, 3   Q loads (one box of 64 columns x HPG heads x 128/HPG nodes is a whole 128-row tile of Q), and the
//          finite check of V: a row that does not see a token has P = 0 there, and 0 * NaN would still reach its
//          O through the MMA, so what is not finite is replaced by 0 before the MMA reads it.  Rows that
//          do see such a value get it back at the segment's end, off the hot path.
// TMEM: S0 | S1 | O0 | O1 (128 + 128 + D + D of 512 columns).  Every barrier has one waiting role, which waits for
// each of its phases in order (or, for a group's O, knows the one before to be over).  Every wait is bounded.
#include "msa_device.cuh"
#include "msa_internal.h"

#include <algorithm>

namespace msa {
namespace {

constexpr int kThreads = 384;           // 168 registers a thread
constexpr int kMaxCtas = 160;           // partial slots in the workspace; at most one CTA per SM
constexpr int kOkRing = 8;              // finite-check barriers, by item
constexpr int kTileCost = 3;            // of a tile, in items, where the ranges are cut
constexpr int kSortedBit = 1 << 30;     // of a tile's place in `order`: not the nodes' own order
constexpr int kDraftBit = 1 << 30;      // of a tile's item count: its last item is the drafted tokens
constexpr float kRaise = 40.0f;         // raise the reference once a logit is this far above (log2 units)
constexpr float kRaiseSum = 1099511627776.0f;   // 2^kRaise
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// One block of a tile's union: its page, the number of cached tokens in it, the nodes that selected it.
struct __align__(16) Item {
    int32_t page, n_tok;
    uint32_t nodes[2];
};

// What the plan says of a tile; n_items 0: nothing to do.
struct __align__(16) Tile {
    int32_t n_items;    // | kDraftBit
    int32_t nodes, row0;   // its nodes, the request's first row
    int32_t ord;        // where its nodes' numbers begin in `order` | kSortedBit
};

// 128 rows of a cut tile: the ranges (CTAs) that hold it, and whose rows they are.
struct __align__(16) Cut {
    int32_t first, last, half, g, row0, nodes, ord, pad;
};

struct Layout {
    int per_tile;       // nodes of a tile
    int chunks;         // tiles per (request, group)
    int cap;            // items of a tile, at most
    long long tiles;
    size_t tile, cut, n_cut, order, dmask, items, part, bytes;
};

__host__ __device__ constexpr size_t part_floats(int D) { return size_t(256) * D + 512; }   // O, then (m, l) per row

inline Layout layout(int n_rows, int n_req, const Shape &s) {
    Layout w;
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    w.per_tile = 256 / s.hpg;
    const int nodes = std::min(n_rows, kTreeMaxNodes);
    w.chunks = std::max(1, (nodes + w.per_tile - 1) / w.per_tile);
    w.cap = int(std::min<long long>(1LL * std::min(nodes, w.per_tile) * s.topk, s.max_blocks)) + 1;
    w.tiles = 1LL * n_req * w.chunks * s.G;
    w.tile = 0;
    w.cut = up(size_t(w.tiles) * sizeof(Tile));
    w.n_cut = w.cut + up(size_t(w.tiles) * 2 * sizeof(Cut));
    w.order = w.n_cut + 256;
    w.dmask = w.order + up(size_t(n_req) * s.G * kTreeMaxNodes);
    w.items = w.dmask + up(size_t(n_rows) * s.G * 8);
    w.part = w.items + up(size_t(w.tiles) * w.cap * sizeof(Item));
    w.bytes = w.part + size_t(2 * kMaxCtas) * part_floats(s.D) * 4;
    return w;
}

// ------------------------------------------------------------------ plan

constexpr int kPlanThreads = 256;
constexpr int kMaxWords = 16384 / 32;   // bitmap over blocks

// Which 128-row halves of a tile an item's nodes are in.
template <int HPG>
__device__ __forceinline__ uint32_t half_bits(uint32_t n0, uint32_t n1) {
    if constexpr (HPG == 4) return (n0 ? 1u : 0u) | (n1 ? 2u : 0u);
    return (n0 & 0xffffu ? 1u : 0u) | (n0 >> 16 ? 2u : 0u);
}
template <int HPG>
__device__ __forceinline__ uint32_t half_bits(const Item &it) {
    return half_bits<HPG>(it.nodes[0], it.nodes[1]);
}

// Exclusive prefix of v over the CTA's threads; *total gets the sum.
template <class T>
__device__ __forceinline__ T plan_scan(T v, T *wsum, T *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    T before = incl - v, sum = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        const T x = wsum[w];
        if (w < warp) before += x;
        sum += x;
    }
    *total = sum;
    return before;
}

template <int D, int HPG>
__global__ void __launch_bounds__(kPlanThreads, 2) k_tree_plan(
    const int32_t *__restrict__ sel, const int32_t *__restrict__ block_table, const int32_t *__restrict__ ctx_lens,
    const int32_t *__restrict__ node_off, const uint64_t *__restrict__ anc, int n_rows, int n_pages, int G, int topk,
    int max_blocks, int chunks, int cap, Tile *__restrict__ tiles, int32_t *__restrict__ n_cut,
    uint8_t *__restrict__ order, unsigned long long *__restrict__ dmask, Item *__restrict__ items,
    uint4 *__restrict__ out, float *__restrict__ lse, int32_t *err) {
    constexpr int PER = 256 / HPG;                     // nodes of a tile, at most 64
    constexpr int NPM = 128 / HPG;                     // nodes of 128 rows
    constexpr int CAP = kTreeMaxNodes * 32;            // selected blocks, at most
    constexpr int EPT = CAP / kPlanThreads;
    __shared__ uint32_t bits[kMaxWords];
    __shared__ uint32_t rank[kMaxWords];               // set bits below the word
    __shared__ uint32_t words_of[2][CAP][2];           // nodes of the union's blocks: by number, by the hashed places
    __shared__ uint16_t block_of[CAP];
    __shared__ unsigned long long in_first, in_second; // nodes whose block is ctx / 128, or the next one
    __shared__ uint32_t has[kTreeMaxNodes];            // bit 0 / 1: the node selected that block
    __shared__ uint32_t key[kTreeMaxNodes];
    __shared__ uint8_t place[kTreeMaxNodes];
    __shared__ uint32_t draft_at[2];                   // places whose nodes see drafted tokens
    __shared__ int wsum[kPlanThreads / 32];
    __shared__ unsigned long long wsum3[2][kPlanThreads / 32];
    const int tid = threadIdx.x;
    const int b = blockIdx.x / G, g = blockIdx.x - b * G;
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x == 0 && tid == 0) *n_cut = 0;
    int row0;
    const int ctx = ctx_lens[b];
    const int n = tree_rows_of(node_off, b, n_rows, err, tid == 0 && g == 0, &row0);
    auto tile_of = [&](int chunk) { return (b * chunks + chunk) * G + g; };
    if (n <= 0 || ctx < 0) {
        if (n > 0 && tid == 0) raise_flag(err, MSA_FLAG_BOUNDS);
        if (tid < chunks) tiles[tile_of(tid)] = Tile{0, 0, 0, 0};
        return;
    }
    // this thread's entries of the selection, loaded together (-1 where there is none)
    const int n_ent = n * topk;
    int ent[EPT];
#pragma unroll
    for (int x = 0; x < EPT; ++x) {
        const int e = tid + x * kPlanThreads;
        ent[x] = e < n_ent ? sel[(size_t(row0 + e / topk) * G + g) * topk + e % topk] : -1;
    }
    const unsigned long long path = tid < n ? anc[row0 + tid] : 0ull;
    const int words = (max_blocks + 31) >> 5;
    for (int i = tid; i < words; i += kPlanThreads) bits[i] = 0;
    uint32_t(*nodes_of)[2] = words_of[0];              // in the order that is taken
    for (int i = tid; i < 2 * min(n_ent, CAP); i += kPlanThreads) (&words_of[0][0][0])[i] = (&words_of[1][0][0])[i] = 0;
    if (tid < kTreeMaxNodes) has[tid] = 0, key[tid] = ~0u;
    if (tid == 0) in_first = in_second = 0, draft_at[0] = draft_at[1] = 0;
    __syncthreads();
    const int j0 = ctx >> 7;
    if (tid < n) {
        const int j = (ctx + __popcll(path) - 1) >> 7;
        if (j == j0) atomicOr(&in_first, 1ull << tid);
        else if (j == j0 + 1) atomicOr(&in_second, 1ull << tid);
    }
#pragma unroll
    for (int x = 0; x < EPT; ++x) {
        const int j = ent[x], i = (tid + x * kPlanThreads) / topk;
        if (j < 0) continue;
        if (j >= max_blocks) {
            raise_flag(err, MSA_FLAG_BOUNDS);
            ent[x] = -1;
            continue;
        }
        if (j == j0) atomicOr(&has[i], 1u);
        else if (j == j0 + 1) atomicOr(&has[i], 2u);
        if (j < j0 || (j == j0 && (ctx & 127))) atomicOr(&bits[j >> 5], 1u << (j & 31));
        else ent[x] = -1;   // a block without cached tokens
    }
    __syncthreads();
    // rank of every word, two words per thread; every selected block's place in the union and its nodes
    const int w0 = 2 * tid, w1 = w0 + 1;
    const int p0 = w0 < words ? __popc(bits[w0]) : 0, p1 = w1 < words ? __popc(bits[w1]) : 0;
    int total;
    const int before = plan_scan(p0 + p1, wsum, &total);
    if (w0 < words) rank[w0] = before;
    if (w1 < words) rank[w1] = before + p0;
    if (tid < n) place[tid] = uint8_t(tid);
    __syncthreads();
    bool sorted = HPG == 8 && n > NPM;   // (with HPG = 4, Q comes in boxes of neighbouring rows)
#pragma unroll
    for (int x = 0; x < EPT; ++x) {
        const int j = ent[x], i = (tid + x * kPlanThreads) / topk;
        if (j < 0) continue;
        const int k = rank[j >> 5] + __popc(bits[j >> 5] & ((1u << (j & 31)) - 1));
        ent[x] = k;              // from here on: the block's place in the union
        atomicOr(&nodes_of[k][i >> 5], 1u << (i & 31));
        block_of[k] = uint16_t(j);   // the same from every node that selected it
    }
    __syncthreads();
    if (sorted) {
#pragma unroll
        for (int x = 0; x < EPT; ++x) {
            const int k = ent[x], i = (tid + x * kPlanThreads) / topk;
            if (k < 0 || 2 * (__popc(nodes_of[k][0]) + __popc(nodes_of[k][1])) > n) continue;
            atomicMin(&key[i], (uint32_t(block_of[k]) + 1u) * 2654435761u);
        }
        __syncthreads();
        if (tid < n) {
            const uint32_t mine = key[tid];
            int p = 0;
            for (int m = 0; m < n; ++m) p += key[m] < mine || (key[m] == mine && m < tid);
            place[tid] = uint8_t(p);
        }
        __syncthreads();
#pragma unroll
        for (int x = 0; x < EPT; ++x) {
            const int k = ent[x], i = (tid + x * kPlanThreads) / topk;
            if (k < 0) continue;
            const int p = place[i];
            atomicOr(&words_of[1][k][p >> 5], 1u << (p & 31));
        }
        __syncthreads();
        // What either order costs: tiles that read a block, and 128-row halves that it is a unit of.
        unsigned long long cost = 0, costs;   // by number in the low word
        for (int k = tid; k < total; k += kPlanThreads)
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const uint32_t w = words_of[y >> 1][k][y & 1];
                cost += (unsigned long long)((w != 0) + ((w & 0xffffu) != 0) + (w >> 16 != 0)) << (32 * (y >> 1));
            }
        plan_scan(cost, wsum3[0], &costs);
        sorted = uint32_t(costs >> 32) < uint32_t(costs);
        if (sorted) nodes_of = words_of[1];
        else if (tid < n) place[tid] = uint8_t(tid);
        __syncthreads();
    }
    // the drafted tokens that each node sees, and the nodes by place
    if (tid < n) {
        unsigned long long m = 0;
        if (has[tid] & 1) m |= in_first;
        if (has[tid] & 2) m |= in_second;
        m &= path & (n == 64 ? ~0ull : (1ull << n) - 1);
        dmask[size_t(row0 + tid) * G + g] = m;
        const int p = place[tid];
        if (m) atomicOr(&draft_at[p >> 5], 1u << (p & 31));
        order[size_t(blockIdx.x) * kTreeMaxNodes + p] = uint8_t(tid);
    }
    __syncthreads();
    for (int chunk = 0; chunk < chunks; ++chunk) {
        const int tile = tile_of(chunk), nt = min(PER, n - chunk * PER);
        if (nt <= 0) {
            if (tid == 0) tiles[tile] = Tile{0, 0, 0, 0};
            continue;
        }
        auto nodes_at = [&](const uint32_t (&w)[2], int h) { return PER == 64 ? w[h] : h ? 0u : w[chunk & 1]; };
        // The union's blocks that a node of this tile selected, in three classes: of the first 128 rows alone, of the
        // second alone, of both.  A run of blocks per thread is counted, then written.
        const int k0 = tid * total / kPlanThreads, k1 = (tid + 1) * total / kPlanThreads;
        auto item_of = [&](int k) { return Item{0, 0, {nodes_at(nodes_of[k], 0), nodes_at(nodes_of[k], 1)}}; };
        unsigned long long mine = 0, sums;   // 21 bits per class
        for (int k = k0; k < k1; ++k) {
            const uint32_t h = half_bits<HPG>(item_of(k));
            if (h) mine += 1ull << (21 * (h - 1));
        }
        unsigned long long before = plan_scan(mine, wsum3[chunk & 1], &sums);
        const int cnt[3] = {int(sums & 0x1fffff), int(sums >> 21 & 0x1fffff), int(sums >> 42)};
        const int n_blocks = cnt[0] + cnt[1] + cnt[2];
        Item *list = items + size_t(tile) * cap;
        for (int k = k0; k < k1; ++k) {
            Item it = item_of(k);
            const uint32_t h = half_bits<HPG>(it);
            if (!h) continue;
            // The classes are merged evenly, each in ascending order, so that the halves take turns and a CTA's range
            // has its share of each: item r of class q goes by (2 r + 1) / (2 cnt[q]), ties by class.
            const int q = int(h) - 1, r = int(before >> (21 * q) & 0x1fffff);
            before += 1ull << (21 * q);
            const int cnt_q = q == 0 ? cnt[0] : q == 1 ? cnt[1] : cnt[2];
            int at = r;
#pragma unroll
            for (int p = 0; p < 3; ++p)
                if (p != q && cnt[p]) at += (((2 * r + 1) * cnt[p] - (p < q ? 0 : 1)) / cnt_q + 1) >> 1;
            const int j = block_of[k];
            it.page = block_table[size_t(b) * max_blocks + j];
            it.n_tok = min(128, ctx - j * 128);
            if (it.page < 0 || it.page >= n_pages) {   // refused: seen by no row
                raise_flag(err, MSA_FLAG_BOUNDS);
                it.page = 0;
                it.nodes[0] = it.nodes[1] = 0;
            }
            list[at] = it;
        }
        const uint32_t d0 = nodes_at(draft_at, 0), d1 = nodes_at(draft_at, 1);
        const bool drafts = d0 | d1;
        if (tid == 0) {
            if (drafts) list[n_blocks] = Item{0, n, {d0, d1}};
            tiles[tile] = Tile{drafts ? (n_blocks + 1) | kDraftBit : n_blocks, nt, row0,
                               (int(blockIdx.x) * kTreeMaxNodes + chunk * PER) | (sorted ? kSortedBit : 0)};
        }
        if (n_blocks == 0 && !drafts) {   // nothing is seen: the rows' results are written here
            constexpr int CH = HPG * D / 8;
            auto row_of = [&](int i) {   // the row of the node at the tile's place i
                int m = 0;
                while (place[m] != chunk * PER + i) ++m;
                return size_t(row0 + m) * G + g;
            };
            for (int i = tid; i < nt * CH; i += kPlanThreads) out[row_of(i / CH) * CH + i % CH] = make_uint4(0, 0, 0, 0);
            for (int i = tid; i < nt * HPG; i += kPlanThreads) lse[row_of(i / HPG) * HPG + i % HPG] = -INFINITY;
        }
    }
}

// ------------------------------------------------------------------ attention

template <int D>
struct TreeSmem {
    static constexpr int NK = D == 128 ? 2 : 5, NV = D == 128 ? 3 : 5;   // V waits one item longer than K
    alignas(1024) uint8_t q[2][128 * D * 2];
    alignas(1024) uint8_t k[NK][128 * D * 2];
    alignas(1024) uint8_t v[NV][128 * D * 2];
    float2 join[128];              // the second group's (max, sum), then both groups' weights
    uint64_t q_full, q_empty;
    uint64_t k_full[NK], k_empty[NK], v_full[NV], v_empty[NV];
    uint64_t v_ok[kOkRing];
    uint64_t s_full[2], p_ready[2], o_done[2];
    uint64_t o_free, drain;
    int2 wsum[kThreads / 32];
    int tile0, at0;
    uint32_t tmem_base;
    int abort, nonfinite;
};

__device__ __forceinline__ float fast_exp2(float x) {   // MUFU.EX2, relative error about 2^-22
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// D / 16 MMAs of S = Q K^T (K = 16 each), A and B K-major with 128-byte swizzle: a k-step advances 32 bytes within
// a 64-column box and 16 KB between boxes (+2 / +1024 in the descriptors' units of 16 bytes).  One asm block: MMAs
// issued one by one lose issue slots to the softmax warps of the sub-partition.  (Issued by a converged
// warp with one lane predicated, the kernel was 8 % slower: 32 lanes polled each barrier.)
template <int D>
__device__ __forceinline__ void mma_s(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
    if constexpr (D == 128) {
        asm volatile(
            "{\n\t.reg .pred f, t;\n\t.reg .b64 a1, a2, a3, a4, a5, a6, a7, b1, b2, b3, b4, b5, b6, b7;\n\t"
            "setp.ne.b32 f, %3, %3;\n\tsetp.eq.b32 t, %3, %3;\n\t"
            "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\tadd.s64 a4, %1, 1024;\n\t"
            "add.s64 a5, %1, 1026;\n\tadd.s64 a6, %1, 1028;\n\tadd.s64 a7, %1, 1030;\n\t"
            "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\tadd.s64 b4, %2, 1024;\n\t"
            "add.s64 b5, %2, 1026;\n\tadd.s64 b6, %2, 1028;\n\tadd.s64 b7, %2, 1030;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, f;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a4, b4, %3, t;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a5, b5, %3, t;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a6, b6, %3, t;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a7, b7, %3, t;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc)
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred f, t;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
            "setp.ne.b32 f, %3, %3;\n\tsetp.eq.b32 t, %3, %3;\n\t"
            "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
            "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, f;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc)
            : "memory");
    }
}

// O (+)= P V over 64 tokens: A = P in TMEM (8 columns per 16 tokens), B = V (2 KB per 16 tokens).
__device__ __forceinline__ void mma_pv64(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, t;\n\t.reg .b64 b1, b2, b3;\n\t.reg .b32 a1, a2, a3;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, %4, %4;\n\t"
        "add.s32 a1, %1, 8;\n\tadd.s32 a2, %1, 16;\n\tadd.s32 a3, %1, 24;\n\t"
        "add.s64 b1, %2, 128;\n\tadd.s64 b2, %2, 256;\n\tadd.s64 b3, %2, 384;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// Two fp32 lanes per instruction; b2 and c2 hold one value in both halves.
__device__ __forceinline__ uint64_t dup2(float x) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ void ffma2(float &d0, float &d1, float a0, float a1, uint64_t b2, uint64_t c2) {
    asm("{\n\t.reg .b64 x, d;\n\tmov.b64 x, {%2, %3};\n\tfma.rn.f32x2 d, x, %4, %5;\n\tmov.b64 {%0, %1}, d;\n\t}"
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

// Both softmax groups.
__device__ __forceinline__ void groups_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// Ranges are cut in units of cost: a tile has `extra` units before its items.  The first unit of range c:
__device__ __forceinline__ int range_begin(int c, int n, int C) {
    if (n < 1 << 24) return int(uint32_t(c) * uint32_t(n) / uint32_t(C));   // c <= kMaxCtas: within 32 bits
    return int((long long)c * n / C);
}
__device__ __forceinline__ int range_owner(int x, int n, int C) { return int(((long long)(x + 1) * C - 1) / n); }

// The CTA's segments in order; every role walks them for itself.
struct Walk {
    const Tile *tiles;
    int x, x1;               // the present tile's first unit of cost; the range's end
    int extra;               // a tile's cost beside its items
    int tile, off, end, n_items, seg;
    Tile t;
    bool drafts, sorted;
    __device__ __forceinline__ bool next() {   // the next segment: items off .. end-1 of `tile`, n_items in it
        if (seg >= 0) {
            x += n_items + extra;
            ++tile;
            off = 0;
        }
        for (;; ++tile) {
            if (x + extra >= x1) return false;   // no item of the next tile, if any, lies before the end
            const int4 v = *reinterpret_cast<const int4 *>(tiles + tile);
            t = Tile{v.x, v.y, v.z, v.w & ~kSortedBit};
            sorted = v.w & kSortedBit;
            n_items = t.n_items & ~kDraftBit;
            if (n_items) break;
        }
        drafts = t.n_items & kDraftBit;
        end = min(n_items, x1 - x - extra);
        ++seg;
        return true;
    }
};

__device__ __forceinline__ uint32_t exp_all_ones(uint32_t w) {   // 0x8000 in each half that is inf or NaN
    return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}

template <int D, int HPG>
__global__ void __launch_bounds__(kThreads, 1) k_attn_tree(
    const uint16_t *__restrict__ q, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap qnode,
    const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
    const __grid_constant__ CUtensorMap knmap, const __grid_constant__ CUtensorMap vnmap,
    const uint16_t *__restrict__ k_cache, const uint16_t *__restrict__ v_cache, const uint16_t *__restrict__ k_new,
    const uint16_t *__restrict__ v_new, int G, int cap, int n_tiles, float sm_scale,
    const uint8_t *__restrict__ order, const Tile *__restrict__ tiles, Cut *__restrict__ cut, int32_t *__restrict__ n_cut,
    const unsigned long long *__restrict__ dmask, const Item *__restrict__ items, float *__restrict__ part,
    uint16_t *__restrict__ out, float *__restrict__ lse, int32_t *err) {
    using Smem = TreeSmem<D>;
    constexpr int NK = Smem::NK, NV = Smem::NV;
    constexpr int NSUB = D / 64;
    constexpr int NPM = 128 / HPG;     // nodes of a 128-row MMA tile
    constexpr uint32_t kIdescS = make_idesc_bf16(128, 128, 0, 0);
    constexpr uint32_t kIdescS64 = make_idesc_bf16(128, 64, 0, 0);
    constexpr uint32_t kIdescO = make_idesc_bf16(128, D, 0, 1);
    extern __shared__ uint8_t smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    if (tid == 0) {
        mbar_init(&sm.q_full, 1);
        mbar_init(&sm.q_empty, 1);
        for (int i = 0; i < NK; ++i) {
            mbar_init(&sm.k_full[i], 1);
            mbar_init(&sm.k_empty[i], 1);
        }
        for (int i = 0; i < NV; ++i) {
            mbar_init(&sm.v_full[i], 1);
            mbar_init(&sm.v_empty[i], 1);
        }
        for (int i = 0; i < kOkRing; ++i) mbar_init(&sm.v_ok[i], 2);
        for (int w = 0; w < 2; ++w) {
            mbar_init(&sm.s_full[w], 1);
            mbar_init(&sm.p_ready[w], 4);
            mbar_init(&sm.o_done[w], 1);
        }
        mbar_init(&sm.o_free, 8);
        mbar_init(&sm.drain, 1);
        sm.abort = 0;
        sm.nonfinite = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&sm.tmem_base, 512);
        tmem_relinquish();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&kmap);
        tma_prefetch_desc(&vmap);
        tma_prefetch_desc(&qmap);
    }
    pdl_wait();   // the plan
    pdl_trigger();
    // this CTA's range: a scan of the tiles' item counts, a run of tiles per thread
    const int t_lo = int((long long)tid * n_tiles / kThreads), t_hi = int((long long)(tid + 1) * n_tiles / kThreads);
    int mine = 0, mine_t = 0;   // items and tiles
    for (int t = t_lo; t < t_hi; ++t) {
        const int c = tiles[t].n_items & ~kDraftBit;
        mine += c;
        mine_t += c > 0;
    }
    int incl = mine, incl_t = mine_t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o), z = __shfl_up_sync(0xffffffffu, incl_t, o);
        if (lane >= o) incl += y, incl_t += z;
    }
    if (lane == 31) sm.wsum[warp] = make_int2(incl, incl_t);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const int2 sums = lane < kThreads / 32 ? sm.wsum[lane] : make_int2(0, 0);
    const int n_items = warp_sum_i(sums.x), n_live = warp_sum_i(sums.y);
    const int extra = n_items >= 4 * int(gridDim.x) ? kTileCost : 1;
    const int before = warp_sum_i(lane < warp ? sums.x + extra * sums.y : 0) + incl - mine + extra * (incl_t - mine_t);
    const int total = n_items + extra * n_live;
    // every range holds an item (it is longer than a tile's extra cost), so that a cut tile's ranges are consecutive CTAs
    const int C = min(int(gridDim.x), max(total / (extra + 1), 1)), cta = blockIdx.x;
    const int x0 = cta < C ? range_begin(cta, total, C) : total, x1 = cta < C ? range_begin(cta + 1, total, C) : total;
    if (x0 < x1 && x0 >= before && x0 < before + mine + extra * mine_t) {
        int t = t_lo, at = before;
        while (t + 1 < t_hi) {
            const int c = tiles[t].n_items & ~kDraftBit;
            if (c && x0 < at + c + extra) break;
            at += c ? c + extra : 0;
            ++t;
        }
        sm.tile0 = t;
        sm.at0 = at;
    }
    __syncthreads();
    const uint32_t tmem = sm.tmem_base;
    // a range that begins within a tile's cost has the tile from its first item on
    const int at0 = x0 < x1 ? sm.at0 : total;
    Walk wk{tiles, at0, x1, extra, x0 < x1 ? sm.tile0 : 0, max(0, x0 - at0 - extra), 0, 0, -1, Tile{}, false, false};

    if (warp == 0) {
        // ------------------------------------------------------------ K/V producer (lane 0)
        if (lane == 0) {
            int it = 0, v_loads = 0;
            bool ok = true;
            // Pages leave L2 first (16 nodes: 48 us, 52 without; 64 nodes, whose two tiles read most pages at about the
            // same time: 146 us and 148).
            const uint64_t policy = l2_policy_evict_first();
            while (ok && wk.next()) {
                const int g = wk.tile % G;
                const Item *list = items + size_t(wk.tile) * cap;
                int page = list[wk.off].page;
                for (int i = wk.off; i < wk.end; ++i, ++it) {
                    const int page_i = page;
                    if (i + 1 < wk.end) page = list[i + 1].page;   // one ahead
                    const bool draft = wk.drafts && i == wk.n_items - 1;
                    const uint32_t bytes = draft ? 64 * D * 2 : 128 * D * 2;
                    const int ks = it % NK, vs = it % NV;
                    if (it >= NK && !mbar_wait(&sm.k_empty[ks], (it / NK - 1) & 1, err, &sm.abort)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&sm.k_full[ks], bytes);
#pragma unroll
                    for (int c = 0; c < NSUB; ++c) {
                        if (draft) tma_load_3d(sm.k[ks] + c * 16384, &knmap, &sm.k_full[ks], c * 64, g, wk.t.row0);
                        else tma_load_4d_hint(sm.k[ks] + c * 16384, &kmap, &sm.k_full[ks], c * 64, g, 0, page_i, policy);
                    }
                    if (it >= NV && !mbar_wait(&sm.v_empty[vs], (it / NV - 1) & 1, err, &sm.abort)) {
                        ok = false;
                        ++it;   // its K is in flight
                        break;
                    }
                    mbar_arrive_expect_tx(&sm.v_full[vs], bytes);
#pragma unroll
                    for (int c = 0; c < NSUB; ++c) {
                        if (draft) tma_load_3d(sm.v[vs] + c * 16384, &vnmap, &sm.v_full[vs], c * 64, g, wk.t.row0);
                        else tma_load_4d_hint(sm.v[vs] + c * 16384, &vmap, &sm.v_full[vs], c * 64, g, 0, page_i, policy);
                    }
                    v_loads = it + 1;
                }
            }
            if (sm.abort) {   // the copies still in flight land before the CTA exits
                for (int s = max(0, it - NK); s < it; ++s) mbar_wait(&sm.k_full[s % NK], (s / NK) & 1, err, nullptr);
                for (int s = max(0, v_loads - NV); s < v_loads; ++s)
                    mbar_wait(&sm.v_full[s % NV], (s / NV) & 1, err, nullptr);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (lane 0)
        if (lane == 0) {
            auto wait = [&](uint64_t *bar, int phase) { return mbar_wait(bar, uint32_t(phase & 1), err, &sm.abort); };
            int it = 0;                       // items of this CTA so far
            uint32_t units = 0;               // parity of the PV units issued for each group (bit w)
            bool ok = true, o_wait = false;
            const uint64_t q_desc = make_smem_desc(smem_u32(sm.q[0]), 16, 1024, 2);
            const uint64_t k_desc = make_smem_desc(smem_u32(sm.k[0]), 16, 1024, 2);
            const uint64_t v_desc = make_smem_desc(smem_u32(sm.v[0]), 16384, 1024, 2);
            constexpr uint64_t kTileStep = sizeof(sm.k[0]) / 16;   // between tiles, in the descriptors' units
            auto issue_s = [&](int w, int m, int slot, bool draft) {
                tc_fence_after();
                mma_s<D>(tmem + uint32_t(w * 128), q_desc + m * kTileStep, k_desc + slot * kTileStep,
                         draft ? kIdescS64 : kIdescS);
                mma_commit(&sm.s_full[w]);
            };
            // O += P V of a unit of item x: both groups have read the O of the segment before, V is checked, P is there
            auto issue_pv = [&](int w, int x, bool acc, bool draft, bool first, bool last) -> bool {
                if (o_wait && !wait(&sm.o_free, wk.seg - 1)) return false;
                o_wait = false;
                if (first && !wait(&sm.v_ok[x % kOkRing], x / kOkRing)) return false;
                if (!wait(&sm.p_ready[w], units >> w)) return false;
                units ^= 1u << w;
                tc_fence_after();
                const int slot = x % NV;
                const uint64_t vd = v_desc + slot * kTileStep;
                const uint32_t d = tmem + uint32_t(256 + w * D), a = tmem + uint32_t(w * 128);
                mma_pv64(d, a, vd, kIdescO, acc);
                if (!draft) mma_pv64(d, a + 32, vd + 512, kIdescO, 1u);
                mma_commit(&sm.o_done[w]);
                if (last) mma_commit(&sm.v_empty[slot]);
                return true;
            };
            while (ok && wk.next()) {
                o_wait = wk.seg > 0;
                if (!wait(&sm.q_full, wk.seg)) break;
                const int len = wk.end - wk.off;
                const bool ends = wk.drafts && wk.end == wk.n_items;   // the last item is the drafted tokens
                if (wk.t.nodes <= NPM) {
                    // one half: every item is a unit, of the groups in turn; S of a unit goes before P V of the one before
                    for (int x = 0; x <= len; ++x) {
                        if (x < len) {
                            const int slot = (it + x) % NK;
                            if (!(ok = wait(&sm.k_full[slot], (it + x) / NK))) break;
                            issue_s(x & 1, 0, slot, ends && x == len - 1);
                            mma_commit(&sm.k_empty[slot]);
                            if (x == len - 1) mma_commit(&sm.q_empty);
                        }
                        if (x > 0 && !(ok = issue_pv((x - 1) & 1, it + x - 1, x > 2, ends && x == len, true, true))) break;
                    }
                    it += len;
                    continue;
                }
                // two halves: a unit is an item and a half of which a node selected it
                const Item *list = items + size_t(wk.tile) * cap;
                // the items' nodes, two items ahead and looked at only when their turn comes
                auto nodes_of = [&](int x) {
                    const uint32_t *w = list[wk.off + min(x, len - 1)].nodes;
                    return HPG == 4 ? *reinterpret_cast<const uint2 *>(w) : make_uint2(w[0], 0u);
                };
                uint2 a0 = nodes_of(0), a1 = nodes_of(1), a2;
                uint32_t begun = 0;                          // halves whose O holds something of this segment
                int w_p = -1, x_p = 0;                       // the unit whose P V is to come, its item
                bool first_p = false, last_p = false;
                for (int x = 0; ok && x <= len; ++x) {       // one round more than items, for the last unit's P V
                    a2 = nodes_of(x + 2);
                    const uint32_t halves = x < len ? half_bits<HPG>(a0.x, a0.y) : 0u;
                    const int slot = (it + x) % NK;
                    if (x < len && !(ok = wait(&sm.k_full[slot], (it + x) / NK))) break;
#pragma unroll 1
                    for (int m = 0; ok && m < 2; ++m) {
                        const bool s = halves >> m & 1;
                        if (!s && (halves || m)) continue;   // (an item of nobody and the tail come by once, for the P V)
                        // S of one half goes before P V of the other's unit; its own P lies where its next S will.
                        // (One place in the code for each: written out for both orders, 64 nodes took 144 us, not 138.)
                        const bool last = m || !(halves & 2);
                        auto do_s = [&]() {
                            issue_s(m, m, slot, ends && x == len - 1);
                            if (last) mma_commit(&sm.k_empty[slot]);
                            if (last && x == len - 1) mma_commit(&sm.q_empty);
                        };
                        const bool early = s && w_p != m;
#pragma unroll 1
                        for (int y = 0; y < 2; ++y) {
                            if (y == (early ? 0 : 1)) {
                                if (s) do_s();
                            } else if (w_p >= 0) {
                                ok = issue_pv(w_p, it + x_p, begun >> w_p & 1, ends && x_p == len - 1, first_p, last_p);
                                if (!ok) break;
                                begun |= 1u << w_p;
                                w_p = -1;
                            }
                        }
                        if (!ok || !s) break;
                        first_p = !(m && (halves & 1));
                        last_p = last;
                        w_p = m;
                        x_p = x;
                    }
                    if (!ok || x == len) break;
                    a0 = a1;
                    a1 = a2;
                    if (!halves) {   // nobody's item (a refused page): its K is let go, and its V in turn
                        mma_commit(&sm.k_empty[slot]);
                        if (x == len - 1) mma_commit(&sm.q_empty);
                        if (!(ok = wait(&sm.v_ok[(it + x) % kOkRing], (it + x) / kOkRing))) break;
                        mma_commit(&sm.v_empty[(it + x) % NV]);
                    }
                }
                it += len;
                if (ok && o_wait) ok = wait(&sm.o_free, wk.seg - 1);   // a segment without units
            }
            mma_commit(&sm.drain);
            mbar_wait(&sm.drain, 0, err, nullptr);
        }
    } else if (warp < 4) {
        // ------------------------------------------------------------ Q loads (warp 2), finite check of V
        const int th = tid - 64;
        int it = 0, loads = 0;
        bool ok = true;
        while (ok && wk.next()) {
            if (warp == 2) {
                bool free_q = true;
                if (lane == 0 && wk.seg > 0) free_q = mbar_wait(&sm.q_empty, (wk.seg - 1) & 1, err, &sm.abort);
                if (__shfl_sync(0xffffffffu, free_q, 0)) {
                    const int nt = wk.t.nodes, g = wk.tile % G;
                    if (lane == 0)
                        mbar_arrive_expect_tx(&sm.q_full, wk.sorted ? nt * (HPG * D * 2) : (nt > NPM ? 2 : 1) * (128 * D * 2));
                    __syncwarp();
                    if (wk.sorted) {   // (HPG = 8) a node's heads are a whole 1024-byte swizzle atom: a box for each node
                        if (lane < nt) {
                            const int row = wk.t.row0 + order[wk.t.ord + lane];
#pragma unroll
                            for (int c = 0; c < NSUB; ++c)
                                tma_load_3d(sm.q[lane / NPM] + c * 16384 + (lane % NPM) * (HPG * 128), &qnode, &sm.q_full,
                                            c * 64, g * HPG, row);
                        }
                    } else if (lane < (nt > NPM ? 2 : 1)) {   // nodes in their own order: one box of 128 rows
                        const int row = wk.t.row0 + wk.t.ord % kTreeMaxNodes + lane * NPM;
#pragma unroll
                        for (int c = 0; c < NSUB; ++c)
                            tma_load_3d(sm.q[lane] + c * 16384, &qmap, &sm.q_full, c * 64, g * HPG, row);
                    }
                    ++loads;
                }
            }
            __syncwarp();
            for (int i = wk.off; i < wk.end; ++i, ++it) {
                const bool draft = wk.drafts && i == wk.n_items - 1;
                const int slot = it % NV;
                if (!__all_sync(0xffffffffu, mbar_wait(&sm.v_full[slot], (it / NV) & 1, err, &sm.abort))) {
                    ok = false;
                    break;
                }
                const int per_box = draft ? 512 : 1024;   // 16-byte chunks of a box
                uint32_t acc = 0;
#pragma unroll
                for (int c = 0; c < NSUB; ++c) {
                    const uint4 *box = reinterpret_cast<const uint4 *>(sm.v[slot] + c * 16384);
#pragma unroll 8
                    for (int k = th; k < per_box; k += 64) {
                        const uint4 v = box[k];
                        acc |= exp_all_ones(v.x) | exp_all_ones(v.y) | exp_all_ones(v.z) | exp_all_ones(v.w);
                    }
                }
                if (acc) {
                    const int n_tok = items[size_t(wk.tile) * cap + i].n_tok;
                    for (int c = 0; c < NSUB; ++c) {
                        uint32_t *box = reinterpret_cast<uint32_t *>(sm.v[slot] + c * 16384);
                        for (int k = th; k < per_box; k += 64)
                            for (int e = 0; e < 4; ++e) {
                                const uint32_t v = box[4 * k + e], hit = exp_all_ones(v);
                                if (!hit) continue;
                                box[4 * k + e] = v & ~((hit >> 15) * 0xffffu);
                                if (k / 8 < n_tok) sm.nonfinite = 1;   // 8 chunks of a box per token
                            }
                    }
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.v_ok[it % kOkRing]);
            }
        }
        if (loads && sm.abort) mbar_wait(&sm.q_full, (loads - 1) & 1, err, nullptr);   // lands before the CTA exits
    } else {
        // ------------------------------------------------------------ softmax groups (warps 4-11)
        const int w = (warp - 4) >> 2;
        const int quad = warp & 3;                 // TMEM lanes this warp may access
        const int row = quad * 32 + lane;
        const uint32_t lane_off = uint32_t(quad * 32) << 16;
        const uint32_t t_s = tmem + lane_off + uint32_t(w * 128);
        const uint32_t t_o = tmem + lane_off + 256u;   // + group * D
        const float scale = sm_scale * kLog2e;
        int units = 0;                             // units of this group so far
        bool ok = true;   // once a wait has run out the groups only keep in step, so that no barrier is missed
        while (wk.next()) {
            const int g = wk.tile % G, nt = wk.t.nodes;
            const int nm = nt > NPM ? 2 : 1;
            const Item *list = items + size_t(wk.tile) * cap;
            const int mt = nm == 2 ? w : 0;
            const int node = mt * NPM + row / HPG;                 // within the tile
            const bool live = node < nt;
            const bool warp_live = mt * NPM + quad * 32 / HPG < nt;
            auto row_of = [&]() { return wk.t.row0 + int(order[wk.t.ord + node]); };   // of a live row
            auto drafts_seen = [&]() { return live ? dmask[size_t(row_of()) * G + g] : 0ull; };
            float m = -INFINITY, l = 0.f;
            int mine_n = 0;
            // This group's items: every second one, or (nm == 2) those that a node of its rows selected, found 32 at a time.
            uint32_t todo = 0;
            int base = wk.off - 32;
            auto step = [&](int i) -> int {
                if (nm == 1) return i < 0 ? wk.off + w : i + 2;
                while (!todo) {
                    base += 32;
                    if (base >= wk.end) return wk.end;
                    const int x = base + lane;
                    todo = __ballot_sync(0xffffffffu, x < wk.end && (half_bits<HPG>(list[min(x, wk.end - 1)]) >> mt & 1));
                }
                const int x = base + __ffs(todo) - 1;
                todo &= todo - 1;
                return x;
            };
            int i_next = step(-1);
            int tok_next = 0;        // its cached tokens and the nodes that selected it, one item ahead
            uint32_t nodes_next = 0;
            auto fetch = [&]() {
                if (i_next >= wk.end) return;
                tok_next = list[i_next].n_tok;
                nodes_next = list[i_next].nodes[HPG == 4 ? mt : 0];
            };
            fetch();
            while (ok && i_next < wk.end) {
                const int i = i_next, n_tok = tok_next;
                const bool sees = live && (nodes_next >> (node & 31) & 1);
                i_next = step(i);
                fetch();
                const bool draft = wk.drafts && i == wk.n_items - 1;
                const unsigned long long dm = draft ? drafts_seen() : 0ull;
                // the tokens of 32 columns from c on that this row sees
                auto seen = [&](int c) -> uint32_t {
                    if (draft) return c < 64 ? uint32_t(dm >> c) : 0u;
                    if (!sees || n_tok <= c) return 0u;
                    return n_tok - c >= 32 ? ~0u : (1u << (n_tok - c)) - 1u;
                };
                const int k = units + mine_n;
                ++mine_n;
                if (!__all_sync(0xffffffffu, mbar_wait(&sm.s_full[w], k & 1, err, &sm.abort))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (warp_live) {
                    const int cols = draft ? 64 : 128;
                    uint64_t acc2[4] = {0, 0, 0, 0};
                    bool done = false;
                    const bool any = __any_sync(0xffffffffu, sees);
                    if (!any) {
                        const uint32_t z[16] = {};
                        for (int c = 0; c < cols; c += 32) tmem_st16(t_s + uint32_t(c >> 1), z);
                        done = true;
                    } else if (!draft && n_tok == 128) {
                        // A whole block.  A row without a reference takes the maximum of its first 32 tokens for one;
                        // no other maximum is taken (a sum past 2^kRaise tells that a logit may be far above the
                        // reference; S is still whole then, and the loop below starts over).  P stays in
                        // registers until the end, so that nothing waits between the chunks and the loads run ahead.
                        uint32_t u[4][32], p[4][16];
                        uint64_t sum[4] = {0, 0, 0, 0};
                        uint64_t nm2;
                        const uint64_t scale2 = dup2(scale);
                        auto chunk = [&](int i) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                float pa, pb;
                                ffma2(pa, pb, __uint_as_float(u[i][2 * e]), __uint_as_float(u[i][2 * e + 1]), scale2, nm2);
                                pa = fast_exp2(pa);
                                pb = fast_exp2(pb);
                                fadd2_acc(sum[e & 3], pa, pb);
                                p[i][e] = pack_bf16x2(pa, pb);
                            }
                        };
                        tmem_ld32(t_s, u[0]);
                        tmem_ld32(t_s + 32u, u[1]);
                        tmem_ld_wait();
                        bool based = !__any_sync(0xffffffffu, sees && m == -INFINITY);
                        if (!based) {
                            float a[4];
#pragma unroll
                            for (int x = 0; x < 4; ++x) a[x] = __uint_as_float(u[0][x]);
#pragma unroll
                            for (int e = 4; e < 28; e += 8)
#pragma unroll
                                for (int x = 0; x < 4; ++x)
                                    a[x] = fmax3(a[x], __uint_as_float(u[0][e + x]), __uint_as_float(u[0][e + 4 + x]));
#pragma unroll
                            for (int x = 0; x < 4; ++x) a[x] = fmaxf(a[x], __uint_as_float(u[0][28 + x]));
                            const float top = fmaxf(fmax3(a[0], a[1], a[2]), a[3]) * scale;
                            if (sees && m == -INFINITY && top > m) m = ceilf(top);
                            based = !__any_sync(0xffffffffu, sees && m == -INFINITY);
                        }
                        // Where a row's first 32 logits are all -inf or NaN it has no reference yet, and the loop below
                        // takes the block: it sets one at the first chunk that has a maximum.
                        if (based) {
                            tmem_ld32(t_s + 64u, u[2]);
                            nm2 = dup2(m == -INFINITY ? 0.f : -m);
                            chunk(0);
                            tmem_ld_wait();
                            tmem_ld32(t_s + 96u, u[3]);
                            chunk(1);
                            chunk(2);
                            tmem_ld_wait();
                            chunk(3);
                            const float add = (sum2(sum[0]) + sum2(sum[1])) + (sum2(sum[2]) + sum2(sum[3]));
                            done = !__any_sync(0xffffffffu, sees && add > kRaiseSum);
                            if (done) {
                                if (!__all_sync(0xffffffffu, sees)) {
#pragma unroll
                                    for (int i = 0; i < 4; ++i)
#pragma unroll
                                        for (int e = 0; e < 16; ++e) p[i][e] = sees ? p[i][e] : 0u;
                                }
                                if (sees) l += add;
#pragma unroll
                                for (int i = 0; i < 4; ++i) tmem_st16(t_s + uint32_t(16 * i), p[i]);
                            }
                        }
                    }
#pragma unroll 1
                    for (int c = done ? cols : 0; c < cols; c += 32) {
                        const uint32_t see = seen(c);
                        uint32_t p[16];
                        if (!__any_sync(0xffffffffu, see)) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) p[e] = 0u;
                            tmem_st16(t_s + uint32_t(c >> 1), p);
                            continue;
                        }
                        uint32_t u[32];
                        tmem_ld32(t_s + uint32_t(c), u);
                        tmem_ld_wait();
                        float v[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(u[e]);
                        if (!__all_sync(0xffffffffu, see == ~0u)) {
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] = see >> e & 1 ? v[e] : -INFINITY;
                        }
                        float a[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x) a[x] = fmaxf(v[x], v[4 + x]);
#pragma unroll
                        for (int e = 8; e < 32; e += 8)
#pragma unroll
                            for (int x = 0; x < 4; ++x) a[x] = fmax3(a[x], v[e + x], v[e + 4 + x]);
                        const float top = fmaxf(fmax3(a[0], a[1], a[2]), a[3]) * scale;   // -inf: nothing seen here
                        if (__any_sync(0xffffffffu, top > m + kRaise || (m == -INFINITY && top > m))) {
                            // a row's first tokens (its O and P are 0 so far), or a logit far above its reference
                            const bool up = top > m + kRaise || (m == -INFINITY && top > m);
                            const float fac = up && m != -INFINITY ? fast_exp2(m - ceilf(top)) : 1.f;
                            if (up) m = ceilf(top);
                            if (__any_sync(0xffffffffu, fac != 1.f)) {
                                l *= fac;
#pragma unroll
                                for (int x = 0; x < 4; ++x) {
                                    l += sum2(acc2[x]) * fac;
                                    acc2[x] = 0;
                                }
                                if (mine_n > 1) {
                                    if (!__all_sync(0xffffffffu, mbar_wait(&sm.o_done[w], (k - 1) & 1, err, &sm.abort))) {
                                        ok = false;
                                        break;
                                    }
                                    tc_fence_after();
#pragma unroll 1
                                    for (int d = 0; d < D; d += 16) {
                                        uint32_t x[16];
                                        tmem_ld16(t_o + uint32_t(w * D + d), x);
                                        tmem_ld_wait();
#pragma unroll
                                        for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * fac);
                                        tmem_st16(t_o + uint32_t(w * D + d), x);
                                    }
                                }
                                tmem_st_wait();   // the rounds before may still be storing it
#pragma unroll 1
                                for (int d = 0; d < (c >> 1); d += 16) {   // this item's P so far
                                    uint32_t x[16];
                                    tmem_ld16(t_s + uint32_t(d), x);
                                    tmem_ld_wait();
#pragma unroll
                                    for (int e = 0; e < 16; ++e) x[e] = pack_bf16x2(bf16_lo(x[e]) * fac, bf16_hi(x[e]) * fac);
                                    tmem_st16(t_s + uint32_t(d), x);
                                }
                                tmem_st_wait();
                            }
                        }
                        const uint64_t scale2 = dup2(scale), nm2 = dup2(m == -INFINITY ? 0.f : -m);
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float pa, pb;
                            ffma2(pa, pb, v[2 * e], v[2 * e + 1], scale2, nm2);
                            pa = fast_exp2(pa);
                            pb = fast_exp2(pb);
                            fadd2_acc(acc2[e & 3], pa, pb);
                            p[e] = pack_bf16x2(pa, pb);
                        }
                        tmem_st16(t_s + uint32_t(c >> 1), p);
                    }
                    l += (sum2(acc2[0]) + sum2(acc2[1])) + (sum2(acc2[2]) + sum2(acc2[3]));
                    tmem_st_wait();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.p_ready[w]);
            }
            units += mine_n;
            const int n1 = (wk.end - wk.off) / 2;   // the second group's units (nm == 1)
            // its own O is complete; the other group's is, once the groups have met
            ok = __all_sync(0xffffffffu, ok && (mine_n == 0 || mbar_wait(&sm.o_done[w], (units - 1) & 1, err, &sm.abort)));
            tc_fence_before();
            // The segment's (max, sum) of the row and the weights of the two O's.
            float wa = 1.f, wb = 0.f;      // of O0 and O1 (nm == 1), or of the group's own O (nm == 2)
            if (nm == 1) {
                if (w == 1) sm.join[row] = make_float2(m, l);
                groups_sync();
                if (w == 0) {
                    const float2 o = sm.join[row];
                    const float top = fmaxf(m, o.x);
                    wa = m == -INFINITY ? 0.f : fast_exp2(m - top);
                    wb = o.x == -INFINITY ? 0.f : fast_exp2(o.x - top);
                    l = l * wa + o.y * wb;
                    m = top;
                    sm.join[row] = make_float2(wa, wb);
                }
                groups_sync();
                if (w == 1) {
                    const float2 o = sm.join[row];
                    wa = o.x;
                    wb = o.y;
                }
            }
            const bool whole = wk.off == 0 && wk.end == wk.n_items;
            const int c_lo = nm == 2 ? 0 : w * (D / 2), c_hi = nm == 2 ? D : c_lo + D / 2;
            float *slot = part + size_t(2 * cta + (wk.off > 0 ? 0 : 1)) * part_floats(D);
            float2 *slot_ml = reinterpret_cast<float2 *>(slot + 256 * D);
            const size_t orow = (size_t(live ? row_of() : wk.t.row0) * G + g) * HPG + row % HPG;
            if (nm == 1) {                         // group 0's total for group 1
                groups_sync();                     // the weights have been read
                if (w == 0) sm.join[row] = make_float2(m, l);
                groups_sync();
                if (w == 1) {
                    m = sm.join[row].x;
                    l = sm.join[row].y;
                }
            }
            tc_fence_after();
            const bool fix = *reinterpret_cast<volatile int *>(&sm.nonfinite);
            const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
            if (warp_live && ok) {
#pragma unroll 1
                for (int c = c_lo; c < c_hi; c += 32) {
                    __syncwarp();
                    uint32_t va[32];
                    float o[32];
                    if (nm == 2) {
                        tmem_ld32(t_o + uint32_t(w * D + c), va);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = mine_n > 0 ? __uint_as_float(va[e]) : 0.f;
                    } else {
                        tmem_ld32(t_o + uint32_t(c), va);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = wa == 0.f ? 0.f : __uint_as_float(va[e]) * wa;
                        if (n1 > 0) {
                            tmem_ld32(t_o + uint32_t(D + c), va);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                o[e] = wb == 0.f ? o[e] : fmaf(__uint_as_float(va[e]), wb, o[e]);
                        }
                    }
                    if (fix && live) {
                        const unsigned long long dm = wk.drafts ? drafts_seen() : 0ull;
                        // values that are not finite were taken out of V: p * v of those this row sees
                        for (int i = wk.off; i < wk.end; ++i) {
                            const Item item = list[i];
                            const bool draft = wk.drafts && i == wk.n_items - 1;
                            if (!(item.nodes[node >> 5] >> (node & 31) & 1)) continue;
                            for (int tok = 0; tok < item.n_tok; ++tok) {
                                if (draft && !(dm >> tok & 1)) continue;
                                const size_t at = draft ? (size_t(wk.t.row0 + tok) * G + g) * D
                                                        : ((size_t(item.page) * 128 + tok) * G + g) * D;
                                const uint4 *v4 = reinterpret_cast<const uint4 *>((draft ? v_new : v_cache) + at + c);
                                const uint4 x[4] = {v4[0], v4[1], v4[2], v4[3]};
                                uint32_t any = 0;
#pragma unroll
                                for (int y = 0; y < 4; ++y)
                                    any |= exp_all_ones(x[y].x) | exp_all_ones(x[y].y) | exp_all_ones(x[y].z) |
                                           exp_all_ones(x[y].w);
                                if (!any) continue;
                                const uint16_t *kr = (draft ? k_new : k_cache) + at, *qr = q + orow * D;
                                float s = 0.f;
                                for (int d = 0; d < D; ++d) s = fmaf(bf16_lo(qr[d]), bf16_lo(kr[d]), s);
                                const float p = fast_exp2(fmaf(s, scale, -m));
#pragma unroll
                                for (int e = 0; e < 32; ++e) {
                                    const uint4 &y = x[e >> 3];
                                    const uint32_t word = (e >> 1 & 3) == 0   ? y.x
                                                          : (e >> 1 & 3) == 1 ? y.y
                                                          : (e >> 1 & 3) == 2 ? y.z
                                                                              : y.w;
                                    const float val = e & 1 ? bf16_hi(word) : bf16_lo(word);
                                    if (isinf(val) || isnan(val)) o[e] = fmaf(p, val, o[e]);
                                }
                            }
                        }
                    }
                    if (whole) {
                        if (live) {
#pragma unroll
                            for (int e = 0; e < 32; e += 8)
                                *reinterpret_cast<uint4 *>(out + orow * D + c + e) =
                                    make_uint4(pack_bf16x2(o[e] * inv, o[e + 1] * inv),
                                               pack_bf16x2(o[e + 2] * inv, o[e + 3] * inv),
                                               pack_bf16x2(o[e + 4] * inv, o[e + 5] * inv),
                                               pack_bf16x2(o[e + 6] * inv, o[e + 7] * inv));
                        }
                    } else {
                        // partial: 16-byte chunks, rows innermost, so that a warp stores whole lines
                        float4 *po = reinterpret_cast<float4 *>(slot) + size_t(mt * (D / 4) + c / 4) * 128 + row;
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            po[size_t(e / 4) * 128] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    }
                }
                if (nm == 2 || w == 0) {
                    if (!whole) slot_ml[mt * 128 + row] = make_float2(m, l);
                    else if (live) lse[orow] = l > 0.f || l != l ? (m + log2f(l)) * kLn2 : -INFINITY;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.o_free);
            if (!whole && wk.off == 0 && tid == 4 * 32)   // the ranges that hold the tile
                for (int h = 0; h < nm; ++h)
                    cut[atomicAdd(n_cut, 1)] = Cut{cta, range_owner(wk.x + extra + wk.n_items - 1, total, C), h, g,
                                                   wk.t.row0, nt - h * NPM, wk.t.ord + h * NPM, 0};
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ join
//
// The partials of a cut tile: O = sum_c 2^(m_c - m) O_c / sum_c 2^(m_c - m) l_c over its ranges c.  A CTA has 128
// rows of a tile and 16 columns at a time, one thread per row and 8 columns, with four ranges' loads in
// flight: latency bounds it.  The list of cut tiles is in no order; the results do not depend on it.
template <int D, int HPG>
__global__ void __launch_bounds__(256, 3) k_tree_join(const Cut *__restrict__ cut, const int32_t *__restrict__ n_cut,
                                                      const uint8_t *__restrict__ order,
                                                      const float *__restrict__ part, int G,
                                                      uint16_t *__restrict__ out, float *__restrict__ lse) {
    constexpr int SLABS = D / 16;
    const int r = threadIdx.x & 127;
    pdl_wait();
    const int tasks = *n_cut * SLABS;
    for (int task = blockIdx.x; task < tasks; task += gridDim.x) {
        const int4 *cv = reinterpret_cast<const int4 *>(cut + task / SLABS);
        const int4 c0v = cv[0], c1v = cv[1];
        const int first = c0v.x, last = c0v.y, half = c0v.z;
        const int node = r / HPG, col = task % SLABS * 16 + (threadIdx.x >> 7) * 8;
        if (node >= c1v.y) continue;
        float m = -INFINITY, l = 0.f, o[8] = {};
        for (int c0 = first; c0 <= last; c0 += 4) {
            float2 ml[4];
            float4 v[4][2];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = min(c0 + i, last);
                // a tile's first range left it in its second slot, the others in their first
                const float *p = part + size_t(2 * c + (c == first)) * part_floats(D);
                ml[i] = __ldcg(reinterpret_cast<const float2 *>(p + 256 * D) + half * 128 + r);
                const float4 *po = reinterpret_cast<const float4 *>(p) + size_t(half * (D / 4) + col / 4) * 128 + r;
                if (c0 + i <= last) {
                    v[i][0] = __ldcg(po);
                    v[i][1] = __ldcg(po + 128);
                } else {
                    ml[i] = make_float2(-INFINITY, 0.f);
                }
            }
            float top = m;
#pragma unroll
            for (int i = 0; i < 4; ++i) top = fmaxf(top, ml[i].x);
            const float nt = top == -INFINITY ? 0.f : -top;
            const float f = fast_exp2(m + nt);
            m = top;
            l *= f;
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] *= f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float w = fast_exp2(ml[i].x + nt);
                l = fmaf(ml[i].y, w, l);
                if (ml[i].x == -INFINITY) continue;   // nothing seen there (its O may hold anything)
                o[0] = fmaf(w, v[i][0].x, o[0]);
                o[1] = fmaf(w, v[i][0].y, o[1]);
                o[2] = fmaf(w, v[i][0].z, o[2]);
                o[3] = fmaf(w, v[i][0].w, o[3]);
                o[4] = fmaf(w, v[i][1].x, o[4]);
                o[5] = fmaf(w, v[i][1].y, o[5]);
                o[6] = fmaf(w, v[i][1].z, o[6]);
                o[7] = fmaf(w, v[i][1].w, o[7]);
            }
        }
        const bool any = l > 0.f || l != l;
        const float rcp = any ? 1.f / l : 0.f;
        const size_t orow = (size_t(c1v.x + order[c1v.z + node]) * G + c0v.w) * HPG + r % HPG;
        *reinterpret_cast<uint4 *>(out + orow * D + col) =
            make_uint4(pack_bf16x2(o[0] * rcp, o[1] * rcp), pack_bf16x2(o[2] * rcp, o[3] * rcp),
                       pack_bf16x2(o[4] * rcp, o[5] * rcp), pack_bf16x2(o[6] * rcp, o[7] * rcp));
        if (col == 0) lse[orow] = any ? (m + log2f(l)) * kLn2 : -INFINITY;
    }
}

template <int D, int HPG>
cudaError_t launch_t(const void *q, const void *k_cache, const void *v_cache, const void *k_new, const void *v_new,
                     const int32_t *bt, const int32_t *ctx, const int32_t *node_off, const uint64_t *anc,
                     const int32_t *sel, int n_rows, int n_req, int n_pages, const Shape &s, void *out, float *lse,
                     void *ws, int32_t *err, cudaStream_t st) {
    const Layout w = layout(n_rows, n_req, s);
    if (w.tiles * (w.cap + kTileCost) > 0x3fffffffLL) return cudaErrorNotSupported;
    alignas(64) CUtensorMap qm, qn, km, vm, kn, vn;
    const char *why = nullptr;
    {
        const uint64_t dims[3] = {uint64_t(D), uint64_t(s.Hq), uint64_t(n_rows)};
        const uint64_t strides[2] = {uint64_t(D) * 2, uint64_t(s.Hq) * D * 2};
        const uint32_t box[3] = {64u, uint32_t(HPG), uint32_t(128 / HPG)}, one[3] = {64u, uint32_t(HPG), 1u};
        if (!encode_tensor_map(&qm, 3, q, dims, strides, box, 128, &why)) return cudaErrorInvalidValue;
        if (!encode_tensor_map(&qn, 3, q, dims, strides, one, 128, &why)) return cudaErrorInvalidValue;
    }
    {
        const uint64_t dims[4] = {uint64_t(D), uint64_t(s.G), 128ull, uint64_t(n_pages)};
        const uint64_t strides[3] = {uint64_t(D) * 2, uint64_t(s.G) * D * 2, 128ull * s.G * D * 2};
        const uint32_t box[4] = {64u, 1u, 128u, 1u};
        if (!encode_tensor_map(&km, 4, k_cache, dims, strides, box, 128, &why)) return cudaErrorInvalidValue;
        if (!encode_tensor_map(&vm, 4, v_cache, dims, strides, box, 128, &why)) return cudaErrorInvalidValue;
    }
    {
        const uint64_t dims[3] = {uint64_t(D), uint64_t(s.G), uint64_t(n_rows)};
        const uint64_t strides[2] = {uint64_t(D) * 2, uint64_t(s.G) * D * 2};
        const uint32_t box[3] = {64u, 1u, 64u};
        if (!encode_tensor_map(&kn, 3, k_new, dims, strides, box, 128, &why)) return cudaErrorInvalidValue;
        if (!encode_tensor_map(&vn, 3, v_new, dims, strides, box, 128, &why)) return cudaErrorInvalidValue;
    }
    uint8_t *base = static_cast<uint8_t *>(ws);
    Tile *tiles = reinterpret_cast<Tile *>(base + w.tile);
    Cut *cut = reinterpret_cast<Cut *>(base + w.cut);
    int32_t *n_cut = reinterpret_cast<int32_t *>(base + w.n_cut);
    uint8_t *order = base + w.order;
    auto *dmask = reinterpret_cast<unsigned long long *>(base + w.dmask);
    Item *items = reinterpret_cast<Item *>(base + w.items);
    float *part = reinterpret_cast<float *>(base + w.part);
    cudaError_t e = launch_kernel(k_tree_plan<D, HPG>, dim3(unsigned(n_req) * unsigned(s.G)), dim3(kPlanThreads), 0, st, true, sel, bt,
                                  ctx, node_off, anc, n_rows, n_pages, s.G, s.topk, s.max_blocks, w.chunks, w.cap,
                                  tiles, n_cut, order, dmask, items, static_cast<uint4 *>(out), lse, err);
    if (e != cudaSuccess) return e;
    const size_t smem = sizeof(TreeSmem<D>) + 1024;
    static_assert(sizeof(TreeSmem<D>) + 1024 <= 232448, "shared memory of a CTA");
    e = cudaFuncSetAttribute(k_attn_tree<D, HPG>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    const int grid = std::min(sm_count(), kMaxCtas);
    e = launch_kernel(k_attn_tree<D, HPG>, dim3(unsigned(grid)), dim3(kThreads), smem, st, true,
                      static_cast<const uint16_t *>(q), qm, qn, km, vm, kn, vn, static_cast<const uint16_t *>(k_cache),
                      static_cast<const uint16_t *>(v_cache), static_cast<const uint16_t *>(k_new),
                      static_cast<const uint16_t *>(v_new), s.G, w.cap, int(w.tiles), s.sm_scale,
                      static_cast<const uint8_t *>(order), static_cast<const Tile *>(tiles), cut, n_cut, static_cast<const unsigned long long *>(dmask),
                      static_cast<const Item *>(items), part, static_cast<uint16_t *>(out), lse, err);
    if (e != cudaSuccess) return e;
    return launch_kernel(k_tree_join<D, HPG>, dim3(unsigned(4 * grid)), dim3(256), 0, st, true, static_cast<const Cut *>(cut),
                         static_cast<const int32_t *>(n_cut), static_cast<const uint8_t *>(order),
                         static_cast<const float *>(part), s.G, static_cast<uint16_t *>(out), lse);
}

}  // namespace

size_t tree_workspace_bytes(int n_rows, int n_req, const Shape &s) { return layout(n_rows, n_req, s).bytes; }

cudaError_t launch_attn_tree(const void *q, const void *k_cache, const void *v_cache, const void *k_new,
                             const void *v_new, const int32_t *block_table, const int32_t *ctx_lens,
                             const int32_t *node_off, const uint64_t *anc, const int32_t *sel, int n_rows, int n_req,
                             int n_pages, const Shape &s, void *out, float *lse, void *ws, int32_t *err,
                             cudaStream_t st) {
#define MSA_AT_CASE(DD, HH)                                                                                      \
    if (s.D == DD && s.hpg == HH)                                                                                \
        return launch_t<DD, HH>(q, k_cache, v_cache, k_new, v_new, block_table, ctx_lens, node_off, anc, sel, n_rows, \
                                n_req, n_pages, s, out, lse, ws, err, st);
    MSA_AT_CASE(128, 8) MSA_AT_CASE(128, 4) MSA_AT_CASE(64, 8) MSA_AT_CASE(64, 4)
#undef MSA_AT_CASE
    return cudaErrorNotSupported;
}

}  // namespace msa
