// Verification of drafted trees against the target's probabilities.
//
// With r_c(t) = max(p(t) - c q(t), 0) the residual after any number of rejections is r_c / M, M its
// sum: rejecting a child takes p' to max(p' - q, 0) normalised, i.e. r_c / M to r_{c + M} / M'.  So a
// node's state is two scalars, a test of a child reads two probabilities, and a rejection costs one pass
// over the node's two rows.  The last pass at the last node also holds the sums that the next token
// is found by.
//
// A cluster of up to 8 CTAs has one request, because a single SM would take tens of microseconds for a
// pass over a large vocabulary: each warp of the cluster has a contiguous run of tokens, leaves the
// run's sum in every CTA's shared memory, and after one cluster barrier warp 0 of each CTA goes on with the
// walk by itself, all of them with the same numbers and so the same decisions.  The next token is then
// found in the one run that holds it.
// 32 requests x 131,072 tokens: 39 us, about five passes of 33 MB for the slowest request (a rejection decides the next
// test, so the passes of a request follow one another; a pass is 3 to 5 us of loads, 2 of sums and cluster barrier and 1 of the decision).
// One request of 32,000 tokens: 12 us.
//
// A rounding of a sum moves a border between two tokens, and the residual may be a flat tail of a row whose likely
// token was rejected, so sums have to be good to a small part of themselves, whatever is in the row.  64-bit
// arithmetic runs at 1/64 of the fp32 rate on this GPU and pairs of fp32 numbers for each residual made the
// pass bound by its arithmetic (3.6 us of 131,072 tokens on 8 CTAs).  A residual's mass is A - c B, A and B the sums
// of p and q over the tokens with p > c q, and those are sums of given fp32 numbers that are not negative: each is
// carried as h + l with the exact error of every addition to h added to l, and l is brought below a step of h after
// every four.  Four of a lane's additions then lose at most 14 * 2^-48 of its sum and the join of the lanes 66 * 2^-48,
// so a sum is off by less than (n + 20) 2^-46 of itself with n tokens per half lane, vocab / (1024 * CTAs of the request):
// 2^-40 for 131,072 tokens on 8 CTAs, 2^-38 on one.  Everything from the run sums on is in 64 bits.
#include "msa_device.cuh"
#include "msa_internal.h"

namespace msa {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kInFlight = 8;    // tokens of each row that a thread has in flight

// What warp 0 asks of its CTA.
enum { kPass, kSelect, kDone };

struct Smem {
    unsigned long long kids[kTreeMaxNodes];                       // children of a node, by number
    int tok[kTreeMaxNodes];
    float u[kTreeMaxNodes], p[kTreeMaxNodes], q[kTreeMaxNodes];   // at the node's token in its parent's rows
    int gone[kTreeMaxNodes];                                      // tokens taken out (no draft distribution)
    float4 part[kWarps];                                          // A and B of each warp's run, h and l
    double run[2][kMaxCluster * kWarps];                          // run sums of the cluster, two passes
    double c, before, want;
    int cmd, at, n_gone, slot;
};

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void st_cluster_f64(double *local, uint32_t rank, double v) {
    uint32_t addr;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(local)), "r"(rank));
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(v) : "memory");
}

// Two fp32 lanes per instruction.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// h + l += v in both lanes: the exact error of h + v goes to l.
__device__ __forceinline__ void add_pair(uint64_t &h, uint64_t &l, uint64_t v) {
    const uint64_t s = add2(h, v), w = sub2(s, h);
    l = add2(l, add2(sub2(h, sub2(s, w)), sub2(v, w)));
    h = s;
}
// h takes what of l it can hold.
__device__ __forceinline__ void settle(uint64_t &h, uint64_t &l) {
    const uint64_t s = add2(h, l);
    l = sub2(l, sub2(s, h));
    h = s;
}

struct Residual {
    double c;
    float chi, clo;   // c
    bool draft;
    // whether p - c q > 0 (NaN: no), for q >= 0: entries of q below 0 and NaN count as 0 (fmaxf)
    __device__ __forceinline__ bool positive(float p, float q) const {
        return draft ? fmaf(-clo, q, fmaf(-chi, q, p)) > 0.f : p > 0.f;
    }
    __device__ __forceinline__ double value(float p, float q) const {
        q = fmaxf(q, 0.f);
        if (!positive(p, q)) return 0.0;
        const double r = draft ? double(p) - c * double(q) : double(p);
        return r > 0.0 ? r : 0.0;
    }
};

template <int VEC>
struct Chunk {
    float v[VEC];
    __device__ __forceinline__ void load(const float *__restrict__ row, int t, int vocab) {
        if constexpr (VEC == 4) {
            const float4 x = t < vocab ? __ldg(reinterpret_cast<const float4 *>(row + t)) : make_float4(0.f, 0.f, 0.f, 0.f);
            v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
        } else {
            v[0] = t < vocab ? __ldg(row + t) : 0.f;
        }
    }
};

// VEC = 4: rows are 16-byte aligned (vocab a multiple of 4), a lane has four neighbouring tokens; else one.
template <int VEC>
__global__ void __launch_bounds__(kThreads, 2) k_verify_tree(
    const float *__restrict__ probs, const float *__restrict__ drafts, int vocab, const int32_t *__restrict__ tokens,
    const int32_t *__restrict__ node_off, const int32_t *__restrict__ parents, const float *__restrict__ u_accept,
    const float *__restrict__ u_next, int n_rows, int cluster, int32_t *__restrict__ path,
    int32_t *__restrict__ n_acc, int32_t *__restrict__ next_token, int32_t *err) {
    constexpr int TILE = 32 * VEC;
    __shared__ Smem sm;
    const int b = blockIdx.x / cluster, rank = blockIdx.x % cluster;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int row0;
    const int n = tree_rows_of(node_off, b, n_rows, err, tid == 0 && rank == 0, &row0);
    if (n == 0) {   // the whole cluster
        if (tid == 0 && rank == 0) {
            n_acc[b] = 0;
            next_token[b] = -1;
        }
        return;
    }
    if (tid < n) sm.kids[tid] = 0;
    __syncthreads();
    if (tid < n) {
        const int par = parents[row0 + tid], tok = tokens[row0 + tid];
        const bool ok = tid > 0 && par >= 0 && par < tid && tok >= 0 && tok < vocab;
        if (rank == 0 && (tid == 0 ? par != -1 : !ok)) raise_flag(err, MSA_FLAG_BOUNDS);
        if (ok) {
            sm.tok[tid] = tok;
            sm.u[tid] = u_accept[row0 + tid];
            sm.p[tid] = probs[size_t(row0 + par) * vocab + tok];
            if (drafts) sm.q[tid] = fmaxf(drafts[size_t(row0 + par) * vocab + tok], 0.f);
            atomicOr(&sm.kids[par], 1ull << tid);
        }
        if (rank == 0) path[row0 + tid] = -1;
    }
    const int slots = cluster * kWarps, my_slot = rank * kWarps + warp;
    const int tiles = (vocab + TILE - 1) / TILE;
    const int tile0 = int((long long)my_slot * tiles / slots), tile1 = int((long long)(my_slot + 1) * tiles / slots);
    if (cluster > 1) cluster_sync();   // every CTA of the cluster runs before its shared memory is written
    else __syncthreads();

    // walk state, the same in every lane of warp 0 of every CTA of the cluster
    int at = 0, count = 0, n_gone = 0, buf = 0;
    unsigned long long kids = sm.kids[0];
    double c = 0.0, mass = 1.0;
    bool whole = false;      // the pass is over p itself (nothing is left of the residual)
    bool summed = false;     // sm.run[buf ^ 1] holds the run sums of the state (at, c, gone)
    bool entered = false;    // `at` is in the path
    for (;;) {
        if (warp == 0) {
            int cmd = -1;
            while (cmd < 0) {
                if (!entered) {
                    if (rank == 0 && lane == 0) path[row0 + count] = at;
                    ++count;
                    entered = true;
                }
                if (kids && !whole) {
                    const int x = __ffsll(kids) - 1;
                    kids &= kids - 1;
                    const int tok = sm.tok[x];
                    const float px = sm.p[x], qx = drafts ? sm.q[x] : 1.f, ux = sm.u[x];
                    bool gone = false;
                    if (!drafts)
                        for (int i = 0; i < n_gone; ++i) gone = gone || sm.gone[i] == tok;
                    auto left = [&]() {   // of the token in the residual
                        const double r = double(px) - (drafts ? c * double(qx) : 0.0);
                        return r > 0.0 && !gone ? r : 0.0;
                    };
                    // In fp32 first, whose roundings stay below 2^-21 of the terms, and in 64 bits where that does not
                    // tell (a 64-bit operation is slow here, and the walk is one after another).
                    const float cf = float(c), rf = gone ? 0.f : fmaxf(drafts ? fmaf(-cf, qx, px) : px, 0.f);
                    const float lf = ux * qx * float(mass);
                    const float slack = fmaf(0x1p-20f, fabsf(px) + cf * qx + fabsf(lf), 1e-36f);
                    if (fabsf(lf - rf) > slack ? lf < rf : double(ux) * double(qx) * mass < left()) {
                        at = x;
                        kids = sm.kids[x];
                        c = 0.0;
                        mass = 1.0;
                        n_gone = 0;
                        summed = entered = false;
                    } else if (drafts) {
                        c += mass;
                        cmd = kPass;
                    } else {
                        mass = fmax(mass - left(), 0.0);   // rounding of p may leave less than nothing
                        if (lane == 0) sm.gone[n_gone] = tok;
                        ++n_gone;
                        __syncwarp();
                    }
                } else {
                    cmd = summed ? kSelect : kPass;
                }
            }
            if (cmd == kSelect) {
                // the run in which the running sum passes u * total; four runs per lane
                const double *run = sm.run[buf ^ 1];
                double own[kMaxCluster * kWarps / 32], incl = 0.0;
#pragma unroll
                for (int i = 0; i < kMaxCluster * kWarps / 32; ++i) {
                    const int s = lane * (kMaxCluster * kWarps / 32) + i;
                    own[i] = s < slots ? run[s] : 0.0;
                    incl += own[i];
                }
                double scan = incl;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const double y = __shfl_up_sync(0xffffffffu, scan, o);
                    if (lane >= o) scan += y;
                }
                const double total = __shfl_sync(0xffffffffu, scan, 31);
                if (!(total > 0.0) || isinf(total)) {
                    if (!whole && !(isinf(total))) {   // nothing is left of the residual: p itself
                        whole = true;
                        c = 0.0;
                        n_gone = 0;
                        cmd = kPass;
                    } else {
                        if (rank == 0 && lane == 0) {
                            raise_flag(err, MSA_FLAG_NAN);
                            next_token[b] = -1;
                            n_acc[b] = count;
                        }
                        cmd = kDone;
                    }
                } else {
                    const double want = double(u_next[b]) * total;
                    double end = scan - incl, found_before = 0.0;
                    int found = slots;
#pragma unroll
                    for (int i = 0; i < kMaxCluster * kWarps / 32; ++i) {
                        // the first run whose end passes `want`; an empty run holds no token
                        const double begin = end;
                        end += own[i];
                        if (found == slots && own[i] > 0.0 && end > want) {
                            found = lane * (kMaxCluster * kWarps / 32) + i;
                            found_before = begin;
                        }
                    }
                    const uint32_t hit = __ballot_sync(0xffffffffu, found < slots);
                    if (hit) {
                        const int src = __ffs(hit) - 1;
                        found = __shfl_sync(0xffffffffu, found, src);
                        found_before = __shfl_sync(0xffffffffu, found_before, src);
                    } else {   // rounding left the total short: the last run with mass
                        int last = -1;
#pragma unroll
                        for (int i = 0; i < kMaxCluster * kWarps / 32; ++i)
                            if (own[i] > 0.0) last = lane * (kMaxCluster * kWarps / 32) + i;
                        found = __reduce_max_sync(0xffffffffu, last);
                        found_before = 0.0;
                    }
                    if (rank == 0 && lane == 0) n_acc[b] = count;
                    if (lane == 0) {
                        sm.slot = found;
                        sm.before = found_before;
                        sm.want = hit ? want : INFINITY;
                    }
                }
            }
            if (lane == 0) {
                sm.cmd = cmd;
                sm.at = at;
                sm.c = c;
                sm.n_gone = n_gone;
            }
        }
        __syncthreads();
        const int cmd = sm.cmd;
        if (cmd == kDone) break;
        const float *p = probs + size_t(row0 + sm.at) * vocab;
        const Residual res{sm.c, float(sm.c), float(sm.c - double(float(sm.c))), drafts != nullptr && sm.c != 0.0};
        const float *q = res.draft ? drafts + size_t(row0 + sm.at) * vocab : p;
        const int gone_n = sm.n_gone;
        if (cmd == kSelect) {
            if (sm.slot != my_slot) break;
            // this warp's run holds the token
            double before = sm.before;
            const double want = sm.want;
            int token = -1;
            for (int tile = tile0; tile < tile1 && token < 0; ++tile) {
                const int t = tile * TILE + lane * VEC;
                Chunk<VEC> cp, cq;
                cp.load(p, t, vocab);
                cq.load(q, t, vocab);
                double r[VEC], incl = 0.0;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    r[e] = res.value(cp.v[e], cq.v[e]);
                    for (int i = 0; i < gone_n; ++i)
                        if (sm.gone[i] == t + e) r[e] = 0.0;
                    incl += r[e];
                }
                double scan = incl;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const double y = __shfl_up_sync(0xffffffffu, scan, o);
                    if (lane >= o) scan += y;
                }
                double run = before + (scan - incl);
                int mine = vocab;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    run += r[e];
                    if (mine == vocab && r[e] > 0.0 && run > want) mine = t + e;
                }
                const int first = __reduce_min_sync(0xffffffffu, mine);
                if (first < vocab) token = first;
                before += __shfl_sync(0xffffffffu, scan, 31);
            }
            if (token < 0) {   // rounding: the run's last token with mass
                for (int tile = tile1 - 1; tile >= tile0 && token < 0; --tile) {
                    const int t = tile * TILE + lane * VEC;
                    Chunk<VEC> cp, cq;
                    cp.load(p, t, vocab);
                    cq.load(q, t, vocab);
                    int mine = -1;
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        bool out = false;
                        for (int i = 0; i < gone_n; ++i) out = out || sm.gone[i] == t + e;
                        // (as the pass decided: a run with mass has such a token)
                        if (res.positive(cp.v[e], fmaxf(cq.v[e], 0.f)) && !out) mine = t + e;
                    }
                    token = __reduce_max_sync(0xffffffffu, mine);
                }
            }
            if (lane == 0) next_token[b] = token;
            break;
        }
        // a pass: this warp's run sum, A - c B
        uint64_t ah = 0, al = 0, bh = 0, bl = 0;   // two tokens' sums each
        const uint64_t nchi2 = pack2(-res.chi, -res.chi), nclo2 = pack2(-res.clo, -res.clo);
        constexpr int U = kInFlight / VEC;   // tiles in flight
        for (int tile = tile0; tile < tile1; tile += U) {
            Chunk<VEC> cp[U], cq[U];
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int t = tile + k < tile1 ? (tile + k) * TILE + lane * VEC : vocab;
                cp[k].load(p, t, vocab);
                if (res.draft) cq[k].load(q, t, vocab);
            }
            if (gone_n > 0) {
#pragma unroll
                for (int k = 0; k < U; ++k)
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        for (int i = 0; i < gone_n; ++i)
                            if (sm.gone[i] == (tile + k) * TILE + lane * VEC + e) cp[k].v[e] = 0.f;
            }
#pragma unroll
            for (int x = 0; x < U * VEC; x += 2) {
                const float p0 = cp[x / VEC].v[x % VEC], p1 = cp[(x + 1) / VEC].v[(x + 1) % VEC];
                if (res.draft) {
                    const float q0 = fmaxf(cq[x / VEC].v[x % VEC], 0.f), q1 = fmaxf(cq[(x + 1) / VEC].v[(x + 1) % VEC], 0.f);
                    const uint64_t q2 = pack2(q0, q1);
                    const float2 r = unpack2(fma2(nclo2, q2, fma2(nchi2, q2, pack2(p0, p1))));
                    add_pair(ah, al, pack2(r.x > 0.f ? p0 : 0.f, r.y > 0.f ? p1 : 0.f));
                    add_pair(bh, bl, pack2(r.x > 0.f ? q0 : 0.f, r.y > 0.f ? q1 : 0.f));
                } else {
                    add_pair(ah, al, pack2(fmaxf(p0, 0.f), fmaxf(p1, 0.f)));   // NaN counts as 0
                }
            }
            settle(ah, al);
            if (res.draft) settle(bh, bl);
        }
        // the two halves and the lanes, A beside B
        const float2 a_h = unpack2(ah), a_l = unpack2(al), b_h = unpack2(bh), b_l = unpack2(bl);
        uint64_t h = pack2(a_h.x, b_h.x), l = pack2(a_l.x, b_l.x);
        add_pair(h, l, pack2(a_h.y, b_h.y));
        l = add2(l, pack2(a_l.y, b_l.y));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const uint64_t h_o = __shfl_xor_sync(0xffffffffu, h, o), l_o = __shfl_xor_sync(0xffffffffu, l, o);
            add_pair(h, l, h_o);
            l = add2(l, l_o);
        }
        if (lane == 0) {
            const float2 hs = unpack2(h), ls = unpack2(l);
            sm.part[warp] = make_float4(hs.x, ls.x, hs.y, ls.y);
        }
        __syncthreads();
        // one warp joins them: the SM has two 64-bit operations a cycle, and 16 warps would queue up for them
        if (warp == 0 && lane < kWarps) {
            const float4 v = sm.part[lane];
            double sum = double(v.x) + double(v.y);
            if (res.draft) sum -= res.c * (double(v.z) + double(v.w));
            if (sum < 0.0) sum = 0.0;   // a rounding of nothing (NaN stays)
            if (cluster == 1) sm.run[buf][lane] = sum;
            else
                for (int r = 0; r < cluster; ++r) st_cluster_f64(&sm.run[buf][rank * kWarps + lane], uint32_t(r), sum);
        }
        if (cluster > 1) cluster_sync();
        else __syncthreads();
        buf ^= 1;
        if (warp == 0) {   // the residual's mass
            double own[kMaxCluster * kWarps / 32];
#pragma unroll
            for (int i = 0; i < kMaxCluster * kWarps / 32; ++i)
                own[i] = lane + 32 * i < slots ? sm.run[buf ^ 1][lane + 32 * i] : 0.0;
            double s = (own[0] + own[1]) + (own[2] + own[3]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            mass = s;
            summed = true;
        }
    }
    if (cluster > 1) cluster_sync();   // no CTA ends while another may still write its shared memory
}

template <int VEC>
cudaError_t launch_t(const float *p, const float *q, int vocab, const int32_t *tokens, const int32_t *node_off,
                     const int32_t *parents, const float *u_accept, const float *u_next, int n_rows, int n_req,
                     int cluster, int32_t *path, int32_t *n_acc, int32_t *next_token, int32_t *err, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(n_req) * unsigned(cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(cluster);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_verify_tree<VEC>, p, q, vocab, tokens, node_off, parents, u_accept, u_next, n_rows,
                              cluster, path, n_acc, next_token, err);
}

}  // namespace

cudaError_t launch_verify_tree(const float *p, const float *q, int vocab, const int32_t *tokens,
                               const int32_t *node_off, const int32_t *parents, const float *u_accept,
                               const float *u_next, int n_rows, int n_req, int32_t *path, int32_t *n_acc,
                               int32_t *next_token, int32_t *err, cudaStream_t st) {
    // CTAs per request: enough that a CTA's part of a row is about 4,096 tokens (eight per thread), as long as
    // all of the batch runs at once (two CTAs per SM)
    int cluster = 1;
    while (cluster < kMaxCluster && vocab / cluster > 4096 && 1LL * n_req * cluster <= sm_count()) cluster *= 2;
    const bool vec = vocab % 4 == 0 && ((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(q)) & 15u) == 0;
    return (vec ? launch_t<4> : launch_t<1>)(p, q, vocab, tokens, node_off, parents, u_accept, u_next, n_rows, n_req,
                                             cluster, path, n_acc, next_token, err, st);
}

}  // namespace msa
