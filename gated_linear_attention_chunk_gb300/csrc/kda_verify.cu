// Verification of drafted trees against the target's probabilities, from given uniform numbers.
//
// The walk of one sequence: at the current node (target row p, draft row q) the children are tried
// in index order; child x with number u is accepted if u q_x R < r_x, with the residual
// r = max(0, p - A q), A = 0 and R = 1 before the first refusal, A += R and R = sum r after one.
// That is repeated rejection sampling with the nested residuals max(0, r - R q) folded into one scalar:
// max(0, max(0, a) - b) = max(0, a - b) for b >= 0.  Without draft rows the drafts are certain: accepted if
// u R < r_x, and a refusal takes x out of r.  At the end the next token is drawn from r by inverse CDF.
//
// One cluster of CTAs per sequence.  Everything the walk compares -- parent, token, number, p_x and q_x
// of every node -- is gathered at once, two nodes per lane of one warp; the walk itself then runs in registers and
// touches a whole row only after a refusal (draft rows given) and for the final draw.  Such a pass cuts
// the row into segments of kSegUnit elements (or a multiple), two per warp at a time, and leaves the segments' sums in shared memory,
// where every CTA of the cluster reads them all in the same order; the draw then needs only the one segment that
// holds its point again.  So a sequence costs about one reading of one row (two with draft rows),
// which bounds it: the rest is the latency of the walk's dependent loads.  128 chains of 4 nodes over 131,072 tokens, fp32: 43 us,
// of them 21.7 in the pass (6.2 TB/s) and about 12 in the steps before and after it (the rest is not accounted for); one tree of 6
// nodes over 32,001: 12 to 18 us a call, by how many siblings are tried after a refusal (a pass more for each).  With draft rows
// the 64 registers that four CTAs per SM leave a thread spill 140 bytes (fp32) or 308 (bf16).  Four CTAs of 256 threads per SM keep all sequences
// resident (one of 512 took 100 us, eight per sequence in two rounds 54, two per sequence 48.5).
//
// Precision: the answers are whole numbers, so a rounding shows only next to a border, where a flat
// distribution over 10^5 tokens has one every 10^-5.  p - A q is carried as an unevaluated fp32 pair with
// the error terms of its product and difference, and so are all sums:
// about 1e-13 of the mass, at the cost of about 20 fp32 operations per element (fp64 arithmetic per element would
// be several times slower than the loads).  The order of the sums is fixed and does not depend on the cluster's size.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_spec.cuh"

namespace cg = cooperative_groups;

namespace kda {
namespace {

using namespace spec;

constexpr int kVerThreads = 256;
constexpr int kVerWarps = kVerThreads / 32;
constexpr int kSegUnit = 256;     // elements of a segment (of one step of it, where a row has more than kMaxSegs)
constexpr int kMaxSegs = 512;     // segments of a row
constexpr int kMaxCluster = 8;    // CTAs per sequence
constexpr int kMaxNodes = KDA_MAX_TREE_NODES;

struct VerifyParams {
    const int32_t *tokens, *cu, *parent;
    const void *target, *draft;
    const float *u_accept, *u_sample;
    int64_t T, ts, ds;
    int N, V;
    int nseg, seg_steps;     // segments of a row, kSegUnit-element steps of a segment
    int32_t *cu_accept, *rows, *next_token;
    uint32_t *status;        // [0] status word, [1] ticket of finished sequences, [2] cu falls somewhere
    uint64_t *accepted;      // [N] accepted nodes as bits; if cu falls, before that whether the sequence begins below an earlier entry
};

// Unevaluated sum of two floats, hi + lo.
struct Pair {
    float hi, lo;
};
__device__ __forceinline__ void add(Pair &a, float hi, float lo) {
    const float s = __fadd_rn(a.hi, hi);
    const float b = __fsub_rn(s, a.hi);
    const float e = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, b)), __fsub_rn(hi, b));
    a.hi = s;
    a.lo = __fadd_rn(a.lo, __fadd_rn(e, lo));
}
// max(0, p - (ah + al) q) as a pair; NaN gives 0.
__device__ __forceinline__ Pair residual(float p, float q, float ah, float al) {
    const float m = __fmul_rn(ah, q);
    const float me = __fmaf_rn(al, q, __fmaf_rn(ah, q, -m));
    const float s = __fsub_rn(p, m);
    const float b = __fsub_rn(s, p);
    const float e = __fsub_rn(__fsub_rn(__fsub_rn(p, __fsub_rn(s, b)), __fadd_rn(m, b)), me);
    const float hi = __fadd_rn(s, e);
    const float lo = __fsub_rn(e, __fsub_rn(hi, s));
    return hi > 0.f ? Pair{hi, lo} : Pair{0.f, 0.f};
}

// A row at any alignment: element e lies at base[e]; a step of a warp covers kSegUnit elements from
// element `e0`, a multiple of kSegUnit before which `shift` elements were moved to the step before so that
// 16-byte loads are aligned.
template <typename T>
struct Row {
    const T *base;
    bool vec;  // base - shift is 16-byte aligned
};

template <typename T>
__device__ __forceinline__ void load_vec(const Row<T> &r, int64_t e, int V, float (&f)[Elem<T>::kVec]) {
    constexpr int W = Elem<T>::kVec;
    if (r.vec && e >= 0 && e + W <= V) {
        unpack16(__ldg(reinterpret_cast<const uint4 *>(r.base + e)), f);
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) f[i] = e + i >= 0 && e + i < V ? Elem<T>::to_f(r.base[e + i]) : 0.f;
    }
}

// Refused certain drafts (two per lane): takes their mass out of the elements e0 + (i * 32 + lane) * W + w of a step.
template <int L, int W>
__device__ __forceinline__ void take_out(float (&v)[L][W], int64_t e0, const int (&gone)[2]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        const int64_t off = gone[g] - e0;
        for (uint32_t hit = __ballot_sync(0xffffffffu, gone[g] >= 0 && off >= 0 && off < L * W * 32); hit; hit &= hit - 1) {
            const int x = __shfl_sync(0xffffffffu, static_cast<int>(off), __ffs(hit) - 1);
#pragma unroll
            for (int i = 0; i < L; ++i)
#pragma unroll
                for (int w = 0; w < W; ++w)
                    if (x == (i * 32 + lane) * W + w) v[i][w] = 0.f;
        }
    }
}

// Sums of the residual over two neighbouring segments by one warp: the first in lane 0, the second in lane 16.  Lanes
// and warps are joined in pairs of fp32 as well: fp64 additions here would take longer than the loads.
template <typename T, bool kDraft>
__device__ __forceinline__ Pair segment_sums(const Row<T> &p, const Row<T> &q, bool use_q, int shift, int V, int64_t first,
                                               int steps, double A, const int (&gone)[2]) {
    constexpr int W = Elem<T>::kVec, L = kSegUnit / 32 / W;  // vectors per lane, segment and step
    const int lane = threadIdx.x & 31;
    const float ah = static_cast<float>(A), al = static_cast<float>(A - static_cast<double>(ah));
    Pair acc[2] = {{0.f, 0.f}, {0.f, 0.f}};
    for (int s = 0; s < steps; ++s) {
        float pv[2][L][W], qv[2][kDraft ? L : 1][W];
        int64_t e0[2];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            e0[g] = first + static_cast<int64_t>(g * steps + s) * kSegUnit;
#pragma unroll
            for (int i = 0; i < L; ++i) load_vec(p, e0[g] + (i * 32 + lane) * W, V, pv[g][i]);
            if (kDraft && use_q) {
#pragma unroll
                for (int i = 0; i < L; ++i) load_vec(q, e0[g] + (i * 32 + lane) * W, V, qv[g][kDraft ? i : 0]);
            }
        }
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            if (!kDraft) take_out(pv[g], e0[g], gone);
#pragma unroll
            for (int i = 0; i < L; ++i)
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    if (kDraft && use_q) {
                        const Pair r = residual(pv[g][i][w], qv[g][kDraft ? i : 0][w], ah, al);
                        add(acc[g], r.hi, r.lo);
                    } else {
                        add(acc[g], pv[g][i][w] > 0.f ? pv[g][i][w] : 0.f, 0.f);
                    }
                }
        }
    }
    const bool low = lane < 16;
    Pair mine = low ? acc[0] : acc[1];
    const Pair give = low ? acc[1] : acc[0];
    add(mine, __shfl_xor_sync(0xffffffffu, give.hi, 16), __shfl_xor_sync(0xffffffffu, give.lo, 16));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
        const float hi = __shfl_xor_sync(0xffffffffu, mine.hi, o), lo = __shfl_xor_sync(0xffffffffu, mine.lo, o);
        add(mine, hi, lo);
    }
    return mine;
}

__device__ __forceinline__ Pair warp_scan(Pair x) {  // inclusive, in lane order
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float hi = __shfl_up_sync(0xffffffffu, x.hi, o), lo = __shfl_up_sync(0xffffffffu, x.lo, o);
        if (lane >= o) add(x, hi, lo);
    }
    return x;
}
__device__ __forceinline__ double value(Pair x) { return static_cast<double>(x.hi) + static_cast<double>(x.lo); }
__device__ __forceinline__ Pair from_lane(Pair x, int lane) {
    return Pair{__shfl_sync(0xffffffffu, x.hi, lane), __shfl_sync(0xffffffffu, x.lo, lane)};
}

// Where a running sum passes a point: of one weight per lane, in lane order, the first lane whose sum, `before`
// included, is above `point` (`before` becomes the sum ahead of it); otherwise hit is false, the last lane with mass or -1
// is returned, and `before` becomes the sum of all.
__device__ __noinline__ int pass_point(Pair weight, double &before, double point, bool &hit) {
    const Pair upto = warp_scan(weight);
    const double sum = before + value(upto);
    const uint32_t over = __ballot_sync(0xffffffffu, weight.hi > 0.f && sum > point);
    const uint32_t some = __ballot_sync(0xffffffffu, weight.hi > 0.f);
    hit = over != 0;
    const int at = over ? __ffs(over) - 1 : some ? 31 - __clz(some) : -1;
    const double own = value(weight);
    if (hit) before = __shfl_sync(0xffffffffu, sum - own, at);
    else before = __shfl_sync(0xffffffffu, sum, 31);
    return at;
}

// The element of the steps [s0, s1) at which the running sum passes `point` (as pass_point).  By one warp: first the
// run of kRun consecutive elements, then the element, one per lane.
template <typename T, bool kDraft>
__device__ __forceinline__ int segment_find(const Row<T> &p, const Row<T> &q, bool use_q, int shift, int V, int64_t s0, int64_t s1,
                                            double A, const int (&gone)[2], double before, double point) {
    constexpr int W = Elem<T>::kVec, kRun = kSegUnit / 32;
    const int lane = threadIdx.x & 31;
    const float ah = static_cast<float>(A), al = static_cast<float>(A - static_cast<double>(ah));
    int best = -1;
    for (int64_t s = s0; s < s1; ++s) {
        const int64_t first = s * kSegUnit - shift, mine0 = first + lane * kRun;
        Pair r[kRun], acc{0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kRun / W; ++i) {
            float pv[W], qv[W];
            load_vec(p, mine0 + i * W, V, pv);
            if (kDraft && use_q) load_vec(q, mine0 + i * W, V, qv);
#pragma unroll
            for (int w = 0; w < W; ++w)
                r[i * W + w] = kDraft && use_q ? residual(pv[w], qv[w], ah, al) : Pair{pv[w] > 0.f ? pv[w] : 0.f, 0.f};
        }
        if (!kDraft) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const int64_t off = gone[g] - first;
                for (uint32_t out = __ballot_sync(0xffffffffu, gone[g] >= 0 && off >= 0 && off < kSegUnit); out; out &= out - 1) {
                    const int x = __shfl_sync(0xffffffffu, static_cast<int>(off), __ffs(out) - 1);
#pragma unroll
                    for (int i = 0; i < kRun; ++i)
                        if (x == lane * kRun + i) r[i] = Pair{0.f, 0.f};
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kRun; ++i) add(acc, r[i].hi, r[i].lo);
        double ahead = before;
        bool hit;
        const int run = pass_point(acc, ahead, point, hit);
        if (run >= 0) {
            Pair mine{0.f, 0.f};
#pragma unroll
            for (int i = 0; i < kRun; ++i) {
                const Pair x = from_lane(r[i], run);
                if (lane == i) mine = x;
            }
            double in = hit ? ahead : -INFINITY;
            bool sure;
            const int e = pass_point(mine, in, point, sure);
            if (e >= 0) best = static_cast<int>(first) + run * kRun + e;
        }
        if (hit) break;
        before = ahead;
    }
    return best;
}

// The children of a node as bits, from the parents that a warp's lanes hold.
__device__ __forceinline__ uint64_t children(const int (&par)[2], int node) {
    return (static_cast<uint64_t>(__ballot_sync(0xffffffffu, par[1] == node)) << 32) | __ballot_sync(0xffffffffu, par[0] == node);
}

// The cluster barrier in two halves, each run by converged warps (__syncwarp before it).
__device__ __forceinline__ void cg_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
__device__ __forceinline__ void cg_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

// What the walk waits for, decided by warp 0 of every CTA alike and read by all of its threads.
enum Step : int { kPassResidual, kPassFinal, kDone };
struct __align__(16) Node {
    double u, p, q;              // its number, and its token's mass in its parent's rows
    int tok, pad;
};
struct Shared {
    Node node[kMaxNodes];
    Pair sums[2][kMaxSegs];      // this CTA's segments (in place), one buffer per pass parity
    Pair all[kMaxSegs];          // every segment of the last pass
    double A, R, total;
    int32_t removed[kMaxNodes];
    uint64_t accepted;
    int nremoved, cur, step, use_q, begins_low;
};

template <typename T, bool kDraft>
__global__ void __launch_bounds__(kVerThreads, 4) verify_kernel(const VerifyParams p) {
    __shared__ Shared sh;
    __shared__ int warp_tot[kVerWarps];
    __shared__ bool is_last;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = static_cast<int>(cluster.num_blocks());
    const int rank = static_cast<int>(cluster.block_rank());
    const int n = static_cast<int>(blockIdx.x) / C;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    const int64_t t0 = p.cu[n], t1 = p.cu[n + 1];
    const float u_draw = p.u_sample[n];
    uint32_t err = 0;
    if (t0 < 0 || t0 > t1 || t1 > p.T || t1 - t0 > kMaxNodes || (n == 0 && t0 != 0)) err = DEV_ERR_SEQLENS;
    const int m = err ? 0 : static_cast<int>(t1 - t0);

    // the nodes, two per lane (node lane and lane + 32), in warp 0 of every CTA
    int par[2] = {-2, -2}, tok[2] = {-1, -1};
    uint64_t accepted = 0;
    int cur = 0;
    double A = 0.0, R = 1.0;
    uint64_t tried = 0;        // children of cur already refused
    bool pending = false;      // a refusal whose R has not been summed yet
    if (warp == 0) {
        bool bad = false;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const int i = lane + 32 * w;
            if (i >= 1 && i < m) {
                par[w] = p.parent ? p.parent[t0 + i] : i - 1;
                tok[w] = p.tokens[t0 + i];
                const float u = p.u_accept[t0 + i];
                if (par[w] < 0 || par[w] >= i || tok[w] < 0 || tok[w] >= p.V) {
                    bad = true;
                } else {
                    Node nd{static_cast<double>(u), 0.0, 1.0, tok[w], 0};
                    nd.p = static_cast<double>(Elem<T>::to_f(static_cast<const T *>(p.target)[(t0 + par[w]) * p.ts + tok[w]]));
                    if (kDraft) nd.q = static_cast<double>(Elem<T>::to_f(static_cast<const T *>(p.draft)[(t0 + par[w]) * p.ds + tok[w]]));
                    sh.node[i] = nd;
                }
            }
        }
        if (__any_sync(0xffffffffu, bad)) err |= DEV_ERR_TREE;
        if (lane == 0) {
            sh.step = (err || m == 0) ? kDone : kPassResidual;
            sh.nremoved = 0;
            sh.accepted = 0;
            sh.begins_low = 0;
            is_last = false;
            if (rank == 0 && err) {
                grid_wait();   // the status word has been cleared
                atomicOr(p.status, err);
            }
        }
        accepted = (err || m == 0) ? 0ull : 1ull;
    }
    __syncthreads();
    bool dead = sh.step == kDone;
    __syncthreads();
    bool told = false;         // this sequence's accepted nodes are published
    // publishes the accepted nodes and counts the sequence off: as soon as the walk has ended, beside the draw's pass
    const bool publisher = rank == 0 && threadIdx.x == 32;
    auto publish = [&] {
        grid_wait();           // the counter has been cleared, the lengths have been checked
        if (__ldcg(p.status + 2) && __ldcg(p.accepted + n)) {
            sh.begins_low = 1;
            atomicOr(p.status, DEV_ERR_SEQLENS);
        }
        p.accepted[n] = sh.begins_low ? 0ull : sh.accepted;
        __threadfence();
        is_last = atomicAdd(p.status + 1, 1u) == static_cast<uint32_t>(p.N) - 1;
        __threadfence();
        told = true;
    };

    // packs every sequence's accepted nodes: the warps but the first of the CTA that counted off last
    bool packed = false;
    auto pack = [&] {
        constexpr int kPackThreads = kVerThreads - 32;
        const int tid = threadIdx.x - 32;
        int base_count = 0;
        for (int base = 0; base < p.N; base += kPackThreads) {
            const int i = base + tid;
            const uint64_t bits = i < p.N ? __ldcg(p.accepted + i) : 0ull;
            const int64_t first = i < p.N ? p.cu[i] : 0;
            const int mine = __popcll(bits);
            int upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += y;
            }
            if (lane == 31) warp_tot[warp] = upto;
            asm volatile("bar.sync 1, %0;" ::"n"(kPackThreads) : "memory");
            int off = base_count, all = base_count;
            for (int w = 1; w < kVerWarps; ++w) {
                if (w < warp) off += warp_tot[w];
                all += warp_tot[w];
            }
            if (i < p.N) {
                p.cu_accept[i + 1] = off + upto;  // (good sequences share no nodes: at most T)
                uint64_t b = bits;
                for (int at = off + upto - mine; b; b &= b - 1, ++at)
                    p.rows[at] = static_cast<int32_t>(first) + __ffsll(static_cast<long long>(b)) - 1;
            }
            base_count = all;
            asm volatile("bar.sync 1, %0;" ::"n"(kPackThreads) : "memory");
        }
        if (tid == 0) p.cu_accept[0] = 0;
        for (int64_t i = base_count + tid; i < p.T; i += kPackThreads) p.rows[i] = -1;
    };

    int token = -1;
    int parity = 0;
    bool fallback = false;
    int nrem = 0;
    while (!dead) {
        // ---- the walk, as far as it goes without a row sum (warp 0; every lane holds the same scalars)
        if (warp == 0) {
            int step = kPassFinal;
            if (!fallback) {
                if (pending) {           // the pass after a refusal gave R
                    R = sh.total;
                    pending = false;
                }
                uint64_t kids = children(par, cur);
                while (kids & ~tried) {
                    const int c = __ffsll(static_cast<long long>(kids & ~tried)) - 1;
                    const Node nd = sh.node[c];
                    double rx = nd.p;
                    if (kDraft) {
                        rx -= A * nd.q;
                    } else if (tried) {  // a token refused before has no mass left
                        const bool same = (tok[0] == nd.tok && ((tried >> lane) & 1)) || (tok[1] == nd.tok && ((tried >> (lane + 32)) & 1));
                        if (__any_sync(0xffffffffu, same)) rx = 0.0;
                    }
                    rx = rx > 0.0 ? rx : 0.0;
                    if (nd.u * nd.q * R < rx) {
                        accepted |= 1ull << c;
                        cur = c;
                        A = 0.0;
                        R = 1.0;
                        tried = 0;
                        nrem = 0;
                        kids = children(par, cur);
                    } else {
                        tried |= 1ull << c;
                        if (kDraft) {
                            A += R;
                            pending = true;
                            break;
                        }
                        R -= rx;
                        if (lane == 0) sh.removed[nrem] = nd.tok;
                        ++nrem;
                    }
                }
                // a refusal with children left to try needs R; otherwise the same pass serves the draw
                if (pending && (kids & ~tried)) step = kPassResidual;
            } else {
                A = 0.0;
                nrem = 0;
            }
            if (lane == 0) {
                sh.A = A;
                sh.cur = cur;
                sh.step = step;
                sh.nremoved = nrem;
                sh.use_q = kDraft && A != 0.0;
                sh.accepted = accepted;
            }
        }
        __syncthreads();
        const int step = sh.step, row = sh.cur, removed = sh.nremoved;
        const bool use_q = kDraft && sh.use_q;
        const double a = sh.A;
        if (publisher && step == kPassFinal && !told) publish();
        // ---- one pass over the current row
        Row<T> pr{static_cast<const T *>(p.target) + (t0 + row) * p.ts, true};
        Row<T> qr{kDraft ? static_cast<const T *>(p.draft) + (t0 + row) * p.ds : nullptr, true};
        const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(pr.base) & 15u) / sizeof(T));
        if (kDraft) qr.vec = ((reinterpret_cast<uintptr_t>(qr.base) / sizeof(T) - shift) * sizeof(T) & 15u) == 0;
        const int64_t steps = (static_cast<int64_t>(p.V) + shift + kSegUnit - 1) / kSegUnit;
        Pair *mine = sh.sums[parity];
        int gone[2];
#pragma unroll
        for (int g = 0; g < 2; ++g) gone[g] = !kDraft && lane + 32 * g < removed ? sh.removed[lane + 32 * g] : -1;
        for (int sg = 2 * (rank + C * warp); sg < p.nseg; sg += 2 * C * kVerWarps) {
            const Pair sum = segment_sums<T, kDraft>(pr, qr, use_q, shift, p.V, static_cast<int64_t>(sg) * p.seg_steps * kSegUnit - shift,
                                                       p.seg_steps, a, gone);
            if (lane == 0) mine[sg] = sum;
            if (lane == 16 && sg + 1 < p.nseg) mine[sg + 1] = sum;
        }
        cluster.sync();
        for (int sg = threadIdx.x; sg < p.nseg; sg += kVerThreads) {
            const Pair *from = cluster.map_shared_rank(mine, (sg >> 1) % C);
            sh.all[sg] = from[sg];
        }
        __syncthreads();
        if (warp == 0) {
            // lane l holds a run of consecutive segments; their scan gives the total, and the run that holds the draw
            const int per = (p.nseg + 31) / 32;
            Pair part{0.f, 0.f};
            for (int i = 0; i < per; ++i)
                if (lane * per + i < p.nseg) add(part, sh.all[lane * per + i].hi, sh.all[lane * per + i].lo);
            const double total = value(from_lane(warp_scan(part), 31));
            if (step == kPassResidual) {
                if (lane == 0) sh.total = total;
            } else if (!(total > 0.0) && !fallback && (use_q || removed > 0)) {
                if (lane == 0) sh.step = kPassResidual;  // a residual without mass: once more, over p itself
            } else {
                if (rank == 0 && total > 0.0) {
                    const double point = static_cast<double>(u_draw) * total;
                    double before = 0.0;
                    bool hit;
                    const int run = pass_point(part, before, point, hit);
                    if (!hit) before = -INFINITY;  // rounding at the far end: the last one with mass throughout
                    const int at = run * per + lane;
                    const int sg = pass_point(lane < per && at < p.nseg ? sh.all[at] : Pair{0.f, 0.f}, before, point, hit);
                    if (!hit) before = -INFINITY;
                    const int64_t s0 = static_cast<int64_t>(run * per + sg) * p.seg_steps;
                    const int64_t s1 = s0 + p.seg_steps < steps ? s0 + p.seg_steps : steps;
                    token = segment_find<T, kDraft>(pr, qr, use_q, shift, p.V, s0, s1, a, gone, before, point);
                }
                if (lane == 0) sh.step = kDone;
            }
        } else if (rank == 0 && step == kPassFinal && is_last && !packed) {
            pack();              // beside the draw
            packed = true;
        }
        __syncthreads();
        dead = sh.step == kDone;
        if (step == kPassFinal && !dead) fallback = true;
        parity ^= 1;
        __syncthreads();
    }

    // ---- the sequence's outputs; the last sequence to finish packs them all
    __syncwarp();
    cg_arrive();
    if (rank == 0 && threadIdx.x == 0) p.next_token[n] = sh.begins_low ? -1 : token;  // (not published yet: no token anyway)
    if (publisher && !told) publish();
    if (rank == 0) {
        __syncthreads();
        if (is_last && !packed && warp > 0) pack();
    }
    grid_wait();
    __syncwarp();
    cg_wait();  // no CTA leaves while another may still read its sums
}

template <typename T, bool kDraft>
kda_status launch_verify(const VerifyParams &p, int cluster, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(p.N) * cluster);
    cfg.blockDim = dim3(kVerThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // may begin beside the clearing of the status
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, verify_kernel<T, kDraft>, p) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace
}  // namespace kda

extern "C" {

size_t kda_draft_verify_workspace_size(int N) {
    return N < 0 ? 0 : KDA_WS_HEADER_BYTES + static_cast<size_t>(N) * sizeof(uint64_t);
}

kda_status kda_draft_verify(const int32_t *tokens, const int32_t *cu_nodes, const int32_t *parent,
                            const void *target_probs, const void *draft_probs, kda_dtype dtype, const float *u_accept,
                            const float *u_sample, int N, int64_t T, int V, int64_t target_stride,
                            int64_t draft_stride, int32_t *cu_accept, int32_t *rows, int32_t *next_token,
                            void *workspace, size_t ws_bytes, void *stream) {
    using namespace kda::spec;
    if (!dtype_ok(dtype)) return KDA_ERR_UNSUPPORTED;
    if (V > (1 << 24)) return KDA_ERR_UNSUPPORTED;
    if (N < 0 || N > (1 << 24) || T < 0 || T > 0x7fffffffLL || V <= 0) return KDA_ERR_INVALID_ARGUMENT;
    if (!target_stride) target_stride = V;
    if (!draft_stride) draft_stride = V;
    if (target_stride < V || draft_stride < V) return KDA_ERR_INVALID_ARGUMENT;
    if (!workspace || !aligned_to(workspace, 16) || ws_bytes < kda_draft_verify_workspace_size(N)) return KDA_ERR_WORKSPACE;
    if (!cu_accept || (T > 0 && !rows) || (N > 0 && (!cu_nodes || !u_sample || !next_token))) return KDA_ERR_INVALID_ARGUMENT;
    if (T > 0 && (!tokens || !target_probs || !u_accept)) return KDA_ERR_INVALID_ARGUMENT;
    const size_t es = elem_size(dtype);
    if (!aligned_to(target_probs, es) || !aligned_to(draft_probs, es)) return KDA_ERR_INVALID_ARGUMENT;
    for (const void *ptr : {static_cast<const void *>(tokens), static_cast<const void *>(cu_nodes),
                            static_cast<const void *>(parent), static_cast<const void *>(u_accept),
                            static_cast<const void *>(u_sample), static_cast<const void *>(cu_accept),
                            static_cast<const void *>(rows), static_cast<const void *>(next_token)})
        if (!aligned_to(ptr, 4)) return KDA_ERR_INVALID_ARGUMENT;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint64_t *accepted = reinterpret_cast<uint64_t *>(static_cast<char *>(workspace) + KDA_WS_HEADER_BYTES);
    if (!check_lengths(workspace, cu_nodes, N, accepted, s)) return KDA_ERR_CUDA;
    if (N == 0) {
        if (cudaMemsetAsync(cu_accept, 0, sizeof(int32_t), s) != cudaSuccess) return KDA_ERR_CUDA;
        if (T > 0 && cudaMemsetAsync(rows, 0xff, static_cast<size_t>(T) * sizeof(int32_t), s) != cudaSuccess) return KDA_ERR_CUDA;
        return KDA_OK;
    }
    kda::VerifyParams p{};
    p.tokens = tokens; p.cu = cu_nodes; p.parent = parent; p.target = target_probs; p.draft = draft_probs;
    p.u_accept = u_accept; p.u_sample = u_sample; p.T = T; p.ts = target_stride; p.ds = draft_stride;
    p.N = N; p.V = V; p.cu_accept = cu_accept; p.rows = rows; p.next_token = next_token;
    p.status = static_cast<uint32_t *>(workspace);
    p.accepted = accepted;
    // a row may start up to 7 elements after a 16-byte boundary
    const int64_t steps = (static_cast<int64_t>(V) + 7 + kda::kSegUnit - 1) / kda::kSegUnit;
    p.seg_steps = static_cast<int>((steps + kda::kMaxSegs - 1) / kda::kMaxSegs);
    p.nseg = static_cast<int>((steps + p.seg_steps - 1) / p.seg_steps);
    const int sms = sm_count();
    if (sms <= 0) return KDA_ERR_CUDA;
    // CTAs per sequence: as many as leave all sequences resident at once (four CTAs per SM), no more than the row's
    // segments can use
    int C = 1;
    while (C < kda::kMaxCluster && static_cast<int64_t>(N) * 2 * C <= 4 * sms && 2 * C * kda::kVerWarps < p.nseg) C *= 2;
    if (dtype == KDA_BF16)
        return draft_probs ? kda::launch_verify<__nv_bfloat16, true>(p, C, s) : kda::launch_verify<__nv_bfloat16, false>(p, C, s);
    return draft_probs ? kda::launch_verify<float, true>(p, C, s) : kda::launch_verify<float, false>(p, C, s);
}

}  // extern "C"
