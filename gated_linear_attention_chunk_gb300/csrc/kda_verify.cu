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
// the row into segments of kSeg elements, a warp each, and leaves the segments' sums in shared memory,
// where every CTA of the cluster reads them all in the same order; the draw then needs only the one segment that
// holds its point again.  So a sequence costs about one reading of one row (two with draft rows),
// which bounds it: the rest is the latency of the walk's dependent loads.
//
// Precision: the answers are whole numbers, so a rounding shows only next to a border, where a flat
// distribution over 10^5 tokens has one every 10^-5.  p - A q is carried as an unevaluated fp32 pair with
// the error terms of its product and difference, sums as pairs within a thread and in fp64 across threads:
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
constexpr int kSegUnit = 1024;    // elements of a segment (of one step of it, where a row has more than kMaxSegs)
constexpr int kLoadUnit = 512;    // elements that a warp has in flight
constexpr int kMaxSegs = 1024;    // segments of a row
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
    uint32_t *status;        // [0] status word, [1] ticket of finished sequences
    uint64_t *accepted;      // [N] accepted nodes as bits
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

// Sum of the residual over the segment steps [s0, s1) by one warp (every lane returns it).
template <typename T, bool kDraft>
__device__ __forceinline__ double segment_sum(const Row<T> &p, const Row<T> &q, bool use_q, int shift, int V, int64_t s0, int64_t s1,
                                              double A, const int32_t *removed, int nremoved) {
    constexpr int W = Elem<T>::kVec, L = kLoadUnit / 32 / W;  // vectors per lane
    const int lane = threadIdx.x & 31;
    const float ah = static_cast<float>(A), al = static_cast<float>(A - static_cast<double>(ah));
    Pair acc{0.f, 0.f};
    for (int64_t e0 = s0 * kSegUnit - shift; e0 < s1 * kSegUnit - shift; e0 += kLoadUnit) {
        float pv[L][W], qv[kDraft ? L : 1][W];
#pragma unroll
        for (int i = 0; i < L; ++i) load_vec(p, e0 + (i * 32 + lane) * W, V, pv[i]);
        if (kDraft && use_q) {
#pragma unroll
            for (int i = 0; i < L; ++i) load_vec(q, e0 + (i * 32 + lane) * W, V, qv[kDraft ? i : 0]);
        }
        for (int j = 0; j < nremoved; ++j) {  // refused certain drafts: no mass
            const int64_t x = removed[j] - e0;
            if (x >= 0 && x < kLoadUnit) {
#pragma unroll
                for (int i = 0; i < L; ++i)
#pragma unroll
                    for (int w = 0; w < W; ++w)
                        if (x == (i * 32 + lane) * W + w) pv[i][w] = 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < L; ++i)
#pragma unroll
            for (int w = 0; w < W; ++w) {
                if (kDraft && use_q) {
                    const Pair r = residual(pv[i][w], qv[kDraft ? i : 0][w], ah, al);
                    add(acc, r.hi, r.lo);
                } else {
                    add(acc, pv[i][w] > 0.f ? pv[i][w] : 0.f, 0.f);
                }
            }
    }
    double sum = static_cast<double>(acc.hi) + static_cast<double>(acc.lo);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
}

__device__ __forceinline__ double warp_scan(double x) {  // inclusive, in lane order
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// The lowest element of the steps [s0, s1) whose running sum, `before` included, passes `point`; the last element with
// mass if rounding leaves none; -1 without mass.  By one warp: the lane sums of 32 consecutive elements each find the
// run, then one element per lane.
template <typename T, bool kDraft>
__device__ __forceinline__ int segment_find(const Row<T> &p, const Row<T> &q, bool use_q, int shift, int V, int64_t s0, int64_t s1,
                                            double A, const int32_t *removed, int nremoved, double before, double point) {
    constexpr int W = Elem<T>::kVec, kRun = kSegUnit / 32;
    const int lane = threadIdx.x & 31;
    const float ah = static_cast<float>(A), al = static_cast<float>(A - static_cast<double>(ah));
    bool found = false;
    int64_t run0 = 0;           // first element of the run that holds the point
    double run_before = 0.0;
    for (int64_t s = s0; s < s1; ++s) {
        const int64_t mine0 = s * kSegUnit - shift + lane * kRun;
        Pair acc{0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kRun / W; ++i) {
            float pv[W], qv[W];
            load_vec(p, mine0 + i * W, V, pv);
            if (kDraft && use_q) load_vec(q, mine0 + i * W, V, qv);
            for (int j = 0; j < nremoved; ++j) {
                const int64_t x = removed[j] - (mine0 + i * W);
#pragma unroll
                for (int w = 0; w < W; ++w)
                    if (x == w) pv[w] = 0.f;
            }
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const Pair r = kDraft && use_q ? residual(pv[w], qv[w], ah, al) : Pair{pv[w] > 0.f ? pv[w] : 0.f, 0.f};
                add(acc, r.hi, r.lo);
            }
        }
        const double mine = static_cast<double>(acc.hi) + static_cast<double>(acc.lo);
        const double upto = warp_scan(mine), excl = before + (upto - mine);
        const uint32_t hit = __ballot_sync(0xffffffffu, mine > 0.0 && before + upto > point);
        const uint32_t some = __ballot_sync(0xffffffffu, mine > 0.0);
        if (hit || some) {      // (without a hit: the last run with mass, until a later step has one)
            const int src = hit ? __ffs(hit) - 1 : 31 - __clz(some);
            found = true;
            run0 = __shfl_sync(0xffffffffu, mine0, src);
            run_before = __shfl_sync(0xffffffffu, excl, src);
        }
        if (hit) break;
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
    if (!found) return -1;
    const int64_t e = run0 + lane;
    double x = 0.0;
    if (e >= 0 && e < V) {
        x = static_cast<double>(Elem<T>::to_f(p.base[e]));
        if (kDraft && use_q) x -= A * static_cast<double>(Elem<T>::to_f(q.base[e]));
        for (int j = 0; j < nremoved; ++j)
            if (removed[j] == e) x = 0.0;
        if (!(x > 0.0)) x = 0.0;
    }
    const double upto = run_before + warp_scan(x);
    const uint32_t hit = __ballot_sync(0xffffffffu, x > 0.0 && upto > point);
    const uint32_t some = __ballot_sync(0xffffffffu, x > 0.0);
    if (!some) return -1;
    return static_cast<int>(run0) + (hit ? __ffs(hit) - 1 : 31 - __clz(some));
}

// The children of a node as bits, from the parents that a warp's lanes hold.
__device__ __forceinline__ uint64_t children(const int (&par)[2], int node) {
    return (static_cast<uint64_t>(__ballot_sync(0xffffffffu, par[1] == node)) << 32) | __ballot_sync(0xffffffffu, par[0] == node);
}

// What the walk waits for, decided by warp 0 of every CTA alike and read by all of its threads.
enum Step : int { kPassResidual, kPassFinal, kDone };
struct __align__(16) Node {
    double u, p, q;              // its number, and its token's mass in its parent's rows
    int tok, pad;
};
struct Shared {
    Node node[kMaxNodes];
    double sums[2][kMaxSegs];    // this CTA's segments (in place), one buffer per pass parity
    double all[kMaxSegs];        // every segment of the last pass
    double A, R, total;
    int32_t removed[kMaxNodes];
    int nremoved, cur, step, use_q;
    int count_before;            // last CTA: running counts
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
            if (rank == 0 && err) atomicOr(p.status, err);
        }
        accepted = (err || m == 0) ? 0ull : 1ull;
    }
    __syncthreads();
    bool dead = sh.step == kDone;
    __syncthreads();
    bool told = false;         // this sequence's accepted nodes are published
    // publishes the accepted nodes and counts the sequence off (early: the packing needs no token)
    auto publish = [&] {
        p.accepted[n] = accepted;
        __threadfence();
        is_last = atomicAdd(p.status + 1, 1u) == static_cast<uint32_t>(p.N) - 1;
        told = true;
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
                if (rank == 0 && step == kPassFinal && !told) publish();
            }
        }
        __syncthreads();
        const int step = sh.step, row = sh.cur, removed = sh.nremoved;
        const bool use_q = kDraft && sh.use_q;
        const double a = sh.A;
        // ---- one pass over the current row
        Row<T> pr{static_cast<const T *>(p.target) + (t0 + row) * p.ts, true};
        Row<T> qr{kDraft ? static_cast<const T *>(p.draft) + (t0 + row) * p.ds : nullptr, true};
        const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(pr.base) & 15u) / sizeof(T));
        if (kDraft) qr.vec = ((reinterpret_cast<uintptr_t>(qr.base) / sizeof(T) - shift) * sizeof(T) & 15u) == 0;
        const int64_t steps = (static_cast<int64_t>(p.V) + shift + kSegUnit - 1) / kSegUnit;
        double *mine = sh.sums[parity];
        for (int sg = rank + C * warp; sg < p.nseg; sg += C * kVerWarps) {
            const int64_t s0 = static_cast<int64_t>(sg) * p.seg_steps;
            const int64_t s1 = s0 + p.seg_steps < steps ? s0 + p.seg_steps : steps;
            const double sum = segment_sum<T, kDraft>(pr, qr, use_q, shift, p.V, s0, s1, a, sh.removed, removed);
            if (lane == 0) mine[sg] = sum;
        }
        cluster.sync();
        for (int sg = threadIdx.x; sg < p.nseg; sg += kVerThreads) {
            const double *from = cluster.map_shared_rank(mine, sg % C);
            sh.all[sg] = from[sg];
        }
        __syncthreads();
        if (warp == 0) {
            // lane l holds a run of consecutive segments; their scan gives the total and finds the draw
            const int per = (p.nseg + 31) / 32;
            double part = 0.0;
            for (int i = 0; i < per; ++i)
                if (lane * per + i < p.nseg) part += sh.all[lane * per + i];
            const double upto = warp_scan(part);
            const double total = __shfl_sync(0xffffffffu, upto, 31);
            if (step == kPassResidual) {
                if (lane == 0) sh.total = total;
            } else {
                // (a residual without mass: once more, over p itself)
                const bool again = !(total > 0.0) && !fallback && (use_q || removed > 0);
                if (again) {
                    if (lane == 0) sh.step = kPassResidual;
                } else {
                    const double point = static_cast<double>(p.u_sample[n]) * total;
                    int sg = -1, top = -1;
                    double run = upto - part, before = 0.0, top_before = 0.0;
                    for (int i = 0; i < per; ++i) {
                        const int at = lane * per + i;
                        if (at >= p.nseg) break;
                        const double x = sh.all[at];
                        if (x > 0.0) {
                            top = at;
                            top_before = run;
                            if (sg < 0 && run + x > point) {
                                sg = at;
                                before = run;
                            }
                        }
                        run += x;
                    }
                    uint32_t any = __ballot_sync(0xffffffffu, sg >= 0);
                    int src = __ffs(any) - 1;
                    if (!any) {  // rounding at the far end: the last segment with mass
                        any = __ballot_sync(0xffffffffu, top >= 0);
                        src = 31 - __clz(any);
                        sg = top;
                        before = top_before;
                    }
                    if (any && rank == 0) {
                        sg = __shfl_sync(0xffffffffu, sg, src);
                        before = __shfl_sync(0xffffffffu, before, src);
                        const int64_t s0 = static_cast<int64_t>(sg) * p.seg_steps;
                        const int64_t s1 = s0 + p.seg_steps < steps ? s0 + p.seg_steps : steps;
                        token = segment_find<T, kDraft>(pr, qr, use_q, shift, p.V, s0, s1, a, sh.removed, removed, before, point);
                    }
                    if (lane == 0) sh.step = kDone;
                }
            }
        }
        __syncthreads();
        dead = sh.step == kDone;
        if (step == kPassFinal && !dead) fallback = true;
        parity ^= 1;
        __syncthreads();
    }

    // ---- the sequence's outputs; the last sequence to finish packs them all
    if (rank == 0 && threadIdx.x == 0) {
        p.next_token[n] = token;
        if (!told) publish();
    }
    if (rank == 0) {
        __syncthreads();
        if (is_last) {
            __threadfence();
            if (threadIdx.x == 0) {
                sh.count_before = 0;
                p.cu_accept[0] = 0;
            }
            __syncthreads();
            for (int base = 0; base < p.N; base += kVerThreads) {
                const int i = base + threadIdx.x;
                const uint64_t bits = i < p.N ? __ldcg(p.accepted + i) : 0ull;
                const int mine = __popcll(bits);
                int upto = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += y;
                }
                if (lane == 31) warp_tot[warp] = upto;
                __syncthreads();
                int off = sh.count_before;
                for (int w = 0; w < warp; ++w) off += warp_tot[w];
                if (i < p.N) {
                    // (overlapping ranges of a bad cu_nodes could count more than T nodes)
                    p.cu_accept[i + 1] = off + upto < p.T ? off + upto : static_cast<int32_t>(p.T);
                    const int64_t first = p.cu[i];
                    uint64_t b = bits;
                    for (int at = off + upto - mine; b && at < p.T; b &= b - 1, ++at)
                        p.rows[at] = static_cast<int32_t>(first) + __ffsll(static_cast<long long>(b)) - 1;
                }
                __syncthreads();
                if (threadIdx.x == kVerThreads - 1) sh.count_before = off + upto;
                __syncthreads();
            }
            for (int64_t i = sh.count_before + threadIdx.x; i < p.T; i += kVerThreads) p.rows[i] = -1;
        }
    }
    cluster.sync();  // no CTA leaves while another may still read its sums
}

template <typename T, bool kDraft>
kda_status launch_verify(const VerifyParams &p, int cluster, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(p.N) * cluster);
    cfg.blockDim = dim3(kVerThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
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
    if (cudaMemsetAsync(workspace, 0, 2 * sizeof(uint32_t), s) != cudaSuccess) return KDA_ERR_CUDA;
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
    p.accepted = reinterpret_cast<uint64_t *>(static_cast<char *>(workspace) + KDA_WS_HEADER_BYTES);
    // a row may start up to 7 elements after a 16-byte boundary
    const int64_t steps = (static_cast<int64_t>(V) + 7 + kda::kSegUnit - 1) / kda::kSegUnit;
    p.seg_steps = static_cast<int>((steps + kda::kMaxSegs - 1) / kda::kMaxSegs);
    p.nseg = static_cast<int>((steps + p.seg_steps - 1) / p.seg_steps);
    const int sms = sm_count();
    if (sms <= 0) return KDA_ERR_CUDA;
    // CTAs per sequence: as many as leave all sequences resident at once (four CTAs per SM), no more than the row's
    // segments can use
    int C = 1;
    while (C < kda::kMaxCluster && static_cast<int64_t>(N) * 2 * C <= 4 * sms && C * kda::kVerWarps < p.nseg) C *= 2;
    if (dtype == KDA_BF16)
        return draft_probs ? kda::launch_verify<__nv_bfloat16, true>(p, C, s) : kda::launch_verify<__nv_bfloat16, false>(p, C, s);
    return draft_probs ? kda::launch_verify<float, true>(p, C, s) : kda::launch_verify<float, false>(p, C, s);
}

}  // extern "C"
