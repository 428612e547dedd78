// RMS norms of q and k per head with learned weights, then rotary positions, in one pass; and the gradient.
//
// A head's row x of d channels, with n = r x, r = (mean x_i^2 + eps)^-1/2, becomes R(p) (w * n): R turns pair j by the angle p
// w_j and scales it by m, as kda_rope does.  With g the output's gradient and b = R^T g (the turn by the opposite angle),
//     dw = sum over rows of b * n,      e = w * b,      dx = r (e - n mean(e * n)),
// and mean(e * n) = r sum(e * x) / d, so that sum(x^2) and sum(e x) are all that a row's lanes have to share.  The gradient
// reads x again in the place of a stored r: it needs n anyway.
//
// The bytes of the rows, read and written once, bound it.  A CTA has rows of q or of k (so that a thread keeps its channels'
// weights, and in the gradient its channels' sums of dw, in registers) of a few tokens; sines and cosines are computed once per
// (token, pair) into shared memory from the exactly reduced angle (kda_rope.cu).  A row belongs to a group of lanes, each with
// two 16-byte columns: the two halves of its pairs, or two neighbours.  A group takes several heads of one token, for which it
// holds the sines in registers.  Rows that are not 16-byte aligned, and halves that do not split into such columns, go through
// shared memory.
//
// 16,384 tokens of 32 + 8 heads of 128, bf16: forward 63 us (5.3 TB/s, 80% of the copy rate; issue 64% busy), gradient 109
// (4.6 TB/s, 69%: 16 warps per SM, whose sums of dw take the registers), its weights' sums 3 of them; fp32 forward 101 (6.6
// TB/s).  8,191 tokens of 32 + 32 heads of 64, fp32: forward 44 us (6.2 TB/s), gradient 67 (6.0 TB/s, 90%).  Through shared
// memory (126 of 128 channels turned, in halves): 139 and 278 us (neighbours: 62 and 103 for 20 of 128).  A decoding step's 512
// tokens: 6 to 9 us, of which the launch is half.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "kda_spec.cuh"

namespace kda {
namespace {

using namespace spec;

constexpr int kNormThreads = 128;    // (256: 71.5 us forward, 119 gradient, where these take 66.5 and 111)
constexpr int kStagedThreads = 128;  // of the path through shared memory
constexpr int kUnroll = 2;           // rows in flight per thread
constexpr int kRounds = 8;           // heads for which a thread keeps a token's sines
constexpr int kBwdPerSm = 4, kStagedPerSm = 6;  // CTAs; of the gradient each has its own sums of dw
// Forward: seven leave 72 registers, of which bf16 spills 56 to 76 bytes, six 80 (8 to 16 bytes).  bf16, 16,384 tokens of 32 +
// 8 heads of 128: 64.0 us with seven, 62.4 with six; fp32, which spills neither way, 101.2 and 105.4.
template <typename T>
constexpr int kFwdPerSm = sizeof(T) == 2 ? 6 : 7;

struct NormParams {
    // [0]: q, [1]: k
    const void *x[2], *g[2], *w[2];
    void *y[2];
    int64_t xs[2], gs[2], ys[2];  // token strides in elements
    int H[2], tokens[2];          // heads; tokens of a CTA at a time
    int share[2];                 // groups of lanes that share a token
    int64_t blocks[2];            // CTAs
    const int32_t *positions;
    const double *inv_freq;
    int64_t T;
    int d, rot;
    int lanes;                    // of a row: a power of two
    bool wide_w, vec_w, vec_rows; // weights are fp32; weights, rows are 16-byte aligned
    float mscale, eps;
    float *part;                  // gradient: [CTA][d] sums of dw
    int fold_at;                  // gradient: a thread's pairs of sums in shared memory, in floats (0: none, its rows are few)
};

// p w_j modulo one turn is exact in 64-bit fixed point; as in kda_rope.cu.
__device__ __forceinline__ void make_turns(uint64_t *turn, const NormParams &p, int threads) {
    for (int j = threadIdx.x; j < p.rot / 2; j += threads) {
        const double f = p.inv_freq[j] * 0.15915494309189533577;  // 1 / (2 pi)
        turn[j] = __double2ull_rz((f - floor(f)) * 18446744073709551616.0);
    }
}
__host__ __device__ __forceinline__ int table_pitch(int rot) { return (rot / 2 + 3) & ~3; }  // floats of a token: rows are 16-byte aligned
__device__ __forceinline__ void make_table(float *cs, float *sn, const uint64_t *turn, const NormParams &p, int64_t t0, int nt, int threads) {
    const int half = p.rot / 2, pitch = table_pitch(p.rot);
    for (int e = threadIdx.x; e < nt * half; e += threads) {
        const int t = e / half, j = e - t * half;
        const uint64_t a = static_cast<uint64_t>(static_cast<int64_t>(p.positions[t0 + t])) * turn[j];
        // the nearest quarter turn, and what is left as an fp32 number of half turns (at most 1/4: 2^-27 off, as against 2^-25
        // without)
        const uint32_t turns = static_cast<uint32_t>(a >> 32), quarter = (turns + 0x20000000u) >> 30;
        const float h = static_cast<float>(static_cast<int32_t>(turns - (quarter << 30))) * 4.656612873077392578e-10f;
        float s, c;
        sincospif(h, &s, &c);
        const float u = quarter & 1u ? -s : c, v = quarter & 1u ? c : s;  // a quarter on: (c, s) -> (-s, c)
        c = quarter & 2u ? -u : u;
        s = quarter & 2u ? -v : v;
        cs[t * pitch + j] = c * p.mscale;
        sn[t * pitch + j] = s * p.mscale;
    }
}
__device__ __forceinline__ float weight_at(const void *w, bool wide, int i) {
    if (!w) return 1.f;
    return wide ? static_cast<const float *>(w)[i] : __bfloat162float(static_cast<const __nv_bfloat16 *>(w)[i]);
}
// V weights from channel i on (a multiple of V); 0 where there is no column.
template <int V>
__device__ __forceinline__ void weights_at(float (&f)[V], const void *w, const NormParams &p, int i, bool there) {
    if (!there || !w || !p.vec_w) {
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] = there ? weight_at(w, p.wide_w, i + j) : 0.f;
    } else if (p.wide_w) {
#pragma unroll
        for (int j = 0; j < V; j += 4)
            *reinterpret_cast<float4 *>(f + j) = *reinterpret_cast<const float4 *>(static_cast<const float *>(w) + i + j);
    } else {
        const __nv_bfloat162 *from = reinterpret_cast<const __nv_bfloat162 *>(static_cast<const __nv_bfloat16 *>(w) + i);
#pragma unroll
        for (int j = 0; j < V; j += 2) {
            const float2 x = __bfloat1622float2(from[j / 2]);
            f[j] = x.x;
            f[j + 1] = x.y;
        }
    }
}
// x^-1/2 to a unit in the last place: a Newton step after rsqrtf's two (not where that is no number).
__device__ __forceinline__ float inverse_root(float x) {
    const float y = rsqrtf(x), z = fmaf(0.5f * y, fmaf(-x * y, y, 1.f), y);
    return x > 0.f && x < INFINITY ? z : y;
}
__device__ __forceinline__ float lanes_sum(float x, int lanes) {
    for (int o = lanes >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Which channels are pairs: (j, j + rot / 2); or (2 j, 2 j + 1), all of them or those below rot.  (16,384 tokens of 32 + 8 heads of
// 128 in bf16, gradient: neighbours 117 us, 120 where their number is looked at; halves are as fast either way.)
enum Layout { kHalves, kNeighbours, kSomeNeighbours };
// A thread's two columns of a row: channels a .. a + V and b .. b + V.
struct Columns {
    int a, b, table;  // table: its first pair (half layout), or a's first pair
    bool has_a, has_b;
    bool turns;       // half layout: its pairs are turned (neighbours: those below rot / 2 are)
};
template <int V, Layout kLayout>
__device__ __forceinline__ Columns columns_of(int lane, int d, int rot) {
    Columns c{};
    constexpr bool kInterleaved = kLayout != kHalves;
    const int pairs = kInterleaved ? 0 : rot / 2 / V;  // lanes that hold both halves of their pairs
    if (lane < pairs) {
        c.a = lane * V;
        c.b = rot / 2 + lane * V;
        c.table = lane * V;
        c.has_a = c.has_b = c.turns = true;
        return c;
    }
    const int base = kInterleaved ? 0 : rot;
    c.a = base + 2 * (lane - pairs) * V;
    c.b = c.a + V;
    c.has_a = c.a < d;
    c.has_b = c.b < d;
    if (kInterleaved) c.table = c.a / 2;
    return c;
}

// The columns' first n pairs (of halves all or none) turned by the angle, or by its opposite (kBack).  co, si: of the pairs (a_i, b_i),
// or of a's and then b's pairs of neighbours, 1 and 0 where there is none: an infinity or a NaN in such a channel is nothing to
// the other.
template <int V, Layout kLayout, bool kBack>
__device__ __forceinline__ void turn_columns(float (&a)[V], float (&b)[V], const float (&co)[V], const float (&si)[V], int n) {
    constexpr bool kInterleaved = kLayout != kHalves;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float &x = kInterleaved ? (i < V / 2 ? a[2 * i] : b[2 * i - V]) : a[i];
        float &y = kInterleaved ? (i < V / 2 ? a[2 * i + 1] : b[2 * i - V + 1]) : b[i];
        const float u = kInterleaved || n > 0 ? x : 0.f, v = kInterleaved || n > 0 ? y : 0.f;
        const float s = kBack ? fmaf(x, co[i], v * si[i]) : fmaf(x, co[i], -(v * si[i]));
        const float t = kBack ? fmaf(y, co[i], -(u * si[i])) : fmaf(u, si[i], y * co[i]);
        const bool pair = kLayout != kSomeNeighbours || i < n;
        x = pair ? s : x;
        y = pair ? t : y;
    }
}

template <typename T>
__device__ __forceinline__ uint4 load16(const T *row, int at, bool there) {
    return there ? *reinterpret_cast<const uint4 *>(row + at) : make_uint4(0u, 0u, 0u, 0u);
}

extern __shared__ __align__(16) char norm_smem[];

// A sum of fp32 numbers that keeps what its roundings leave out.
struct Pair {
    float high, low;
    __device__ __forceinline__ void add(float x) {
        const float s = __fadd_rn(high, x), b = __fsub_rn(s, high);
        low = __fadd_rn(low, __fadd_rn(__fsub_rn(high, __fsub_rn(s, b)), __fsub_rn(x, b)));
        high = s;
    }
    // (beyond fp32's range `high` is what a plain sum has, and what it leaves out no number)
    __device__ __forceinline__ float value() const { return fabsf(high) < INFINITY ? high + low : high; }
};
// Sums of dw: a thread adds up kChain rows or so plainly, then those sums as pairs, which lie in shared memory.  So their
// error does not grow with the rows of a call; rows that are all alike, as a padded batch has them, took plain sums of some
// thousand off by 400 to 730 units of 2^-24.  A call with fewer rows per thread has no pairs (16,384 tokens of 32 + 8 heads of
// 128 make 72); 131,072 such tokens take 811 us with them and 793 without.
constexpr int kChain = 128;

// kFold: a gradient whose threads have more than kChain rows (as a variable in the same kernel it took the others from 111 to
// 114 us).
template <typename T, Layout kLayout, bool kBwd, bool kFold>
__global__ void __launch_bounds__(kNormThreads, kBwd ? kBwdPerSm : kFwdPerSm<T>) norm_rope_kernel(const NormParams p) {
    constexpr int V = Elem<T>::kVec;
    constexpr bool kInterleaved = kLayout != kHalves;
    const int half = p.rot / 2, pitch = table_pitch(p.rot);
    const int which = blockIdx.x < p.blocks[0] ? 0 : 1;
    const int64_t block = blockIdx.x - (which ? p.blocks[0] : 0), blocks = p.blocks[which];
    const int H = p.H[which], tokens = p.tokens[which];
    uint64_t *turn = reinterpret_cast<uint64_t *>(norm_smem);  // [half]
    float *cs = reinterpret_cast<float *>(turn + ((half + 1) & ~1)), *sn = cs + tokens * pitch;
    const int lane = threadIdx.x & (p.lanes - 1), group = threadIdx.x / p.lanes, share = p.share[which];
    const int slot = group / share, head0 = group - slot * share;  // the group's token in the CTA, its first head
    const Columns c = columns_of<V, kLayout>(lane, p.d, p.rot);
    const int turned = kInterleaved ? half - c.table : c.turns ? V : 0;  // pairs of the columns, if that many
    const int64_t step = static_cast<int64_t>(share) * p.d;        // from one of the group's heads to the next
    int64_t t0 = block * tokens;
    const T *x, *g = nullptr;                                      // the group's next head to load, this thread's column a
    T *y;
    int left;                                                      // heads still to load
    const int to_b = c.b - c.a;
    auto begin = [&] {
        const int64_t t = t0 + slot < p.T ? t0 + slot : 0, h = static_cast<int64_t>(head0) * p.d + (c.has_a ? c.a : 0);
        x = static_cast<const T *>(p.x[which]) + t * p.xs[which] + h;
        if constexpr (kBwd) g = static_cast<const T *>(p.g[which]) + t * p.gs[which] + h;
        y = static_cast<T *>(p.y[which]) + t * p.ys[which] + h;
        left = t0 + slot < p.T && slot < tokens ? (H - head0 + share - 1) / share : 0;
    };
    uint4 xa[kUnroll], xb[kUnroll], ga[kUnroll], gb[kUnroll];
    auto load = [&] {
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const bool in = i < left;
            xa[i] = load16(x, 0, in && c.has_a);
            xb[i] = load16(x, to_b, in && c.has_b);
            x += step;
            if constexpr (kBwd) {
                ga[i] = load16(g, 0, in && c.has_a);
                gb[i] = load16(g, to_b, in && c.has_b);
                g += step;
            }
        }
    };
    begin();
    grid_wait();
    load();  // on its way while the frequencies, weights and sines are prepared
    make_turns(turn, p, kNormThreads);
    float wa[V], wb[V];
    weights_at<V>(wa, p.w[which], p, c.a, c.has_a);
    weights_at<V>(wb, p.w[which], p, c.b, c.has_b);
    float da[V] = {}, db[V] = {};  // sums of dw
    int chain = 0;                 // rows in them
    // [2 V] pairs of this thread
    auto folded = [&](int j) {
        return reinterpret_cast<Pair *>(reinterpret_cast<float *>(norm_smem) + p.fold_at) + j * kNormThreads + threadIdx.x;
    };
    auto fold = [&] {
#pragma unroll
        for (int j = 0; j < 2 * V; ++j) {
            Pair s = *folded(j);
            s.add(j < V ? da[j] : db[j - V]);
            *folded(j) = s;
            (j < V ? da[j] : db[j - V]) = 0.f;
        }
        chain = 0;
    };
    if constexpr (kFold) {
        for (int j = 0; j < 2 * V; ++j) *folded(j) = Pair{0.f, 0.f};
    }
    const float inv_d = 1.f / static_cast<float>(p.d);
    const int rounds = (H + share - 1) / share;  // heads of a group, the same for all lanes of a warp: the shuffles below are of whole warps
    __syncthreads();
    for (;;) {
        const int nt = static_cast<int>(p.T - t0 < tokens ? p.T - t0 : tokens);
        make_table(cs, sn, turn, p, t0, nt, kNormThreads);
        __syncthreads();
        float co[V], si[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const bool there = i < turned && slot < nt;
            co[i] = there ? cs[slot * pitch + c.table + i] : 1.f;
            si[i] = there ? sn[slot * pitch + c.table + i] : 0.f;
        }
        for (int r0 = 0; r0 < rounds; r0 += kUnroll) {
            if (r0 > 0) load();
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                const bool in = i < left;
                float a[V], b[V];
                unpack16(xa[i], a);
                unpack16(xb[i], b);
                float ss = 0.f;
#pragma unroll
                for (int j = 0; j < V; ++j) ss = fmaf(a[j], a[j], fmaf(b[j], b[j], ss));
                if constexpr (!kBwd) {
                    const float rn = inverse_root(fmaf(lanes_sum(ss, p.lanes), inv_d, p.eps));
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        a[j] = a[j] * rn * wa[j];
                        b[j] = b[j] * rn * wb[j];
                    }
                    turn_columns<V, kLayout, false>(a, b, co, si, turned);
                } else {
                    float u[V], v[V];
                    unpack16(ga[i], u);
                    unpack16(gb[i], v);
                    turn_columns<V, kLayout, true>(u, v, co, si, turned);
                    float ex = 0.f;
#pragma unroll
                    for (int j = 0; j < V; ++j) ex = fmaf(u[j] * wa[j], a[j], fmaf(v[j] * wb[j], b[j], ex));
                    float rn = inverse_root(fmaf(lanes_sum(ss, p.lanes), inv_d, p.eps));
                    rn = in ? rn : 0.f;  // (a row that is not there is all zeros, and eps may be zero)
                    const float mean = rn * rn * lanes_sum(ex, p.lanes) * inv_d;  // times x: n mean(e n)
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        da[j] = fmaf(u[j], a[j] * rn, da[j]);
                        db[j] = fmaf(v[j], b[j] * rn, db[j]);
                        a[j] = rn * fmaf(-mean, a[j], u[j] * wa[j]);
                        b[j] = rn * fmaf(-mean, b[j], v[j] * wb[j]);
                    }
                }
                if (in) {
                    if (c.has_a) *reinterpret_cast<uint4 *>(y) = pack16(a);
                    if (c.has_b) *reinterpret_cast<uint4 *>(y + to_b) = pack16(b);
                }
                y += step;
            }
            left -= kUnroll;
            if constexpr (kFold) {
                chain += kUnroll;
                if (chain >= kChain) fold();
            }
        }
        __syncthreads();
        t0 += blocks * tokens;
        if (t0 >= p.T) break;
        begin();
        load();
    }
    if constexpr (kBwd) {
        // the groups' sums joined: groups of a warp by shuffles, warps through shared memory, in a fixed order
        float *sums = reinterpret_cast<float *>(norm_smem);  // [warps][d]
        const int warp = threadIdx.x >> 5;
        if constexpr (kFold) {
            fold();
#pragma unroll
            for (int j = 0; j < V; ++j) {
                da[j] = folded(j)->value();
                db[j] = folded(V + j)->value();
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j)
            for (int o = p.lanes; o < 32; o <<= 1) {
                da[j] += __shfl_xor_sync(0xffffffffu, da[j], o);
                db[j] += __shfl_xor_sync(0xffffffffu, db[j], o);
            }
        if ((threadIdx.x & 31) < p.lanes) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (c.has_a) sums[warp * p.d + c.a + j] = da[j];
                if (c.has_b) sums[warp * p.d + c.b + j] = db[j];
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < p.d; i += kNormThreads) {
            float s = 0.f;
            for (int w = 0; w < kNormThreads / 32; ++w) s += sums[w * p.d + i];
            p.part[static_cast<int64_t>(blockIdx.x) * p.d + i] = s;
        }
    }
}

// Any rotated width and alignment: a row staged in shared memory as fp32, its pairs shared out among its lanes.
//
// Floats of a group of lanes in shared memory: rows, and as much as puts the groups of a warp next to one another in the banks
// (gradient of the same 314 -> 278 us; fp32 heads of 64, 73 -> 55 and 171 -> 106).
__host__ __device__ __forceinline__ int staged_span(bool bwd, bool fold, int d, int lanes) {
    return (!bwd ? 1 : fold ? 5 : 3) * d + (lanes & 31);
}

template <typename T, bool kInterleaved, bool kBwd>
__global__ void __launch_bounds__(kStagedThreads) norm_rope_staged_kernel(const NormParams p) {
    constexpr int V = Elem<T>::kVec;
    const int half = p.rot / 2, pitch = table_pitch(p.rot), d = p.d;
    const int which = blockIdx.x < p.blocks[0] ? 0 : 1;
    const int64_t block = blockIdx.x - (which ? p.blocks[0] : 0), blocks = p.blocks[which];
    const int H = p.H[which], tokens = p.tokens[which];
    const int lane = threadIdx.x & (p.lanes - 1), group = threadIdx.x / p.lanes, groups = kStagedThreads / p.lanes;
    uint64_t *turn = reinterpret_cast<uint64_t *>(norm_smem);
    float *cs = reinterpret_cast<float *>(turn + ((half + 1) & ~1)), *sn = cs + tokens * pitch;
    float *w = sn + tokens * pitch;                          // [d]
    const bool pairs = kBwd && p.fold_at;
    const int span = staged_span(kBwd, pairs, d, p.lanes);
    float *mine = w + d + group * span;                      // the group's rows: x, g, sums of dw, [d] pairs of such sums
    float *mine_g = mine + d, *dw = mine + 2 * d, *folded = dw + d;
    int chain = 0;                                           // rows in dw
    auto fold = [&] {
        for (int i = lane; i < d; i += p.lanes) {
            Pair s{folded[i], folded[d + i]};
            s.add(dw[i]);
            folded[i] = s.high;
            folded[d + i] = s.low;
            dw[i] = 0.f;
        }
        chain = 0;
    };
    grid_wait();
    make_turns(turn, p, kStagedThreads);
    for (int i = threadIdx.x; i < d; i += kStagedThreads) w[i] = weight_at(p.w[which], p.wide_w, i);
    if constexpr (kBwd)
        for (int i = lane; i < (pairs ? 3 : 1) * d; i += p.lanes) dw[i] = 0.f;
    const float inv_d = 1.f / static_cast<float>(d);
    const T *x = static_cast<const T *>(p.x[which]), *g = static_cast<const T *>(p.g[which]);
    T *y = static_cast<T *>(p.y[which]);
    auto put = [&](float *to, const uint4 &raw) {
        float f[V];
        unpack16(raw, f);
#pragma unroll
        for (int i = 0; i < V; i += 4) *reinterpret_cast<float4 *>(to + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
    };
    auto fetch = [&](float *to, const T *row) {
        if (p.vec_rows) {
            for (int u = lane; u < d / V; u += p.lanes) put(to + u * V, *reinterpret_cast<const uint4 *>(row + u * V));
        } else {
            for (int i = lane; i < d; i += p.lanes) to[i] = Elem<T>::to_f(row[i]);
        }
    };
    // The group's next row on its way while this one is worked on, where a lane has no more than two columns of it (126 of 128
    // channels turned: 190 us without, 141 with; gradient 380, 314).
    const bool ahead = p.vec_rows && d / V <= 2 * p.lanes;
    uint4 nx[2], ng[2];
    auto load_ahead = [&](int64_t t, int h) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int u = lane + i * p.lanes;
            if (u >= d / V) continue;
            nx[i] = *reinterpret_cast<const uint4 *>(x + t * p.xs[which] + static_cast<int64_t>(h) * d + u * V);
            if constexpr (kBwd) ng[i] = *reinterpret_cast<const uint4 *>(g + t * p.gs[which] + static_cast<int64_t>(h) * d + u * V);
        }
    };
    __syncthreads();
    for (int64_t t0 = block * tokens; t0 < p.T; t0 += blocks * tokens) {
        const int nt = static_cast<int>(p.T - t0 < tokens ? p.T - t0 : tokens), rows = nt * H;
        if (ahead && group < rows) load_ahead(t0 + group / H, group % H);
        make_table(cs, sn, turn, p, t0, nt, kStagedThreads);
        __syncthreads();
        for (int r0 = 0; r0 < rows; r0 += groups) {
            const int r = r0 + group;
            const bool in = r < rows;
            const int t = in ? r / H : 0, h = in ? r - t * H : 0;
            const float *tc = cs + t * pitch, *ts = sn + t * pitch;
            if (in && ahead) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int u = lane + i * p.lanes;
                    if (u >= d / V) continue;
                    put(mine + u * V, nx[i]);
                    if constexpr (kBwd) put(mine_g + u * V, ng[i]);
                }
                const int next = r + groups;
                if (next < rows) load_ahead(t0 + next / H, next % H);
            } else if (in) {
                fetch(mine, x + (t0 + t) * p.xs[which] + static_cast<int64_t>(h) * d);
                if constexpr (kBwd) fetch(mine_g, g + (t0 + t) * p.gs[which] + static_cast<int64_t>(h) * d);
            }
            __syncwarp();
            float ss = 0.f, ex = 0.f;
            if (in)
                for (int i = lane; i < d; i += p.lanes) ss = fmaf(mine[i], mine[i], ss);
            if constexpr (kBwd) {
                if (in) {
                    for (int j = lane; j < half; j += p.lanes) {  // b = R^T g, in place
                        const int i0 = kInterleaved ? 2 * j : j, i1 = kInterleaved ? 2 * j + 1 : j + half;
                        const float u = mine_g[i0], v = mine_g[i1];
                        mine_g[i0] = u * tc[j] + v * ts[j];
                        mine_g[i1] = v * tc[j] - u * ts[j];
                    }
                }
                __syncwarp();
                if (in)
                    for (int i = lane; i < d; i += p.lanes) ex = fmaf(mine_g[i] * w[i], mine[i], ex);
            }
            const float rn = inverse_root(fmaf(lanes_sum(ss, p.lanes), inv_d, p.eps));
            if constexpr (kBwd) {
                const float mean = rn * rn * lanes_sum(ex, p.lanes) * inv_d;
                if (in)
                    for (int i = lane; i < d; i += p.lanes) {
                        const float a = mine[i], u = mine_g[i];
                        dw[i] = fmaf(u, a * rn, dw[i]);
                        mine[i] = rn * fmaf(-mean, a, u * w[i]);
                    }
            } else if (in) {
                for (int j = lane; j < half; j += p.lanes) {
                    const int i0 = kInterleaved ? 2 * j : j, i1 = kInterleaved ? 2 * j + 1 : j + half;
                    const float u = mine[i0] * rn * w[i0], v = mine[i1] * rn * w[i1];
                    mine[i0] = u * tc[j] - v * ts[j];
                    mine[i1] = u * ts[j] + v * tc[j];
                }
                for (int i = p.rot + lane; i < d; i += p.lanes) mine[i] = mine[i] * rn * w[i];
            }
            __syncwarp();
            if (in) {
                T *row = y + (t0 + t) * p.ys[which] + static_cast<int64_t>(h) * d;
                if (p.vec_rows) {
                    for (int u = lane; u < d / V; u += p.lanes) {
                        float f[V];
#pragma unroll
                        for (int i = 0; i < V; i += 4) {
                            const float4 z = *reinterpret_cast<const float4 *>(mine + u * V + i);
                            f[i] = z.x, f[i + 1] = z.y, f[i + 2] = z.z, f[i + 3] = z.w;
                        }
                        *reinterpret_cast<uint4 *>(row + u * V) = pack16(f);
                    }
                } else {
                    for (int i = lane; i < d; i += p.lanes) row[i] = Elem<T>::from_f(mine[i]);
                }
            }
            if (pairs && ++chain >= kChain) fold();  // (a lane has the same channels throughout)
            __syncwarp();
        }
        if (pairs && t0 + blocks * tokens >= p.T) {
            fold();
            for (int i = lane; i < d; i += p.lanes) dw[i] = Pair{folded[i], folded[d + i]}.value();
        }
        __syncthreads();
    }
    if constexpr (kBwd) {
        const float *all = w + d + 2 * d;  // (dw of the first group)
        for (int i = threadIdx.x; i < d; i += kStagedThreads) {
            float s = 0.f;
            for (int k = 0; k < groups; ++k) s += all[k * span + i];
            p.part[static_cast<int64_t>(blockIdx.x) * d + i] = s;
        }
    }
}

// dw from the CTAs' sums: 32 channels of q or k per CTA, 32 warps that take every 32nd sum (eight: 1 us longer).  Sums are pairs
// of fp32: chains of some hundred plain additions lost as much as the threads' own (fp64 took 6 us longer).
constexpr int kWeightWarps = 32;
__global__ void __launch_bounds__(32 * kWeightWarps) norm_weights_kernel(const float *part, int64_t blocks_q, int64_t blocks_k, int d,
                                                                        float *dq, float *dk) {
    __shared__ Pair share[kWeightWarps][33];
    grid_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, first = blockIdx.x * 32;
    const bool k = blockIdx.y == 1;
    float *to = k ? dk : dq;
    if (!to) return;
    const float *from = part + (k ? blocks_q * d : 0);
    const int64_t n = k ? blocks_k : blocks_q;
    Pair s{0.f, 0.f};
    if (first + lane < d) {
#pragma unroll 8
        for (int64_t i = warp; i < n; i += kWeightWarps) s.add(from[i * d + first + lane]);
    }
    share[warp][lane] = s;
    __syncthreads();
    s = share[lane][warp];  // of channel first + warp
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float high = __shfl_xor_sync(0xffffffffu, s.high, o), low = __shfl_xor_sync(0xffffffffu, s.low, o);
        s.add(high);
        s.low += low;
    }
    if (lane == 0 && first + warp < d) to[first + warp] = s.value();
}

// CTAs of the gradient for q and k: as many as are resident, shared out by heads, but no more than there are groups of tokens.
int64_t groups_of(int64_t T, int tokens) { return (T + tokens - 1) / tokens; }
int64_t most_ctas(int sms, bool columns) { return static_cast<int64_t>(sms) * (columns ? kBwdPerSm : kStagedPerSm); }
constexpr int kSmsAtMost = 160;  // what the workspace allows for

template <typename T, bool kInterleaved, bool kBwd>
kda_status launch(NormParams p, bool columns, float *dwq, float *dwk, cudaStream_t s) {
    constexpr int V = Elem<T>::kVec;
    const int sms = sm_count() < kSmsAtMost ? sm_count() : kSmsAtMost;
    if (sms <= 0) return KDA_ERR_CUDA;
    const int threads = columns ? kNormThreads : kStagedThreads;
    const int want = columns ? (p.d / V + 1) / 2 : (p.d + 7) / 8;  // lanes with something to do
    p.lanes = columns ? 1 : 8;
    while (p.lanes < want && p.lanes < 32) p.lanes *= 2;
    const int groups = threads / p.lanes;
    // heads of a group of lanes (columns), rows of a CTA (staged): as many as leave four CTAs or so per SM, and at most kRounds
    const int64_t total = p.T * (p.H[0] + p.H[1]), part = total / (static_cast<int64_t>(sms) * 4 * groups);
    const int heads = static_cast<int>(part < 1 ? 1 : part > kRounds ? kRounds : part);
    const int64_t most_tokens = p.rot > 0 ? 8192 / p.rot : 64;     // 32 KB of sines and cosines
    int tokens = 1;
    bool fold = false;
    for (int i = 0; i < 2; ++i) {
        p.share[i] = 1;
        if (p.H[i] == 0) {
            p.tokens[i] = 1;
            p.blocks[i] = 0;
            continue;
        }
        while (p.share[i] < groups && (p.share[i] * heads < p.H[i] || groups / p.share[i] > most_tokens)) p.share[i] *= 2;
        int64_t n = groups / p.share[i];
        if (!columns) {
            n = static_cast<int64_t>(heads) * groups / p.H[i];
            n = n > most_tokens ? most_tokens : n;
            n = n < 1 ? 1 : n > 64 ? 64 : n;
        }
        p.tokens[i] = static_cast<int>(n);
        tokens = p.tokens[i] > tokens ? p.tokens[i] : tokens;
        p.blocks[i] = groups_of(p.T, p.tokens[i]);
        if (kBwd) {
            int64_t share_i = most_ctas(sms, columns) * p.H[i] / (p.H[0] + p.H[1]);
            share_i = share_i < 1 ? 1 : share_i;
            p.blocks[i] = p.blocks[i] < share_i ? p.blocks[i] : share_i;
            // rows of a group of lanes
            const int64_t rounds = groups_of(groups_of(p.T, p.tokens[i]), static_cast<int>(p.blocks[i]));
            const int64_t each = columns ? groups_of(p.H[i], p.share[i]) : groups_of(static_cast<int64_t>(p.tokens[i]) * p.H[i], groups);
            fold |= rounds * each > kChain;
        }
    }
    if (p.blocks[0] + p.blocks[1] > 0x7fffffffLL) return KDA_ERR_INVALID_ARGUMENT;
    const unsigned grid = static_cast<unsigned>(p.blocks[0] + p.blocks[1]);
    const int half = p.rot / 2;
    size_t smem = ((half + 1) & ~1) * 8 + 2 * static_cast<size_t>(tokens) * table_pitch(p.rot) * 4;
    if (columns) {
        const size_t sums = kBwd ? static_cast<size_t>(kNormThreads / 32) * p.d * 4 : 0;
        smem = smem > sums ? smem : sums;
        if (fold) {
            p.fold_at = static_cast<int>(smem / 4);
            smem += 2 * V * kNormThreads * sizeof(Pair);
        }
        auto go = [&](auto folds) {
            auto run = [&](auto layout) {
                constexpr auto kernel = norm_rope_kernel<T, decltype(layout)::value, kBwd, decltype(folds)::value>;
                return smem_opt_in<kernel>(64 * 1024) && launch_after(kernel, dim3(grid), kNormThreads, smem, s, p) == cudaSuccess;
            };
            if constexpr (!kInterleaved) return run(std::integral_constant<Layout, kHalves>{});
            else if (p.rot == p.d) return run(std::integral_constant<Layout, kNeighbours>{});
            else return run(std::integral_constant<Layout, kSomeNeighbours>{});
        };
        if (!(fold ? go(std::bool_constant<kBwd>{}) : go(std::false_type{}))) return KDA_ERR_CUDA;
    } else {
        p.fold_at = fold ? 1 : 0;
        smem += (static_cast<size_t>(p.d) + static_cast<size_t>(groups) * staged_span(kBwd, fold, p.d, p.lanes)) * 4;
        if (!smem_opt_in<norm_rope_staged_kernel<T, kInterleaved, kBwd>>(128 * 1024)) return KDA_ERR_CUDA;
        if (launch_after(norm_rope_staged_kernel<T, kInterleaved, kBwd>, dim3(grid), kStagedThreads, smem, s, p) != cudaSuccess)
            return KDA_ERR_CUDA;
    }
    if (kBwd && (dwq || dwk)) {
        const dim3 g(static_cast<unsigned>((p.d + 31) / 32), 2);
        const float *part = p.part;
        if (launch_after(norm_weights_kernel, g, 32 * kWeightWarps, 0, s, part, p.blocks[0], p.blocks[1], p.d, dwq, dwk) != cudaSuccess)
            return KDA_ERR_CUDA;
    }
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

struct NormArgs {
    const void *q, *k, *gq, *gk, *wq, *wk;
    void *yq, *yk;
    kda_dtype dtype, wdtype;
    const int32_t *positions;
    const double *inv_freq;
    int64_t T;
    int Hq, Hk, d, rot;
    int64_t qs, ks, gqs, gks, yqs, yks;
    int interleaved;
    float mscale, eps;
    float *dwq, *dwk;
    void *workspace;
    size_t ws_bytes;
    bool backward;
};

size_t bwd_workspace(int d) { return KDA_WS_HEADER_BYTES + static_cast<size_t>(most_ctas(kSmsAtMost, false) + 2) * d * sizeof(float); }

kda_status norm_rope(const NormArgs &a, void *stream) {
    if (!dtype_ok(a.dtype) || !dtype_ok(a.wdtype)) return KDA_ERR_UNSUPPORTED;
    const int d = a.d;
    if (d <= 0 || d % 8 != 0 || d > 1024) return KDA_ERR_UNSUPPORTED;
    if (a.rot < 0 || a.rot > d || a.rot % 2 != 0 || a.T < 0 || a.Hq <= 0 || a.Hk < 0 || a.Hq > 65536 || a.Hk > 65536)
        return KDA_ERR_INVALID_ARGUMENT;
    if (!(a.eps >= 0.f && a.eps < 3.0e38f)) return KDA_ERR_INVALID_ARGUMENT;
    const int Hk = a.k || a.T == 0 ? a.Hk : 0;  // (an empty tensor may have no address)
    const size_t es = elem_size(a.dtype), ws = elem_size(a.wdtype);
    const int64_t V = 16 / static_cast<int64_t>(es);
    bool vec = true;
    // a packed stride in the place of 0, and whether every row of the tensor is 16-byte aligned
    auto rows = [&](const void *ptr, int64_t stride, int H, int64_t *out) {
        const int64_t width = static_cast<int64_t>(H) * d;
        *out = stride ? stride : width;
        vec = vec && (H == 0 || (aligned_to(ptr, 16) && *out % V == 0));
        return H == 0 || (*out >= width && aligned_to(ptr, es) && (a.T == 0 || ptr));
    };
    NormParams p{};
    if (!rows(a.q, a.qs, a.Hq, &p.xs[0]) || !rows(a.k, a.ks, Hk, &p.xs[1]) || !rows(a.yq, a.yqs, a.Hq, &p.ys[0]) ||
        !rows(a.yk, a.yks, Hk, &p.ys[1]))
        return KDA_ERR_INVALID_ARGUMENT;
    if (a.backward && (!rows(a.gq, a.gqs, a.Hq, &p.gs[0]) || !rows(a.gk, a.gks, Hk, &p.gs[1]))) return KDA_ERR_INVALID_ARGUMENT;
    if (!aligned_to(a.wq, ws) || !aligned_to(a.wk, ws) || !aligned_to(a.dwq, 4) || !aligned_to(a.dwk, 4) || (a.dwk && !Hk))
        return KDA_ERR_INVALID_ARGUMENT;
    if (!aligned_to(a.positions, 4) || !aligned_to(a.inv_freq, 8) || (a.T > 0 && (!a.positions || (a.rot > 0 && !a.inv_freq))))
        return KDA_ERR_INVALID_ARGUMENT;
    if (a.backward && (!a.workspace || !aligned_to(a.workspace, 16) || a.ws_bytes < bwd_workspace(d))) return KDA_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (a.T == 0) {
        for (float *dw : {a.dwq, a.dwk})
            if (dw && cudaMemsetAsync(dw, 0, static_cast<size_t>(d) * 4, s) != cudaSuccess) return KDA_ERR_CUDA;
        return KDA_OK;
    }
    p.x[0] = a.q; p.x[1] = a.k; p.g[0] = a.gq; p.g[1] = a.gk; p.w[0] = a.wq; p.w[1] = a.wk; p.y[0] = a.yq; p.y[1] = a.yk;
    p.H[0] = a.Hq; p.H[1] = Hk;
    p.positions = a.positions; p.inv_freq = a.inv_freq; p.T = a.T; p.d = d; p.rot = a.rot;
    p.wide_w = a.wdtype == KDA_F32; p.vec_w = aligned_to(a.wq, 16) && aligned_to(a.wk, 16); p.vec_rows = vec; p.mscale = a.mscale; p.eps = a.eps;
    if (a.backward) p.part = reinterpret_cast<float *>(static_cast<char *>(a.workspace) + KDA_WS_HEADER_BYTES);
    const int inter = a.interleaved != 0;
    const bool columns = vec && d / V <= 64 && (inter || (a.rot / 2) % V == 0);
    auto go = [&](auto type) {
        using T = decltype(type);
        if (a.backward) return inter ? launch<T, true, true>(p, columns, a.dwq, a.dwk, s) : launch<T, false, true>(p, columns, a.dwq, a.dwk, s);
        return inter ? launch<T, true, false>(p, columns, nullptr, nullptr, s) : launch<T, false, false>(p, columns, nullptr, nullptr, s);
    };
    return a.dtype == KDA_BF16 ? go(__nv_bfloat16{}) : go(float{});
}

}  // namespace
}  // namespace kda

extern "C" {

kda_status kda_norm_rope(const void *q, const void *k, kda_dtype dtype, const void *q_weight, const void *k_weight, kda_dtype weight_dtype,
                         const int32_t *positions, const double *inv_freq, int64_t T, int Hq, int Hk, int d, int rot,
                         int64_t q_stride, int64_t k_stride, int interleaved, float mscale, float eps, void *q_out, void *k_out,
                         int64_t q_out_stride, int64_t k_out_stride, void *stream) {
    kda::NormArgs a{};
    a.q = q; a.k = k; a.wq = q_weight; a.wk = k_weight; a.yq = q_out; a.yk = k_out; a.dtype = dtype; a.wdtype = weight_dtype;
    a.positions = positions; a.inv_freq = inv_freq; a.T = T; a.Hq = Hq; a.Hk = Hk; a.d = d; a.rot = rot;
    a.qs = q_stride; a.ks = k_stride; a.yqs = q_out_stride; a.yks = k_out_stride; a.interleaved = interleaved;
    a.mscale = mscale; a.eps = eps;
    return kda::norm_rope(a, stream);
}

size_t kda_norm_rope_bwd_workspace_size(int d) { return d <= 0 || d % 8 != 0 || d > 1024 ? 0 : kda::bwd_workspace(d); }

kda_status kda_norm_rope_bwd(const void *q, const void *k, const void *d_q_out, const void *d_k_out, kda_dtype dtype, const void *q_weight,
                             const void *k_weight, kda_dtype weight_dtype, const int32_t *positions, const double *inv_freq,
                             int64_t T, int Hq, int Hk, int d, int rot, int64_t q_stride, int64_t k_stride, int64_t d_q_out_stride,
                             int64_t d_k_out_stride, int interleaved, float mscale, float eps, void *d_q, void *d_k,
                             int64_t d_q_stride, int64_t d_k_stride, float *d_q_weight, float *d_k_weight, void *workspace,
                             size_t ws_bytes, void *stream) {
    kda::NormArgs a{};
    a.q = q; a.k = k; a.gq = d_q_out; a.gk = d_k_out; a.wq = q_weight; a.wk = k_weight; a.yq = d_q; a.yk = d_k;
    a.dtype = dtype; a.wdtype = weight_dtype; a.positions = positions; a.inv_freq = inv_freq; a.T = T; a.Hq = Hq; a.Hk = Hk; a.d = d; a.rot = rot;
    a.qs = q_stride; a.ks = k_stride; a.gqs = d_q_out_stride; a.gks = d_k_out_stride; a.yqs = d_q_stride; a.yks = d_k_stride;
    a.interleaved = interleaved; a.mscale = mscale; a.eps = eps; a.dwq = d_q_weight; a.dwk = d_k_weight;
    a.workspace = workspace; a.ws_bytes = ws_bytes; a.backward = true;
    return kda::norm_rope(a, stream);
}

}  // extern "C"
