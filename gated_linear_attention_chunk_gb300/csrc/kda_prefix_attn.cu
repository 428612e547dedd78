// Attention of groups of sequences over the prefix that each group shares, joined with what the rows have from their own keys.
//
// The tokens of a group and the G = Hq / Hkv query heads of a KV head are the rows of one matrix product per KV head, so that
// the prefix's keys and values are read once for all of them.  One pass with a running maximum and sum per row (base-2
// exponentials of scale log2(e) q.k).  The work is cut evenly (kda_prefix_attn.cuh).  A unit (group, KV head, block of rows)
// that lies within one CTA is finished there; the parts of the others leave their sums, maximum and weight sum in the
// workspace, and join_kernel adds them in order.  So a result's bits depend on the batch's sizes, but not on chance.
//
// The keys' bytes bound it up to about 280 rows per KV head, the tensor cores beyond (bf16), the fp32 units (fp32).  Measured,
// 32 / 8 heads of 128, bf16: 16 prompts of up to 8,192 tokens with eight samples each 68 us (272 MB: 4.0 TB/s, 60% of the copy
// rate); one prompt of 131,072 with 512 tokens 845 us (1.3 PFLOP/s, 68% of measured); one prompt of 2,048 with eight 21 us
// (latency).  fp32, 3 prompts of up to 4,099, 45 tokens, 12 / 4 heads of 64: 36 us (latency).
//
// The plan checks the lengths and numbers the steps.  With more than kPlanGroups groups it is a launch of its own, otherwise
// every CTA makes it for itself.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_prefix_attn.cuh"

namespace kda {
namespace {

using namespace prefix;

constexpr int kPlanThreads = 256;
constexpr int kSmsAtMost = 160;  // what the workspace allows for

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PrefixParams p) {
    __shared__ PlanScratch scratch;
    grid_go();
    make_plan(p, scratch);
}

// ---------------------------------------------------------------------------------------------------------------
// fp32 (16 to 60 bytes of spills at two CTAs per SM): blocks of 64 rows against tiles of 64 keys on the fp32 units: a thread
// has 4 x 4 scores, then 4 rows of dv / 16 columns.  A tile's products are summed apart and then added to what there is, which
// keeps long sums as exact as short ones.
// ---------------------------------------------------------------------------------------------------------------
constexpr int kRows = 64, kKeys = 64, kThreads = 256;

// Values have a place of their own where two CTAs fit an SM all the same; otherwise they follow the keys into theirs.
template <int DK, int DV>
struct Tile {
    static constexpr int kPitchK = DK + 4, kPitchP = kKeys + 4;
    static constexpr bool kApart = 2 * 4 * (kRows * DK + kKeys * (kPitchK + DV) + kRows * kPitchP) <= 216 * 1024;
    static constexpr int kWide = kApart ? kPitchK + DV : kPitchK > DV ? kPitchK : DV;
    static constexpr int kFloats = kRows * DK + kKeys * kWide + kRows * kPitchP;
};

// 16 bytes into shared memory, zeros where there is nothing to read.
__device__ __forceinline__ void copy16(float *to, const float *from, bool there) {
    const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(to));
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(from), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory"); }

template <int DK, int DV>
__global__ void __launch_bounds__(kThreads, 2) prefix_kernel(const PrefixParams p) {
    using L = Tile<DK, DV>;
    using T = float;
    constexpr int V = Elem<T>::kVec, C = DV / 16;
    extern __shared__ __align__(16) float smem[];
    float *qs = smem, *ks = qs + kRows * DK, *vs = L::kApart ? ks + kKeys * L::kPitchK : ks, *ps = ks + kKeys * L::kWide;
    __shared__ int64_t row_k[2][kKeys], row_v[2][kKeys];  // of this tile and the next: offsets of the keys' and values' rows, -1: none
    static_assert(sizeof(PlanScratch) <= L::kFloats * 4, "the plan's scratch lies over the tiles");
    grid_wait();
    grid_go();
    if (!p.planned) make_plan(p, *reinterpret_cast<PlanScratch *>(smem));
    uint32_t met = 0;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const float c2 = p.scale * kLog2e;
    const T *kbase = reinterpret_cast<const T *>(p.c.k), *vbase = reinterpret_cast<const T *>(p.c.v), *base = static_cast<const T *>(p.q);
    SegmentWalk w;
    for (w.start(p); w.live(); w.next(p)) {
        const int64_t rows = static_cast<int64_t>(w.tokens) * p.G, r0 = static_cast<int64_t>(w.block) * kRows;
        // A tile's rows are looked up while the one before is worked on, and its keys, and values where they have a place,
        // copied ahead.  (16 prompts of up to 4,096, 16 samples each, 32 / 8 heads of 64: 192 us where they are waited for one
        // after the other, 153 so; of 128, 332 and 256.)
        auto look_up = [&](int t) {
            if (threadIdx.x >= kKeys || t >= w.k1) return false;
            const uint32_t j = static_cast<uint32_t>(t) * kKeys + threadIdx.x;
            int64_t a = -1, b = -1;
            bool wrong = false;
            if (j < static_cast<uint32_t>(w.len)) {
                const uint32_t pg = j / static_cast<uint32_t>(p.c.page_size);
                const int64_t slot = j - pg * p.c.page_size;
                const int page = p.c.table[w.g * p.c.table_stride + pg];
                wrong = page < 0 || page >= p.c.num_pages;
                if (!wrong) {
                    a = page * p.c.kp + slot * p.c.kr + w.head * p.c.kh;
                    b = page * p.c.vp + slot * p.c.vr + w.head * p.c.vh;
                }
            }
            row_k[t & 1][threadIdx.x] = a;
            row_v[t & 1][threadIdx.x] = b;
            return wrong;
        };
        auto copy_keys = [&](int t) {
            for (int i = threadIdx.x; i < kKeys * (DK / V); i += kThreads) {
                const int r = i / (DK / V), u = i - r * (DK / V);
                const int64_t from = row_k[t & 1][r];
                copy16(ks + r * L::kPitchK + u * V, from >= 0 ? kbase + from + u * V : base, from >= 0);
            }
            copies_commit();
        };
        auto copy_values = [&](int t) {
            for (int i = threadIdx.x; i < kKeys * (DV / V); i += kThreads) {
                const int r = i / (DV / V), u = i - r * (DV / V);
                const int64_t from = row_v[t & 1][r];
                copy16(vs + r * DV + u * V, from >= 0 ? vbase + from + u * V : base, from >= 0);
            }
            copies_commit();
        };
        __syncthreads();
        const bool wrong_first = look_up(w.k0);
        for (int i = threadIdx.x; i < kRows * (DK / V); i += kThreads) {
            const int r = i / (DK / V), u = i - r * (DK / V);
            const uint32_t at = static_cast<uint32_t>(r0) + r, tok = at / static_cast<uint32_t>(p.G);  // (T Hq is below 2^31)
            const bool there = r0 + r < rows;
            const T *from = base + (static_cast<int64_t>(w.t0) + tok) * p.qs + (w.head * p.G + static_cast<int>(at - tok * p.G)) * DK + u * V;
            copy16(qs + r * DK + u * V, there ? from : base, there);
        }
        uint32_t err = __syncthreads_or(wrong_first) ? DEV_ERR_PAGE : 0;
        copy_keys(w.k0);
        if (L::kApart) copy_values(w.k0);
        float m[4], l[4], o[4][C];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int j = 0; j < C; ++j) o[i][j] = 0.f;
        }
        for (int t = w.k0; t < w.k1; ++t) {
            const int key0 = t * kKeys, keys = w.len - key0 < kKeys ? w.len - key0 : kKeys;
            const bool more = t + 1 < w.k1;
            const bool wrong = look_up(t + 1);
            if (L::kApart) copies_wait<1>();
            else copies_wait<0>();
            if (__syncthreads_or(wrong)) err = DEV_ERR_PAGE;
            float s[4][4] = {};
#pragma unroll 4
            for (int k = 0; k < DK; k += 4) {
                float4 a[4], b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4 *>(qs + (ty * 4 + i) * DK + k);
#pragma unroll
                for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4 *>(ks + (tx + 16 * j) * L::kPitchK + k);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        s[i][j] = fmaf(a[i].x, b[j].x, fmaf(a[i].y, b[j].y, fmaf(a[i].z, b[j].z, fmaf(a[i].w, b[j].w, s[i][j]))));
            }
            float f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float top = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (tx + 16 * j < keys) top = fmaxf(top, s[i][j] * c2);
#pragma unroll
                for (int x = 8; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                top = fmaxf(top, m[i]);
                const float base = top == -INFINITY ? 0.f : top;
                f[i] = exp2f(m[i] - base);
                m[i] = top;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float e = tx + 16 * j < keys ? exp2f(fmaf(s[i][j], c2, -base)) : 0.f;
                    ps[(ty * 4 + i) * L::kPitchP + tx + 16 * j] = e;
                    sum += e;
                }
#pragma unroll
                for (int x = 8; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
                l[i] = fmaf(l[i], f[i], sum);
            }
            __syncthreads();
            if (!L::kApart) copy_values(t);
            else if (more) copy_keys(t + 1);
            if (L::kApart && more) copies_wait<1>();
            else copies_wait<0>();
            __syncthreads();
            float acc[4][C] = {};
#pragma unroll 2
            for (int k = 0; k < kKeys; k += 4) {
                float4 a[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4 *>(ps + (ty * 4 + i) * L::kPitchP + k);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    float v[C];
#pragma unroll
                    for (int j = 0; j < C; j += 4)
                        *reinterpret_cast<float4 *>(v + j) = *reinterpret_cast<const float4 *>(vs + (k + x) * DV + j * 16 + tx * 4);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float e = x == 0 ? a[i].x : x == 1 ? a[i].y : x == 2 ? a[i].z : a[i].w;
#pragma unroll
                        for (int j = 0; j < C; ++j) acc[i][j] = fmaf(e, v[j], acc[i][j]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < C; ++j) o[i][j] = fmaf(o[i][j], f[i], acc[i][j]);
            if (!more) continue;
            __syncthreads();
            if (L::kApart) copy_values(t + 1);
            else copy_keys(t + 1);
        }
        met |= err;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty * 4 + i;
            if (r0 + r >= rows || (err && w.whole)) continue;
            if (!w.whole) {
                const int64_t at = static_cast<int64_t>(w.slot) * p.pitch + r;
#pragma unroll
                for (int j = 0; j < C; j += 4)
                    *reinterpret_cast<float4 *>(p.part_o + at * DV + j * 16 + tx * 4) = make_float4(o[i][j], o[i][j + 1], o[i][j + 2], o[i][j + 3]);
                if (tx == 0) p.part_ml[at] = make_float2(m[i], err ? -1.f : l[i]);
                continue;
            }
            const int64_t tok = (r0 + r) / p.G, row = (w.t0 + tok) * p.Hq + w.head * p.G + (r0 + r - tok * p.G);
            const Join x = join_tail(m[i], l[i], p.lse_tail != nullptr, p.lse_tail ? p.lse_tail[row] : 0.f);
#pragma unroll
            for (int j = 0; j < C; ++j) {
                const int64_t at = row * DV + (j / 4) * 64 + tx * 4 + j % 4;
                float y = x.prefix != 0.f ? o[i][j] * x.prefix : 0.f;
                if (x.tail != 0.f) y = fmaf(x.tail, Elem<T>::to_f(static_cast<const T *>(p.o_tail)[at]), y);
                static_cast<T *>(p.o)[at] = Elem<T>::from_f(y);
            }
            __syncwarp(0xffffu << (threadIdx.x & 16));  // (lse may be lse_tail)
            if (tx == 0 && p.lse) p.lse[row] = x.lse;
        }
    }
    if (threadIdx.x == 0) p.errors[blockIdx.x] = met;
}

// The rows that no CTA has finished: a warp per (token, query head), the parts added in order.  What it reads of the call's
// inputs it reads before it waits for the kernel ahead.  That is safe because the kernel ahead lets it begin (grid_go) only
// after its own grid_wait, when everything before the call has ended; and because what it may read while that kernel writes,
// o_tail and lse_tail where they are o and lse, is of rows that kernel finishes itself (n == 1 below), and is dropped.  A row
// that is joined here is written here alone.
template <typename T, int DV>
__global__ void __launch_bounds__(128) join_kernel(const PrefixParams p) {
    constexpr int VL = DV / 32;
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const bool there = row < p.T * p.Hq;
    const int64_t tok = there ? row / p.Hq : 0;
    const int h = there ? static_cast<int>(row - tok * p.Hq) : 0;
    int g = warp_find([&](int i) { return p.cu[i]; }, p.N, tok);
    const bool has_tail = p.lse_tail != nullptr && there;
    const float lse_tail = has_tail ? p.lse_tail[row] : 0.f;
    float tail[VL] = {};
    if (has_tail) {
#pragma unroll
        for (int x = 0; x < VL; ++x) tail[x] = Elem<T>::to_f(static_cast<const T *>(p.o_tail)[row * DV + lane * VL + x]);
    }
    grid_wait();
    const GroupInfo all = p.info[p.N];
    GroupInfo s = p.info[g];
    if (blockIdx.x == 0 && threadIdx.x < 32) {  // the errors
        uint32_t met = static_cast<uint32_t>(all.tokens);
        for (int c = lane; c < p.ctas; c += 32) met |= p.errors[c];
        met = __reduce_or_sync(0xffffffffu, met);
        if (lane == 0) *p.status = met;
    }
    if (!there) return;
    if (tok < s.t0 || tok >= s.t0 + s.tokens) {  // behind the last group, or cu_tokens falls: then the plan's order counts
        if (all.tokens == 0) return;
        g = warp_find([&](int i) { return p.info[i].t0; }, p.N, tok);
        s = p.info[g];
        if (tok < s.t0 || tok >= s.t0 + s.tokens) return;
    }
    float m = -INFINITY, l = 0.f, o[VL] = {};
    if (s.tiles > 0) {
        const int64_t total = all.step0, r = (tok - s.t0) * p.G + h % p.G;
        const int block = static_cast<int>(r / p.rows), at = static_cast<int>(r - static_cast<int64_t>(block) * p.rows);
        const bool by_parts = all.parts != 0;
        // its slots (runs: one per CTA, whose second slot it is unless the CTA begins within the unit)
        int n;
        int64_t first;
        int c0 = 0;
        if (by_parts) {
            n = s.parts;
            first = s.step0 + static_cast<int64_t>(h / p.G) * s.parts * s.blocks + block;
        } else {
            const int lead = all.blocks;
            const int64_t s0 = s.step0 + (static_cast<int64_t>(h / p.G) * s.blocks + block) * (s.tiles + lead);
            c0 = cta_of(total, s0 + lead, p.ctas);
            n = cta_of(total, s0 + lead + s.tiles - 1, p.ctas) - c0 + 1;
            first = 2 * c0 + (first_step(total, c0, p.ctas) >= s0 ? 0 : 1);
        }
        if (n == 1) return;
        auto place = [&](int i) {
            const int64_t slot = by_parts ? first + static_cast<int64_t>(i) * s.blocks : i == 0 ? first : 2 * static_cast<int64_t>(c0 + i);
            return slot * p.pitch + at;
        };
        auto has = [&](int i) { return by_parts || first_step(total, c0 + i, p.ctas) < first_step(total, c0 + i + 1, p.ctas); };
        // a lane looks a part up, then all add it
        auto look = [&](int i) {
            float2 ml = make_float2(0.f, 0.f);
            if (i < n && has(i)) ml = p.part_ml[place(i)];
            return ml;
        };
        const float2 own = look(lane);
        bool bad = own.y < 0.f;
        m = own.y != 0.f ? own.x : -INFINITY;
        for (int i = 32 + lane; i < n; i += 32) {
            const float2 ml = look(i);
            if (ml.y != 0.f) m = fmaxf(m, ml.x);
            bad |= ml.y < 0.f;
        }
        if (__any_sync(0xffffffffu, bad)) return;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
        const float base = m == -INFINITY ? 0.f : m;
        for (int i0 = 0; i0 < n; i0 += 32) {
            const float2 ml = i0 == 0 ? own : look(i0 + lane);
            const float f = ml.y != 0.f ? exp2f(ml.x - base) : 0.f;
            const float fl = ml.y != 0.f ? f * ml.y : 0.f;
            const int64_t slot = i0 + lane < n ? place(i0 + lane) : 0;
            const uint32_t some = __ballot_sync(0xffffffffu, ml.y != 0.f);
            const int parts = n - i0 < 32 ? n - i0 : 32;
#pragma unroll 4
            for (int k = 0; k < parts; ++k) {
                const float fk = __shfl_sync(0xffffffffu, f, k);
                l += __shfl_sync(0xffffffffu, fl, k);
                const int64_t from = __shfl_sync(0xffffffffu, slot, k);
                if (!(some >> k & 1u)) continue;
#pragma unroll
                for (int x = 0; x < VL; x += 2) {
                    const float2 v = *reinterpret_cast<const float2 *>(p.part_o + from * DV + lane * VL + x);
                    o[x] = fmaf(fk, v.x, o[x]);
                    o[x + 1] = fmaf(fk, v.y, o[x + 1]);
                }
            }
        }
    }
    const Join j = join_tail(m, l, has_tail, lse_tail);
    T *to = static_cast<T *>(p.o) + row * DV + lane * VL;
#pragma unroll
    for (int x = 0; x < VL; ++x) {
        float y = j.prefix != 0.f ? o[x] * j.prefix : 0.f;
        if (j.tail != 0.f) y = fmaf(j.tail, tail[x], y);
        to[x] = Elem<T>::from_f(y);
    }
    if (lane == 0 && p.lse) p.lse[row] = j.lse;
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

struct Layout {
    size_t info, errors, part_ml, part_o, total;
};
int pitch_of(int64_t rows, int block) { return static_cast<int>(rows < block ? (rows + 7) / 8 * 8 : block); }
Layout layout_of(int N, int64_t T, int Hq, int Hkv, int dv) {
    Layout l{};
    size_t off = KDA_WS_HEADER_BYTES;
    auto take = [&](size_t bytes) { const size_t at = off; off = align256(off + bytes); return at; };
    l.info = take((static_cast<size_t>(N) + 1) * sizeof(GroupInfo));
    l.errors = take(2 * kSmsAtMost * 4);
    // bf16: one CTA per SM, two slots each, or up to kMostRounds parts where there is more than one block; fp32: two CTAs,
    // smaller blocks
    const int64_t rows = T * (Hq / Hkv), a = (rows > kTcBlock ? kMostRounds : 2) * pitch_of(rows, kTcBlock), b = 4 * pitch_of(rows, kRows);
    const size_t slots = static_cast<size_t>(kSmsAtMost) * (a > b ? a : b);
    l.part_ml = take(slots * sizeof(float2));
    l.part_o = take(slots * dv * sizeof(float));
    l.total = off;
    return l;
}

template <int DK, int DV>
kda_status launch_f32(const PrefixParams &p, cudaStream_t s) {
    constexpr int bytes = Tile<DK, DV>::kFloats * 4;
    if (!smem_opt_in<prefix_kernel<DK, DV>>(bytes)) return KDA_ERR_CUDA;
    return launch_after(prefix_kernel<DK, DV>, dim3(p.ctas), kThreads, bytes, s, p) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

template <typename T, int DV>
cudaError_t launch_join(const PrefixParams &p, cudaStream_t s) {
    return launch_after(join_kernel<T, DV>, dim3(static_cast<unsigned>((p.T * p.Hq + 3) / 4)), 128, 0, s, p);
}

kda_status launch(PrefixParams p, bool wide, int dk, int dv, cudaStream_t s) {
    int sms = sm_count();
    if (sms <= 0) return KDA_ERR_CUDA;
    sms = sms < kSmsAtMost ? sms : kSmsAtMost;
    if (wide) {
        p.ctas = 2 * sms;
        p.rows = kRows;
        p.tile_keys = kKeys;
    } else {
        p.ctas = sms;
        p.rows = kTcBlock;
        tc_cut(&p);
    }
    p.wide = wide;
    p.pitch = pitch_of(p.T * p.G, p.rows);
    p.planned = p.N > kPlanGroups;
    if (p.planned) plan_kernel<<<1, kPlanThreads, 0, s>>>(p);
    if (wide) {
        const kda_status st = dk == 128 ? (dv == 128 ? launch_f32<128, 128>(p, s) : launch_f32<128, 64>(p, s))
                                        : (dv == 128 ? launch_f32<64, 128>(p, s) : launch_f32<64, 64>(p, s));
        if (st != KDA_OK) return st;
    } else if (launch_prefix_tc(p, dk, dv, s) != cudaSuccess) {
        return KDA_ERR_CUDA;
    }
    const cudaError_t e = wide ? (dv == 128 ? launch_join<float, 128>(p, s) : launch_join<float, 64>(p, s))
                               : (dv == 128 ? launch_join<__nv_bfloat16, 128>(p, s) : launch_join<__nv_bfloat16, 64>(p, s));
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace
}  // namespace kda

extern "C" {

size_t kda_prefix_attn_workspace_size(int N, int64_t T, int Hq, int Hkv, int dv) {
    if (N < 0 || N > (1 << 20) || T < 0 || T > 0x7fffffffLL || Hq <= 0 || Hkv <= 0 || Hq > 4096 || Hq % Hkv || !kda::spec::dim_ok(dv)) return 0;
    return kda::layout_of(N, T, Hq, Hkv, dv).total;
}

kda_status kda_prefix_attn(const void *q, kda_dtype dtype, const kda_paged_kv *prefixes, const int32_t *cu_tokens, int N, int64_t T, int Hq,
                           int Hkv, int dk, int dv, int64_t q_stride, float scale, const void *o_tail, const float *lse_tail, void *o,
                           float *lse, void *workspace, size_t ws_bytes, void *stream) {
    using namespace kda::spec;
    if (!dtype_ok(dtype) || !dim_ok(dk) || !dim_ok(dv)) return KDA_ERR_UNSUPPORTED;
    if (N < 0 || N > (1 << 20) || T < 0 || T > 0x7fffffffLL || Hq <= 0 || Hkv <= 0 || Hq > 4096 || Hq % Hkv || T * Hq > 0x7fffffffLL)
        return KDA_ERR_INVALID_ARGUMENT;
    Pages c;
    const kda_status st = check_pages(prefixes, dtype, N, &c);
    if (st != KDA_OK) return st;
    if (c.page_size > 1 && (c.kr < dk || c.vr < dv)) return KDA_ERR_INVALID_ARGUMENT;
    const int64_t vec = 16 / static_cast<int64_t>(elem_size(dtype));
    if (!q_stride) q_stride = static_cast<int64_t>(Hq) * dk;
    if (q_stride < static_cast<int64_t>(Hq) * dk || q_stride % vec) return KDA_ERR_INVALID_ARGUMENT;
    if (N > 0 && (!cu_tokens || !aligned_to(cu_tokens, 4))) return KDA_ERR_INVALID_ARGUMENT;
    if (T > 0 && (!q || !o || !o_tail != !lse_tail)) return KDA_ERR_INVALID_ARGUMENT;
    if (!aligned_to(q, 16) || !aligned_to(o, 16) || !aligned_to(o_tail, 16) || !aligned_to(lse, 4) || !aligned_to(lse_tail, 4))
        return KDA_ERR_INVALID_ARGUMENT;
    const kda::Layout l = kda::layout_of(N, T, Hq, Hkv, dv);
    if (!workspace || !aligned_to(workspace, 16) || ws_bytes < l.total) return KDA_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (N == 0 || T == 0) return cudaMemsetAsync(workspace, 0, sizeof(uint32_t), s) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
    char *ws = static_cast<char *>(workspace);
    kda::prefix::PrefixParams p{};
    p.q = q; p.o_tail = o_tail; p.lse_tail = lse_tail; p.o = o; p.lse = lse; p.c = c; p.cu = cu_tokens;
    p.T = T; p.qs = q_stride; p.N = N; p.Hq = Hq; p.Hkv = Hkv; p.G = Hq / Hkv; p.scale = scale;
    p.status = reinterpret_cast<uint32_t *>(ws);
    p.info = reinterpret_cast<kda::prefix::GroupInfo *>(ws + l.info);
    p.errors = reinterpret_cast<uint32_t *>(ws + l.errors);
    p.part_ml = reinterpret_cast<float2 *>(ws + l.part_ml);
    p.part_o = reinterpret_cast<float *>(ws + l.part_o);
    return kda::launch(p, dtype == KDA_F32, dk, dv, s);
}

}  // extern "C"
