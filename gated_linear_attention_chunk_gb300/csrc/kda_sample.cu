// Tokens drawn from logits by given uniform numbers, after temperature, top-k, top-p and min-p, and the filtered distributions.
//
// With M the row's largest logit and e_i = exp((l_i - M) / t), the tokens are put in the order of K_i = (l_i descending, i
// ascending).  Every filter keeps a first run of that order: top-k its first k, top-p the shortest run of those with a mass of
// p of theirs, min-p the e_i >= min_p.  So the filters come down to one limit K*, and the token is the lowest i
// with sum_{j <= i, K_j <= K*} e_j > u sum_{K_j <= K*} e_j.
//
// One cluster of CTAs per row; the row's bytes, read once, are the floor (the later passes over it find it in L2).  To find K*
// the tokens are counted in 4096 bins by distance from M.
//   top-k: the counts tell the bin of the k-th token.  The tokens up to it, if they are at most 2048, are sorted by one CTA,
//          which takes all further steps on them.
//   top-p: a bin's count and the sum of its tokens' places in it estimate its mass to about 10^-3, which brackets the bins that
//          the border is in (a few of 4096).  One pass over the row sums all masses and those before the bracket, warp by warp, and lists
//          the tokens of the bracket (up to 2048), which one CTA sorts.  Whether the border is among them is seen from these sums.
//   otherwise (a flat or narrow distribution, thousands of equal logits): 2048 bins with exact counts and masses, and the bin
//          that the rank or the mass falls into is cut into 2048 bins of K again until 2048 tokens are left.
//
// Precision: the answers are whole numbers, so a rounding shows only next to a border, where a flat distribution over 10^5
// tokens has one every 10^-5.  Masses are 64-bit integers in units of 2^-44 of the largest (2^-(63 - b) for 2^b tokens where
// b > 19): their sums are exact, whatever the order, so that neither atomics nor the cluster's size change a result.  What a mass
// is made of is 2^x, x = (l - M) log2(e) / t to about 2^-33, from a table of 2^(i/256) and a cubic: off by about 2e-10 of
// itself.  Then it is rounded to a unit, by 2^-45 of the largest up to 2^19 tokens: of a flat tail of V tokens that far down
// all may go the same way, 2^-26 of the largest together at 2^19 and 2^-16 at 2^24 (64-bit sums have no room for finer units).
//
// The arithmetic of the masses bounds a call without top-k (30 operations per token, two tokens at a time where there are such
// instructions): 512 rows of 131,072 in bf16 by temperature alone take 113 us (issue 57% busy, 1.2 TB/s; 38 to 42 bytes of
// spills at 64 registers).  With filters it is the steps between the passes as well: a CTA has 64 tokens per thread of such a
// row, and spends about as many instructions on sums over warps and cluster.  128 rows of 131,072, fp32: 112 us with top-p, 73
// with top-k below 200, 30 greedy; 256 rows of 100,003 in bf16 with all distributions written 172 to 183 with filters and 113
// without (54 of them the draw); one row of 32,001 11 to 18 (cluster barriers). Tried and not kept: rows through a ring of
// asynchronous copies (slower: the passes do not wait for memory), two to four columns ahead in registers (109 to 116 us for
// 112, spills), counting threads' maxima before tokens for top-k (top-k 73 -> 64 us, but top-p 112 -> 119: the registers), a
// cluster's size by waves (see launch_sample).
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_f32x2.cuh"
#include "kda_spec.cuh"

namespace cg = cooperative_groups;

namespace kda {
namespace {

using namespace spec;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kCoarse = 4096;      // bins of counts
constexpr int kBins = 2048;        // bins of counts and masses
constexpr int kList = 2048;        // tokens that are put in order by sorting
constexpr int kPer = kList / kThreads;
constexpr int kMaxCluster = 8;
constexpr float kSpan = 20.f;      // the bins cover distances from M of up to 20 t, the last one has the rest
// With top-k they cover 40 at least: likely tokens at low temperatures leave the k-th far behind them.  (128 rows of 131,072
// whose other tokens lie 20 t and more below three: 184 us the general way, 75 so.)
constexpr float kRankSpan = 40.f;
constexpr float kHottest = 1e30f;  // higher temperatures count as this one
static_assert(3 * kBins >= kCoarse && 3 * kBins * 4 >= kList * 8, "all lie over the bins");

// 2^(i / 256) as th (1 + tl), the exponential's series in fp64.  th's bits come without i << 15: see weigh2.
struct Exp2Table {
    uint32_t th[256];
    float tl[256];
};
constexpr Exp2Table make_exp2_table() {
    Exp2Table t{};
    for (int i = 0; i < 256; ++i) {
        const double x = i * 0.69314718055994530942 / 256;
        double term = 1, sum = 1;
        for (int k = 1; k < 24; ++k) {
            term *= x / k;
            sum += term;
        }
        const uint32_t mant = static_cast<uint32_t>((sum - 1) * 8388608.0 + 0.5);  // 2^23
        const double high = 1 + mant / 8388608.0;
        t.th[i] = 0x3f800000u + mant - (static_cast<uint32_t>(i) << 15);
        t.tl[i] = static_cast<float>(sum / high - 1);
    }
    return t;
}
__device__ constexpr Exp2Table kExp2 = make_exp2_table();

struct SampleParams {
    const void *logits;
    void *probs;
    int64_t ls, ps;              // row strides in elements
    const float *u, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    int32_t *token;
    int V, slice;                // slice: 16-byte columns of a CTA
    int extra;                   // bits that a unit of mass is larger than 2^-44
    int place_bits, count_shift; // a bin's word: the sum of its tokens' places of so many bits, and from bit count_shift on their number
    bool wide_probs;
};

// The bin that a rank or a mass falls into.
struct Found {
    uint64_t mass_before;        // of the bins before the one
    int64_t count_before;
    int bin, count;              // count: the tokens in it
};

// A row's constants.
struct RowConst {
    float top;                   // M
    float sub;                   // x = (l - sub) log2(e) / t - a: sub is M where M log2(e) / t >= 128 (the difference is then exact
    float cut;                   //   wherever there is a mass), else 0; l - sub counts as at least cut, which has no mass
    float c_hi, c_lo;            // log2(e) / t as a pair
    float a_hi, a_lo;            // a as a pair, a_hi a multiple of 2^-16
    float low;                   // the lowest logit that min_p keeps
    float bin_scale;             // bins per unit of distance
};

// What the CTAs of a cluster tell one another: [r] is written by CTA r into every CTA's copy, then comes a barrier.
struct Shared {
    float top[kMaxCluster];                     // largest logit
    uint32_t best[kMaxCluster];                 // its lowest index (greedy)
    int64_t part_count[kMaxCluster];            // tokens in the CTA's share of the bins
    uint64_t part_mass[kMaxCluster];
    float part_about[kMaxCluster];              // about its mass
    int4 bracket[kMaxCluster];                  // within its share: first and last bin, tokens before the first and up to the last
    uint64_t key_min[kMaxCluster], key_max[kMaxCluster];    // of the tokens in a bin
    uint64_t total[kMaxCluster], above[kMaxCluster];        // mass of the CTA's tokens; of those before the bracket
    uint64_t kept[kMaxCluster];                 // of the kept ones
    Found found;                                // written by the CTA that has the bin
    uint64_t limit, limit_mass;                 // K* and the mass up to it, by the first CTA
    int listed;                                 // tokens in the first CTA's list
    // the CTA's own
    int own_listed, own_first;
    double min_shift;                           // t ln(min_p)
    uint64_t warp_mass[kWarps], warp_above[kWarps];
    int64_t warp_count[kWarps];
    float warp_top[kWarps], warp_about[kWarps];
    int4 warp_bracket[kWarps];
    uint64_t warp_key[2][kWarps];
    uint64_t list_mass[kThreads / 4];
    uint2 table[256];
};

constexpr int kSmemBytes = 3 * kBins * 4 + kList * 8 + static_cast<int>(sizeof(Shared));

// l's place in the order: larger logits first, then lower indices (-0 and 0 are equal).
__device__ __forceinline__ uint64_t key_of(float l, uint32_t index) {
    uint32_t b = __float_as_uint(l + 0.f);
    b = b & 0x80000000u ? ~b : b | 0x80000000u;
    return (static_cast<uint64_t>(~b) << 32) | index;
}
__device__ __forceinline__ float logit_of(uint64_t key) {
    const uint32_t b = ~static_cast<uint32_t>(key >> 32);
    return __uint_as_float(b & 0x80000000u ? b & 0x7fffffffu : ~b);
}

constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer, in the low bits
constexpr uint32_t kMagicBits = 0x4B400000u;

// e of two logits as high (1 + rel), rel below 2^-9, and its rounded value.
struct Exp2Parts {
    F2 high, rel, value;
};
__device__ __forceinline__ Exp2Parts exp2_parts(float l0, float l1, const RowConst &c, const uint2 *table) {
    const F2 minus = f2(-1.f);
    const float2 d = both(add2(f2(l0, l1), f2(-c.sub)));
    const F2 l = f2(fmaxf(d.x, c.cut), fmaxf(d.y, c.cut));  // (NaN becomes cut as well)
    // x = h + h_lo + l c_lo - a_hi - a_lo, rounded to n / 256; h - (a_hi + n / 256) is exact
    const F2 h = mul2(l, f2(c.c_hi)), h_lo = fma2(l, f2(c.c_hi), mul2(h, minus));
    const F2 t = fma2(add2(h, f2(-c.a_hi)), f2(256.f), f2(kMagic));
    const F2 b = fma2(add2(t, f2(-kMagic)), f2(1.f / 256.f), f2(c.a_hi));
    const F2 f = add2(fma2(b, minus, h), add2(fma2(l, f2(c.c_lo), h_lo), f2(-c.a_lo)));  // |f| <= 2^-9 or so
    // 2^f - 1: ln 2, its square / 2, its cube / 6
    const F2 poly = fma2(f, fma2(f, f2(0.0555041087f), f2(0.240226507f)), f2(0.693147181f));
    const float2 tt = both(t);
    const uint32_t j0 = __float_as_uint(tt.x), j1 = __float_as_uint(tt.y);
    const uint2 e0 = table[j0 & 255u], e1 = table[j1 & 255u];
    Exp2Parts r;
    // j << 15 is the exponent's step and i << 15, which the table's entry is without
    r.high = f2(__uint_as_float(e0.x + (j0 << 15)), __uint_as_float(e1.x + (j1 << 15)));
    r.rel = fma2(f, poly, f2(__uint_as_float(e0.y), __uint_as_float(e1.y)));
    r.value = fma2(r.high, r.rel, r.high);
    return r;
}
// Masses in two parts, of 2^22 units and of one; sums carry kMagicBits per token.
struct Parts {
    uint32_t high, low;
};
struct Parts2 {
    Parts p[2];
};
__device__ __forceinline__ Parts2 weigh2(float l0, float l1, const RowConst &c, const uint2 *table, float unit) {
    const Exp2Parts e = exp2_parts(l0, l1, c, table);
    const F2 magic = f2(kMagic), t = fma2(e.value, f2(4194304.f), magic);
    const F2 rest = fma2(add2(t, f2(-kMagic)), f2(-1.f / 4194304.f), e.high);  // exact
    const F2 low = fma2(fma2(e.high, e.rel, rest), f2(unit), magic);
    const float2 a = both(t), b = both(low);
    return Parts2{{{__float_as_uint(a.x), __float_as_uint(b.x)}, {__float_as_uint(a.y), __float_as_uint(b.y)}}};
}

// The cluster barrier in two halves, each run by converged warps.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

extern __shared__ __align__(16) char sample_smem[];

template <typename T>
struct Sampler {
    static constexpr int W = Elem<T>::kVec;
    const SampleParams &p;
    cg::cluster_group cluster;
    int C, rank, warp, lane;
    // Shared memory.
    // [kBins] each; together the kCoarse counts
    static __device__ __forceinline__ uint32_t *count() { return reinterpret_cast<uint32_t *>(sample_smem); }
    static __device__ __forceinline__ uint32_t *mass_lo() { return count() + kBins; }
    static __device__ __forceinline__ uint32_t *mass_hi() { return count() + 2 * kBins; }
    // [kList]: tokens of this CTA, or of all in the first one; the second list lies over the bins
    static __device__ __forceinline__ uint64_t *list() { return reinterpret_cast<uint64_t *>(sample_smem + 3 * kBins * 4); }
    static __device__ __forceinline__ uint64_t *list2() { return reinterpret_cast<uint64_t *>(sample_smem); }
    static __device__ __forceinline__ Shared &shared() { return *reinterpret_cast<Shared *>(sample_smem + 3 * kBins * 4 + kList * 8); }
    const T *row;
    int shift, col0, cols, span;           // elements before the row in its first column; columns; of a warp
    RowConst c;
    bool inf_top;                          // M is +inf: such logits count as 0 and all others as -inf
    float unit;                            // units of mass in one

    __device__ __forceinline__ uint4 fetch(int i) const {                   // column col0 + i; what is not in the row is -inf
        const int e = (col0 + i) * W - shift;  // (V is at most 2^24)
        if (e >= 0 && e + W <= p.V) return *reinterpret_cast<const uint4 *>(row + e);
        float f[W];
#pragma unroll
        for (int j = 0; j < W; ++j) f[j] = e + j >= 0 && e + j < p.V ? Elem<T>::to_f(row[e + j]) : -INFINITY;
        return pack16(f);
    }
    __device__ __forceinline__ void unpack(uint4 x, float (&f)[W]) const {
        unpack16(x, f);
        if (inf_top) {
#pragma unroll
            for (int j = 0; j < W; ++j) f[j] = f[j] == INFINITY ? 0.f : -INFINITY;
        }
    }
    // This warp's columns, a lane's next to one another's, the next one on its way: f(column, logits) until it says no.
    template <typename F>
    __device__ __forceinline__ void columns(F f) const {
        const int end = min(cols, (warp + 1) * span);
        int i = warp * span + lane;
        uint4 next = make_uint4(0u, 0u, 0u, 0u);
        if (i < end) next = fetch(i);
        for (; i < end; i += 32) {
            const uint4 now = next;
            if (i + 32 < end) next = fetch(i + 32);
            float x[W];
            unpack(now, x);
            f(i, x);
        }
    }
    __device__ __forceinline__ uint32_t index_of(int i) const { return static_cast<uint32_t>((col0 + i) * W - shift); }
    // Every element that can be drawn at all: f(logit, index).
    template <typename F>
    __device__ __forceinline__ void each(F f) const {
        columns([&](int i, const float (&x)[W]) {
            const uint32_t at = index_of(i);
#pragma unroll
            for (int j = 0; j < W; ++j)
                if (x[j] > -INFINITY) f(x[j], at + j);
        });
    }
    __device__ __forceinline__ uint64_t whole(uint32_t high, uint32_t low, uint32_t tokens) const {  // sums of Parts without their kMagicBits
        const int64_t l = static_cast<int32_t>(low - tokens * kMagicBits);
        return (static_cast<uint64_t>(high - tokens * kMagicBits) << (22 - p.extra)) + static_cast<uint64_t>(l);
    }
    __device__ __forceinline__ uint64_t mass_of(float l) const {
        const Parts2 m = weigh2(l, l, c, shared().table, unit);
        return whole(m.p[0].high, m.p[0].low, 1);
    }
    // Sums of masses; the parts are 32 bits wide and are taken over after at most 512 tokens.
    struct Sum {
        Parts parts{0, 0};
        uint32_t tokens = 0;
        uint64_t total = 0;
    };
    __device__ __forceinline__ void add(Sum &x, const Parts &m) const {
        x.parts.high += m.high;
        x.parts.low += m.low;
        ++x.tokens;
    }
    __device__ __forceinline__ void take_over(Sum &x, uint32_t at) const {
        if (x.tokens < at) return;
        x.total += whole(x.parts.high, x.parts.low, x.tokens);
        x.parts = Parts{0, 0};
        x.tokens = 0;
    }
    // The masses of what `keep` leaves of this thread's tokens.
    template <typename F>
    __device__ __forceinline__ uint64_t sum_masses(F keep) const {
        Sum sum;
        columns([&](int i, float (&x)[W]) {
            if (!keep(x, index_of(i))) return;
#pragma unroll
            for (int j = 0; j < W; j += 2) {
                const Parts2 m = weigh2(x[j], x[j + 1], c, shared().table, unit);
                add(sum, m.p[0]);
                add(sum, m.p[1]);
            }
            take_over(sum, 504);
        });
        take_over(sum, 0);
        return sum.total;
    }
    template <typename X>
    __device__ __forceinline__ X *of(X *ptr, int r) { return cluster.map_shared_rank(ptr, r); }
    // x as entry `rank` of an array in every CTA; by a converged warp whose lanes all have it.
    template <typename X>
    __device__ __forceinline__ void tell(X *entries, X x) {
        if (lane < C) *of(entries + rank, lane) = x;
    }
    // Over the warps' entries: the sum of those before this warp's, and of all.
    template <typename X>
    __device__ __forceinline__ void over_warps(const X *entries, X *before, X *all) const {
        X x = lane < kWarps ? entries[lane] : X(0), y = lane < warp ? x : X(0);
#pragma unroll
        for (int o = kWarps / 2; o > 0; o >>= 1) {
            x += __shfl_xor_sync(0xffffffffu, x, o);
            y += __shfl_xor_sync(0xffffffffu, y, o);
        }
        *all = __shfl_sync(0xffffffffu, x, 0);
        *before = __shfl_sync(0xffffffffu, y, 0);
    }
    __device__ __forceinline__ uint64_t warp_total(uint64_t x) const {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        return x;
    }

    __device__ __forceinline__ float distance(float l) const { return (c.top - l) * c.bin_scale; }  // in bins
    __device__ __forceinline__ int bin_of(float l) const { return static_cast<int>(fminf(distance(l) * 0.5f, kBins - 1.f)); }

    // ---- counts in kCoarse bins: running counts of the CTA's share of them; with a share of the mass, the bins that its border is
    // probably in (to < 0: none) and the tokens in them ----
    int before_n;            // tokens in the shares before this CTA's
    __device__ void tally_counts(float share, int *from, int *to, int *tokens) {
        for (int i = threadIdx.x; i < kCoarse; i += kThreads) count()[i] = 0u;
        if (threadIdx.x == 0) shared().listed = shared().own_listed = 0;
        __syncthreads();
        const float places = static_cast<float>(1 << p.place_bits), most = static_cast<float>((kCoarse << p.place_bits) - 1);
        const float scale = c.bin_scale * places;  // (exact: bins and places are cut at the same points as by distance())
        const uint32_t mask = (1u << p.place_bits) - 1u, one = 1u << p.count_shift;
        // Tokens beyond the last place are counted by each thread for itself: they would all meet at one word.  (128 rows of
        // 131,072, top-p: 120 us where they are counted like the others, 112 so; where all but three tokens lie there 150 and
        // 89.)
        uint32_t far = 0;
        columns([&](int, const float (&x)[W]) {
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const float d = (c.top - x[j]) * scale;
                // rounded down, in the low bits
                const uint32_t at = __float_as_uint(__fadd_rd(d, 8388608.f)) & 0x7fffffu;
                if (d < most) atomicAdd(count() + (at >> p.place_bits), one + (at & mask));
                else far += x[j] > -INFINITY ? 1u : 0u;
            }
        });
        far = __reduce_add_sync(0xffffffffu, far);
        if (lane == 0 && far > 0) atomicAdd(count() + kCoarse - 1, far * (one + mask));
        cluster.sync();
        // 8 / C bins per thread, each from C CTAs: eight reads on their way together
        constexpr int kMost = kCoarse / kThreads;
        static_assert(kMost == kMaxCluster, "a read per CTA and bin");
        const int mine = kCoarse / C, first = rank * mine, per = kMost / C;
        uint32_t got[kMost], n[kMost];
        float about[kMost];
#pragma unroll
        for (int x = 0; x < kMost; ++x) got[x] = *of(count() + first + threadIdx.x * per + x / C, x % C);
        uint32_t sum = 0;
        float mass = 0.f;
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
            uint32_t here = 0, place = 0;
            if (i < per) {
#pragma unroll
                for (int x = 0; x < kMost; ++x)
                    if (x / C == i) {
                        here += got[x] >> p.count_shift;
                        place += got[x] & (one - 1u);
                    }
                // its tokens at the middle of their places
                const float d = static_cast<float>(first + threadIdx.x * per + i) +
                                (__fdividef(static_cast<float>(place), static_cast<float>(here)) + 0.5f) / places;
                if (here > 0) mass = fmaf(static_cast<float>(here), exp2f(d * (-kSpan / kCoarse * 1.44269504f)), mass);
                sum += here;
            }
            n[i] = sum;
            about[i] = mass;
        }
        uint32_t upto = sum;
        float upto_mass = mass;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
            const float ym = __shfl_up_sync(0xffffffffu, upto_mass, o);
            if (lane >= o) upto += y, upto_mass += ym;
        }
        if (lane == 31) shared().warp_count[warp] = upto, shared().warp_about[warp] = upto_mass;
        __syncthreads();
        int64_t bn, tn;
        float bm, tm;
        over_warps(shared().warp_count, &bn, &tn);
        over_warps(shared().warp_about, &bm, &tm);
        bn += upto - sum;
        bm += upto_mass - mass;
        if (warp == 0) {
            tell(shared().part_count, tn);
            tell(shared().part_about, tm);
        }
        cluster.sync();
        int before = 0;
        float all = 0.f;
        total_n = 0;
        for (int r = 0; r < C; ++r) {
            if (r < rank) before += static_cast<int>(shared().part_count[r]), bm += shared().part_about[r];
            total_n += shared().part_count[r], all += shared().part_about[r];
        }
        before_n = before;
        *to = -1;
        *tokens = 0;
        // (every CTA has read the words by now)
#pragma unroll
        for (int i = 0; i < kMost; ++i)
            if (i < per) count()[first + threadIdx.x * per + i] = static_cast<uint32_t>(bn) + n[i];
        if (share <= 0.f) {
            __syncthreads();
            return;
        }
        // a token is at most half a place off, and the sums have their roundings
        const float slack = 1.5e-4f + kSpan / kCoarse * 0.5f / places;
        const float least = share * all * (1.f - slack), most_mass = share * all * (1.f + slack);
        int4 x = make_int4(kCoarse, -1, 0, 0);
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
            if (i >= per) continue;
            const uint32_t below = i ? n[i - 1] : 0u;
            const float low = bm + (i ? about[i - 1] : 0.f), high = bm + about[i];
            if (n[i] == below || !(low < most_mass) || !(high >= least)) continue;
            const int b = first + threadIdx.x * per + i;
            if (x.y < 0) x.x = b, x.z = before + static_cast<int>(static_cast<uint32_t>(bn) + below);
            x.y = b;
            x.w = before + static_cast<int>(static_cast<uint32_t>(bn) + n[i]);
        }
        auto join = [](int4 a, int4 y) {
            if (y.y < 0) return a;
            if (a.y < 0) return y;
            return make_int4(min(a.x, y.x), max(a.y, y.y), min(a.z, y.z), max(a.w, y.w));
        };
        auto across = [&](int4 a) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                a = join(a, make_int4(__shfl_xor_sync(0xffffffffu, a.x, o), __shfl_xor_sync(0xffffffffu, a.y, o),
                                      __shfl_xor_sync(0xffffffffu, a.z, o), __shfl_xor_sync(0xffffffffu, a.w, o)));
            return a;
        };
        x = across(x);
        if (lane == 0) shared().warp_bracket[warp] = x;
        __syncthreads();
        if (warp == 0) tell(shared().bracket, across(lane < kWarps ? shared().warp_bracket[lane] : make_int4(kCoarse, -1, 0, 0)));
        cluster.sync();
        x = shared().bracket[0];
        for (int r = 1; r < C; ++r) x = join(x, shared().bracket[r]);
        *from = x.x;
        *to = x.y;
        *tokens = x.w - x.z;
    }
    // The bin of the k-th token in every CTA's shared().found; count: all tokens up to the end of it.
    __device__ Found locate_rank(int k) {
        const int mine = kCoarse / C, first = rank * mine;
        for (int b = first + threadIdx.x; b < first + mine; b += kThreads) {
            const int cb = before_n + (b > first ? static_cast<int>(count()[b - 1]) : 0), cu = before_n + static_cast<int>(count()[b]);
            if (cb < k && k <= cu)
                for (int r = 0; r < C; ++r) *of(&shared().found, r) = Found{0, cb, b, cu};
        }
        cluster.sync();
        return shared().found;
    }
    // A list of n keys, sorted by this CTA.  Thread t has the places t, t + 512, ..: neighbours up to 16 apart are in one warp.
    __device__ void sort(uint64_t *keys, int n) const {
        int size = 32;
        while (size < n) size *= 2;
        __syncthreads();
        uint64_t v[kPer];
#pragma unroll
        for (int y = 0; y < kPer; ++y) {
            const int i = threadIdx.x + y * kThreads;
            v[y] = i < n ? keys[i] : ~0ull;
        }
        for (int k = 2; k <= size; k <<= 1)
            for (int j = k >> 1; j > 0; j >>= 1) {
                if (j >= 32) {
                    __syncthreads();
#pragma unroll
                    for (int y = 0; y < kPer; ++y)
                        if (threadIdx.x + y * kThreads < size) keys[threadIdx.x + y * kThreads] = v[y];
                    __syncthreads();
                }
#pragma unroll
                for (int y = 0; y < kPer; ++y) {
                    const int i = threadIdx.x + y * kThreads;
                    if (y > 0 && y * kThreads >= size) continue;
                    uint64_t other;
                    if (j >= 32) other = i < size ? keys[i ^ j] : ~0ull;
                    else other = __shfl_xor_sync(0xffffffffu, v[y], j);
                    const bool low = ((i & j) == 0) == ((i & k) == 0);  // keeps the smaller
                    v[y] = low == (other < v[y]) ? other : v[y];
                }
            }
        __syncthreads();
#pragma unroll
        for (int y = 0; y < kPer; ++y)
            if (threadIdx.x + y * kThreads < size) keys[threadIdx.x + y * kThreads] = v[y];
        __syncthreads();
    }
    // Running sums over at most kList values, kPer neighbours per thread: m becomes the sum up to and with each.  For the whole
    // CTA.
    __device__ uint64_t scan(uint64_t (&m)[kPer]) {
        uint64_t own = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) own += m[i];
        uint64_t sum = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        __syncthreads();
        if (lane == 31) shared().warp_mass[warp] = sum;
        __syncthreads();
        uint64_t before, all;
        over_warps(shared().warp_mass, &before, &all);
        before += sum - own;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            before += m[i];
            m[i] = before;
        }
        return all;
    }
    // x in [0, 1) as 64 bits behind the point.
    static __device__ __forceinline__ uint64_t fraction(float x) {
        const uint32_t b = __float_as_uint(x), e = b >> 23;
        const uint64_t m = e ? (b & 0x7fffffu) | 0x800000u : b;  // x = m 2^(max(e, 1) - 150)
        const int by = static_cast<int>(e ? e : 1u) - 86;
        return by >= 0 ? m << by : by > -64 ? m >> -by : 0;
    }
    // The smallest mass that is at least share times `mass`.
    __device__ __forceinline__ uint64_t share_of(float share, uint64_t mass) const {
        const uint64_t frac = fraction(share), t = __umul64hi(frac, mass) + (frac * mass != 0 ? 1 : 0);
        return t < 1 ? 1 : t;
    }
    __device__ __forceinline__ uint64_t point_of(float u, uint64_t mass) const {  // floor(u mass)
        return __umul64hi(fraction(u > 0.f ? fminf(u, 0.99999994f) : 0.f), mass);
    }

    // ---- the way for any distribution: exact counts and masses, level by level ----
    int64_t part_n, total_n;     // tokens in the shares before this CTA's, and all
    uint64_t part_m, total_m;
    bool deep;                   // the histogram is of a later level
    __device__ void tally(bool by_key, uint64_t lo, uint64_t hi, int key_shift, bool masses) {
        for (int i = threadIdx.x; i < kBins; i += kThreads) count()[i] = mass_lo()[i] = mass_hi()[i] = 0u;
        __syncthreads();
        each([&](float l, uint32_t at) {
            int b;
            if (by_key) {
                const uint64_t k = key_of(l, at);
                if (k < lo || k > hi) return;
                b = static_cast<int>((k - lo) >> key_shift);
            } else {
                b = bin_of(l);
            }
            atomicAdd(count() + b, 1u);
            if (!masses) return;
            const uint64_t m = mass_of(l);
            if (m == 0) return;
            const uint32_t low = static_cast<uint32_t>(m), old = atomicAdd(mass_lo() + b, low);
            const uint32_t high = static_cast<uint32_t>(m >> 32) + (old + low < old ? 1u : 0u);
            if (high) atomicAdd(mass_hi() + b, high);
        });
        cluster.sync();
        // this CTA's share of the bins, summed over the cluster, as running sums (in place once every CTA has read them)
        const int mine = kBins / C, first = rank * mine, per = (mine + kThreads - 1) / kThreads;
        int64_t n = 0;
        uint64_t m = 0;
        int64_t upto_n[kBins / kThreads];
        uint64_t upto_m[kBins / kThreads];
#pragma unroll
        for (int i = 0; i < kBins / kThreads; ++i) {
            const int b = first + threadIdx.x * per + i;
            if (i < per && b < first + mine) {
                for (int r = 0; r < C; ++r) {
                    n += *of(count() + b, r);
                    if (masses) m += (static_cast<uint64_t>(*of(mass_hi() + b, r)) << 32) + *of(mass_lo() + b, r);
                }
            }
            upto_n[i] = n;
            upto_m[i] = m;
        }
        int64_t sn = n;
        uint64_t sm = m;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t yn = __shfl_up_sync(0xffffffffu, sn, o);
            const uint64_t ym = __shfl_up_sync(0xffffffffu, sm, o);
            if (lane >= o) sn += yn, sm += ym;
        }
        if (lane == 31) shared().warp_count[warp] = sn, shared().warp_mass[warp] = sm;
        __syncthreads();
        int64_t bn, tn;
        uint64_t bm, tm;
        over_warps(shared().warp_count, &bn, &tn);
        over_warps(shared().warp_mass, &bm, &tm);
        bn += sn - n;
        bm += sm - m;
        if (warp == 0) {
            tell(shared().part_count, tn);
            tell(shared().part_mass, tm);
        }
        cluster.sync();
#pragma unroll
        for (int i = 0; i < kBins / kThreads; ++i) {
            const int b = first + threadIdx.x * per + i;
            if (i >= per || b >= first + mine) continue;
            const uint64_t x = bm + upto_m[i];
            count()[b] = static_cast<uint32_t>(bn + upto_n[i]);
            mass_lo()[b] = static_cast<uint32_t>(x);
            mass_hi()[b] = static_cast<uint32_t>(x >> 32);
        }
        total_n = 0, total_m = 0, part_n = 0, part_m = 0;
        for (int r = 0; r < C; ++r) {
            const int64_t cn = shared().part_count[r];
            const uint64_t cm = shared().part_mass[r];
            if (r < rank) part_n += cn, part_m += cm;
            total_n += cn;
            total_m += cm;
        }
        __syncthreads();
    }
    // The bin that the rank, or the mass, falls into, in every CTA's shared().found.
    __device__ Found locate(bool by_mass, uint64_t target, int64_t n0, uint64_t m0) {
        const int mine = kBins / C, first = rank * mine;
        auto mass_at = [&](int b) { return (static_cast<uint64_t>(mass_hi()[b]) << 32) + mass_lo()[b]; };
        for (int b = first + threadIdx.x; b < first + mine; b += kThreads) {
            const int64_t cb = n0 + part_n + (b > first ? count()[b - 1] : 0u), cu = n0 + part_n + count()[b];
            const uint64_t mb = m0 + part_m + (b > first ? mass_at(b - 1) : 0), mu = m0 + part_m + mass_at(b);
            const bool here = by_mass ? mb < target && target <= mu : static_cast<uint64_t>(cb) < target && target <= static_cast<uint64_t>(cu);
            if (here)
                for (int r = 0; r < C; ++r) *of(&shared().found, r) = Found{mb, cb, b, static_cast<int>(cu - cb)};
        }
        cluster.sync();
        return shared().found;
    }
    // K* for a rank or a mass that some token reaches, and the mass up to it.
    __device__ void solve(bool by_mass, uint64_t target, bool masses, uint64_t *limit, uint64_t *mass) {
        Found f = locate(by_mass, target, 0, 0);
        bool by_key = false;
        uint64_t lo = 0, hi = 0;
        while (f.count > kList) {
            // the keys in the bin, and 2048 bins of them
            uint64_t kmin = ~0ull, kmax = 0;
            const int bin = f.bin;
            each([&](float l, uint32_t at) {
                const uint64_t k = key_of(l, at);
                if (by_key ? k >= lo && k <= hi : bin_of(l) == bin) {
                    kmin = k < kmin ? k : kmin;
                    kmax = k > kmax ? k : kmax;
                }
            });
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const uint64_t a = __shfl_xor_sync(0xffffffffu, kmin, o), b = __shfl_xor_sync(0xffffffffu, kmax, o);
                kmin = a < kmin ? a : kmin;
                kmax = b > kmax ? b : kmax;
            }
            if (lane == 0) shared().warp_key[0][warp] = kmin, shared().warp_key[1][warp] = kmax;
            __syncthreads();
            if (warp == 0) {
                for (int w = 1; w < kWarps; ++w) {
                    kmin = shared().warp_key[0][w] < kmin ? shared().warp_key[0][w] : kmin;
                    kmax = shared().warp_key[1][w] > kmax ? shared().warp_key[1][w] : kmax;
                }
                tell(shared().key_min, kmin);
                tell(shared().key_max, kmax);
            }
            cluster.sync();
            for (int r = 0; r < C; ++r) {
                const uint64_t a = shared().key_min[r], b = shared().key_max[r];
                kmin = r == 0 || a < kmin ? a : kmin;
                kmax = r == 0 || b > kmax ? b : kmax;
            }
            int key_shift = 0;
            while (((kmax - kmin) >> key_shift) >= kBins) ++key_shift;
            tally(true, kmin, kmax, key_shift, masses);
            deep = true;
            f = locate(by_mass, target, f.count_before, f.mass_before);
            by_key = true;
            lo = kmin + (static_cast<uint64_t>(f.bin) << key_shift);
            hi = lo + ((1ull << key_shift) - 1);
            hi = hi > kmax ? kmax : hi;
        }
        // the bin's tokens into the first CTA's list
        if (threadIdx.x == 0) shared().listed = 0;
        cluster.sync();
        const int bin = f.bin;
        gather([&](float l, uint32_t at) {
            if (!by_key) return bin_of(l) == bin;
            const uint64_t k = key_of(l, at);
            return k >= lo && k <= hi;
        });
        cluster.sync();
        if (rank == 0) settle(list(), by_mass, target, masses, f.count, f.count_before, f.mass_before);
        cluster.sync();
        *limit = shared().limit;
        *mass = shared().limit_mass;
    }
    // The keys of some tokens into the first CTA's list (shared().listed is 0 there).
    template <typename F>
    __device__ __forceinline__ void gather(F pick) {
        int *listed = of(&shared().listed, 0);
        uint64_t *to = of(list(), 0);
        columns([&](int i, const float (&x)[W]) {
            const uint32_t at = index_of(i);
            uint32_t some = 0;
#pragma unroll
            for (int j = 0; j < W; ++j) some |= x[j] > -INFINITY && pick(x[j], at + j) ? 1u << j : 0u;
            if (some == 0) return;
#pragma unroll
            for (int j = 0; j < W; ++j)
                if (some >> j & 1u) {
                    const int n = atomicAdd(listed, 1);
                    if (n < kList) to[n] = key_of(x[j], at + j);
                }
        });
    }
    // By the first CTA: K* among n tokens, for every CTA.
    __device__ void settle(uint64_t *keys, bool by_mass, uint64_t target, bool masses, int n, int64_t count_before, uint64_t mass_before) {
        if (n <= kThreads / 4) {
            // few: four threads count and sum what is not behind a token (sorting takes 45 barriers' time, this two)
            __syncthreads();
            const int at = threadIdx.x >> 2, part = threadIdx.x & 3;
            const uint64_t key = at < n ? keys[at] : 0, own = masses && at < n ? mass_of(logit_of(key)) : 0;
            if (part == 0) shared().list_mass[at] = own;
            __syncthreads();
            uint64_t m = 0, count_upto = 0;
            for (int j = part; j < n; j += 4)
                if (keys[j] <= key) m += shared().list_mass[j], ++count_upto;
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                m += __shfl_xor_sync(0xffffffffu, m, o);
                count_upto += __shfl_xor_sync(0xffffffffu, count_upto, o);
            }
            const uint64_t upto = mass_before + m;
            const bool here = by_mass ? upto - own < target && target <= upto : static_cast<uint64_t>(count_before) + count_upto == target;
            if (at < n && part == 0 && here)
                for (int r = 0; r < C; ++r) *of(&shared().limit, r) = key, *of(&shared().limit_mass, r) = upto;
            return;
        }
        sort(keys, n);
        uint64_t m[kPer], own[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int at = kPer * threadIdx.x + i;
            own[i] = m[i] = masses && at < n ? mass_of(logit_of(keys[at])) : 0;
        }
        scan(m);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int at = kPer * threadIdx.x + i;
            if (at >= n) continue;
            const uint64_t upto = mass_before + m[i], cu = static_cast<uint64_t>(count_before) + at + 1;
            const bool here = by_mass ? upto - own[i] < target && target <= upto : cu == target;
            if (here)
                for (int r = 0; r < C; ++r) *of(&shared().limit, r) = keys[at], *of(&shared().limit_mass, r) = upto;
        }
    }

    // A token's e times a factor of at most 1, wherever the token lies: x = (l - M) log2(e) / t as a pair, of which l - M is
    // rounded, and what that leaves out is exact.  Below half of fp32's smallest number it is 0, as for a masked token.
    __device__ __forceinline__ float faint(float l, float factor) const {
        const float d = __fsub_rn(l, c.top), v = __fsub_rn(d, l), d_lo = __fsub_rn(__fsub_rn(l, __fsub_rn(d, v)), __fadd_rn(c.top, v));
        const float h = __fmul_rn(d, c.c_hi);
        if (!(h > -151.f)) return 0.f;
        const float lo = fmaf(d, c.c_hi, -h) + fmaf(d, c.c_lo, d_lo * c.c_hi), n = rintf(h);
        // the power of two in two steps: fp32's smallest numbers are rounded to once
        const float scale = __int_as_float((static_cast<int>(n) + 64 + 127) << 23);
        return exp2f((h - n) + lo) * factor * 5.42101086e-20f * scale;
    }
    // The distribution: tokens up to the limit have e / total, the others none.  Element by element, so that a warp's stores
    // are consecutive whatever the row's alignment; two at a time, as there are such instructions.  The last step: c.cut goes
    // down to where the exponentials end (125 halvings below M, or 63 where l - sub is exact no further); what lies below is
    // faint.
    __device__ void write(int64_t row_at, uint64_t limit, float inv_total) {
        const int64_t first = static_cast<int64_t>(col0) * W - shift;
        const int from = static_cast<int>(first < 0 ? 0 : first);
        const int64_t end = first + static_cast<int64_t>(cols) * W;
        const int to = static_cast<int>(end < p.V ? end : p.V);
        float *wide = static_cast<float *>(p.probs) + row_at * p.ps;
        __nv_bfloat16 *narrow = static_cast<__nv_bfloat16 *>(p.probs) + row_at * p.ps;
        const float least_kept = logit_of(limit);  // (a NaN where there is no limit: every logit is then kept)
        const uint32_t last_kept = static_cast<uint32_t>(limit);
        c.cut = c.sub != 0.f ? -63.f / c.c_hi : c.top - 125.f / c.c_hi;
        for (int i0 = from + threadIdx.x; i0 < to; i0 += 2 * kThreads) {
            float l[2], x[2];
            bool kept[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int i = i0 + j * kThreads;
                l[j] = i < to ? Elem<T>::to_f(row[i]) : -INFINITY;
                if (inf_top) l[j] = l[j] == INFINITY ? 0.f : -INFINITY;
                kept[j] = l[j] > -INFINITY && !(l[j] < least_kept) && (l[j] != least_kept || static_cast<uint32_t>(i) <= last_kept);
            }
            x[0] = x[1] = 0.f;
            if (kept[0] || kept[1]) {
                const float2 e = both(exp2_parts(l[0], l[1], c, shared().table).value);
                x[0] = e.x * inv_total;
                x[1] = e.y * inv_total;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (!kept[j]) x[j] = 0.f;
                    else if (l[j] - c.sub < c.cut) x[j] = faint(l[j], inv_total);
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int i = i0 + j * kThreads;
                if (i >= to) break;
                if (p.wide_probs) wide[i] = x[j];
                else narrow[i] = __float2bfloat16_rn(x[j]);
            }
        }
    }

    // The token at a point of the kept mass, by the CTA that holds it; shared().warp_mass: the kept masses of its warps'
    // tokens.  The tokens of the one warp that has it are shared out among all threads, a few neighbours each, round by round.
    __device__ void draw(int64_t at, uint64_t limit, uint64_t before, uint64_t point) {
        const uint64_t own = lane < kWarps ? shared().warp_mass[lane] : 0;
        uint64_t start = own;
#pragma unroll
        for (int o = 1; o < kWarps; o <<= 1) {
            const uint64_t y = __shfl_up_sync(0xffffffffu, start, o);
            if (lane >= o) start += y;
        }
        start += before - own;
        const uint32_t has = __ballot_sync(0xffffffffu, point >= start && point < start + own);
        if (has == 0) return;
        const int owner = __ffs(has) - 1;
        before = __shfl_sync(0xffffffffu, start, owner);
        const float least_kept = logit_of(limit);
        const uint32_t last_kept = static_cast<uint32_t>(limit);
        constexpr int kEach = 4;
        const int first = owner * span * W, stop = min(cols, (owner + 1) * span) * W;
        for (int e0 = first; e0 < stop; e0 += kThreads * kEach) {
            const int e = e0 + threadIdx.x * kEach;  // elements of the CTA's slice: a part of one column
            uint64_t m[kEach], mine = 0;
            float x[W];
            if (e < stop) unpack(fetch(e / W), x);
            const uint32_t index = index_of(0) + e;
#pragma unroll
            for (int j = 0; j < kEach; ++j) {
                float l = x[j];
                if constexpr (W > kEach) l = e & kEach ? x[kEach + j] : l;
                const bool kept = e < stop && l > -INFINITY && !(l < least_kept) && (l != least_kept || index + j <= last_kept);
                m[j] = kept ? mass_of(l) : 0;
                mine += m[j];
            }
            uint64_t upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t y = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += y;
            }
            __syncthreads();
            if (lane == 31) shared().warp_above[warp] = upto;
            __syncthreads();
            uint64_t here, round;
            over_warps(shared().warp_above, &here, &round);
            here += before + upto - mine;
            before += round;
            if (here <= point && point < here + mine) {
#pragma unroll
                for (int j = 0; j < kEach; ++j) {
                    if (here <= point && point < here + m[j]) p.token[at] = static_cast<int32_t>(index + j);
                    here += m[j];
                }
            }
            if (point < before) return;
        }
    }

    // Top-k of few tokens, by the first CTA: n keys in its list, of which k are kept, then the other filters and the draw.
    __device__ void finish_list(int64_t at, int n, int k, bool mass_on, float top_p) {
        sort(list(), n);
        uint64_t m[kPer];
        auto first_k = [&](int kept) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int x = kPer * threadIdx.x + i;
                m[i] = x < kept ? mass_of(logit_of(list()[x])) : 0;
            }
            return scan(m);
        };
        uint64_t total = first_k(k);
        if (threadIdx.x == 0) shared().listed = k;
        __syncthreads();
        const uint64_t target = mass_on ? share_of(top_p, total) : 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int x = kPer * threadIdx.x + i;
            if (x >= k) continue;
            // the first that is not kept: the one after the border, or the first below min_p's logit
            const uint64_t before = i ? m[i - 1] : m[0] - mass_of(logit_of(list()[x]));
            if (x > 0 && ((mass_on && before >= target) || logit_of(list()[x]) < c.low)) atomicMin(&shared().listed, x);
        }
        __syncthreads();
        const int kept = shared().listed;
        if (p.probs && threadIdx.x == 0)
            for (int r = 0; r < C; ++r) *of(&shared().limit, r) = list()[kept - 1];
        // by index
        for (int i = threadIdx.x; i < kept; i += kThreads) list2()[i] = (list()[i] << 32) | static_cast<uint32_t>(i);
        sort(list2(), kept);
        uint64_t own[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int x = kPer * threadIdx.x + i;
            own[i] = m[i] = x < kept ? mass_of(logit_of(list()[static_cast<uint32_t>(list2()[x])])) : 0;
        }
        total = scan(m);
        if (p.probs && threadIdx.x == 0)
            for (int r = 0; r < C; ++r) *of(&shared().limit_mass, r) = total;
        if (!p.token) return;
        const uint64_t point = point_of(p.u[at], total);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (point < m[i] && point >= m[i] - own[i]) p.token[at] = static_cast<int32_t>(list2()[kPer * threadIdx.x + i] >> 32);
    }
    __device__ __forceinline__ float inverse(uint64_t total) const {  // of a mass in ones
        return __fdiv_rn(unit, __ull2float_rn(total));
    }

    __device__ void run() {
        cluster_arrive();  // waited for before anything is written into another CTA: by then it has begun
        const int64_t at = blockIdx.x / C;
        row = static_cast<const T *>(p.logits) + at * p.ls;
        shift = static_cast<int>((reinterpret_cast<uintptr_t>(row) / sizeof(T)) % W);
        const int all = (p.V + shift + W - 1) / W;
        col0 = rank * p.slice;
        cols = min(p.slice, all - col0);
        cols = cols < 0 ? 0 : cols;
        span = (cols + kThreads - 1) / kThreads * 32;
        inf_top = deep = false;
        unit = __int_as_float((127 + 44 - p.extra) << 23);
        for (int i = threadIdx.x; i < 256; i += kThreads) shared().table[i] = make_uint2(kExp2.th[i], __float_as_uint(kExp2.tl[i]));
        grid_wait();
        // (c.cut, 47 halvings below M, is then always within fp32's range: hotter than 3e36 it was not, and what is -inf had a
        // mass)
        const float asked = p.temperature ? p.temperature[at] : 1.f, t = asked > kHottest ? kHottest : asked;
        const bool greedy = !(t > 1e-30f);
        const float min_p = p.min_p ? p.min_p[at] : 0.f;
        const bool floor_on = min_p > 0.f && !greedy;
        const float top_p = p.top_p ? p.top_p[at] : 1.f;
        const int k = top_p <= 0.f ? 1 : p.top_k ? p.top_k[at] : 0;  // (no mass asked for: the first token)
        bool rank_on = k > 0 && k < p.V;
        if (threadIdx.x == kThreads - 1 && floor_on)
            shared().min_shift = min_p < 1.f ? static_cast<double>(t) * log(static_cast<double>(min_p)) : 0.0;
        // the row, and its largest logit
        float top = -INFINITY;
        const int end = min(cols, (warp + 1) * span);
#pragma unroll 4
        for (int i = warp * span + lane; i < end; i += 32) {
            float f[W];
            unpack16(fetch(i), f);
#pragma unroll
            for (int j = 0; j < W; ++j) top = fmaxf(top, f[j]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (lane == 0) shared().warp_top[warp] = top;
        __syncthreads();
        cluster_wait();
        if (warp == 0) {
            top = lane < kWarps ? shared().warp_top[lane] : -INFINITY;
#pragma unroll
            for (int o = kWarps / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            tell(shared().top, __shfl_sync(0xffffffffu, top, 0));
        }
        cluster.sync();
        top = shared().top[0];
        for (int r = 1; r < C; ++r) top = fmaxf(top, shared().top[r]);

        inf_top = top == INFINITY;
        top = inf_top ? 0.f : top;
        c = RowConst{};
        c.top = top;
        c.low = -INFINITY;
        c.cut = -3.4e38f;
        if (!greedy && top > -INFINITY) {
            // log2(e) / t and M log2(e) / t as pairs of fp32
            c.c_hi = __fdiv_rn(1.44269504f, t);
            c.c_lo = __fdiv_rn(__fadd_rn(__fmaf_rn(-c.c_hi, t, 1.44269504f), 1.92596299e-8f), t);
            const float h = __fmul_rn(top, c.c_hi);
            const bool far = !(fabsf(h) < 128.f);
            c.sub = far ? top : 0.f;
            c.a_hi = far ? 0.f : rintf(h * 65536.f) * (1.f / 65536.f);
            c.a_lo = far ? 0.f : __fadd_rn(__fsub_rn(h, c.a_hi), __fmaf_rn(top, c.c_lo, __fmaf_rn(top, c.c_hi, -h)));
            c.cut = (far ? 0.f : top) - 47.f / c.c_hi;
            // (a rank's place has nothing to do with the temperature, but does with the logits' scale)
            c.bin_scale = kCoarse / (rank_on ? fmaxf(kSpan * t, kRankSpan) : kSpan * t);
            // the lowest logit whose e is at least min_p
            if (floor_on) c.low = __double2float_ru(static_cast<double>(top) + shared().min_shift);
        }
        if (top == -INFINITY) {      // nothing can be drawn
            if (p.token && rank == 0 && threadIdx.x == 0) p.token[at] = -1;
            if (p.probs) write(at, 0, 0.f);
            return;
        }
        if (greedy) {
            uint32_t best = 0xffffffffu;
            each([&](float l, uint32_t i) { best = l == c.top && i < best ? i : best; });
            best = __reduce_min_sync(0xffffffffu, best);
            if (lane == 0) shared().warp_key[0][warp] = best;
            __syncthreads();
            if (warp == 0) {
                for (int w = 0; w < kWarps; ++w) best = min(best, static_cast<uint32_t>(shared().warp_key[0][w]));
                tell(shared().best, best);
            }
            cluster.sync();
            best = shared().best[0];
            for (int r = 1; r < C; ++r) best = min(best, shared().best[r]);
            if (p.token && rank == 0 && threadIdx.x == 0) p.token[at] = static_cast<int32_t>(best);
            if (p.probs) write(at, key_of(c.top, best), 1.f);  // (its e is exp(0): c_hi is zero)
            return;
        }
        const bool mass_on = top_p > 0.f && top_p < 1.f;
        uint64_t limit = ~0ull;
        bool summed = false;         // shared().warp_mass holds the kept masses
        if (rank_on || mass_on) {
            int from, to, tokens;
            tally_counts(rank_on ? 0.f : top_p, &from, &to, &tokens);
            if (rank_on && k >= total_n) {
                rank_on = false;
                to = -1;
            }
            bool any = true;         // the way for any distribution
            if (rank_on) {
                const Found f = locate_rank(k);
                if (f.count <= kList) {
                    const bool last = f.bin == kCoarse - 1;
                    gather([&](float l, uint32_t) { return last || distance(l) < static_cast<float>(f.bin + 1); });
                    cluster.sync();
                    if (rank == 0) finish_list(at, f.count, k, mass_on, top_p);
                    if (p.probs) {
                        cluster.sync();
                        write(at, shared().limit, inverse(shared().limit_mass));
                    }
                    return;
                }
            } else if (mass_on) {
                if (to >= 0 && tokens <= kList) {
                    const float a = static_cast<float>(from), z = static_cast<float>(to + 1);
                    const bool last = to == kCoarse - 1;
                    Sum sum, high;
                    columns([&](int i, const float (&x)[W]) {
                        uint32_t some = 0;
#pragma unroll
                        for (int j = 0; j < W; j += 2) {
                            const Parts2 m = weigh2(x[j], x[j + 1], c, shared().table, unit);
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const float d = distance(x[j + y]);  // (NaN compares as neither)
                                add(sum, m.p[y]);
                                if (d < a) add(high, m.p[y]);
                                some |= !(d < a) && (d < z || (last && x[j + y] > -INFINITY)) ? 1u << (j + y) : 0u;
                            }
                        }
                        if (some) {
#pragma unroll
                            for (int j = 0; j < W; ++j)
                                if (some >> j & 1u) list()[atomicAdd(&shared().own_listed, 1)] = key_of(x[j], index_of(i) + j);
                        }
                        take_over(high, 504);  // (no sooner than the sum of all)
                        take_over(sum, 504);
                    });
                    take_over(sum, 0);
                    take_over(high, 0);
                    uint64_t total = sum.total, above = high.total;
                    total = warp_total(total);
                    above = warp_total(above);
                    if (lane == 0) shared().warp_mass[warp] = total, shared().warp_above[warp] = above;
                    __syncthreads();
                    const int mine = shared().own_listed;
                    if (warp == 0) {
                        uint64_t x, y, none;
                        over_warps(shared().warp_mass, &none, &x);
                        over_warps(shared().warp_above, &none, &y);
                        tell(shared().total, x);
                        tell(shared().above, y);
                        // a place for its tokens in the first CTA's list
                        if (lane == 0) shared().own_first = mine > 0 ? atomicAdd(of(&shared().listed, 0), mine) : 0;
                    }
                    __syncthreads();
                    uint64_t *to_list = of(list2(), 0) + shared().own_first;
                    for (int i = threadIdx.x; i < mine; i += kThreads) to_list[i] = list()[i];
                    cluster.sync();
                    total = above = 0;
                    for (int r = 0; r < C; ++r) total += shared().total[r], above += shared().above[r];
                    const uint64_t target = share_of(top_p, total);
                    if (rank == 0) {
                        if (threadIdx.x == 0)
                            for (int r = 0; r < C; ++r) *of(&shared().limit_mass, r) = 0;
                        settle(list2(), true, target, true, shared().listed, 0, above);
                    }
                    cluster.sync();
                    any = above >= target || shared().limit_mass == 0;  // the border lies elsewhere
                    limit = any ? limit : shared().limit;
                    if (!any && (!floor_on || key_of(c.low, 0xffffffffu) >= limit)) {
                        // the kept masses: those before the bracket, and the kept ones in it
                        summed = true;
                        if (threadIdx.x < kWarps) shared().warp_mass[threadIdx.x] = shared().warp_above[threadIdx.x];
                        __syncthreads();
                        for (int i = threadIdx.x; i < mine; i += kThreads) {
                            const uint64_t key = list()[i];
                            if (key > limit) continue;
                            const int col = (static_cast<int>(static_cast<uint32_t>(key)) + shift) / W - col0;
                            atomicAdd(reinterpret_cast<unsigned long long *>(&shared().warp_mass[col / span]),
                                      static_cast<unsigned long long>(mass_of(logit_of(key))));
                        }
                        __syncthreads();
                    }
                }
            } else {
                any = false;
            }
            if (any) {
                cluster.sync();  // the others may still be reading the counts
                tally(false, 0, 0, 0, mass_on);
                uint64_t mass = total_m;
                if (rank_on) solve(false, static_cast<uint64_t>(k), mass_on, &limit, &mass);
                if (mass_on) {
                    // the first token whose mass, with all before it, reaches p of theirs
                    if (deep) tally(false, 0, 0, 0, true);
                    uint64_t upto_here;
                    solve(true, share_of(top_p, mass), true, &limit, &upto_here);
                }
            }
        }
        if (floor_on) {
            const uint64_t floor_limit = key_of(c.low, 0xffffffffu);
            limit = floor_limit < limit ? floor_limit : limit;
        }
        if (!summed) {
            // the kept masses, warp by warp in the order of the indices
            uint64_t sum;
            if (limit == ~0ull) {
                sum = sum_masses([](float (&)[W], uint32_t) { return true; });
            } else {
                const float least_kept = logit_of(limit);
                const uint32_t last_kept = static_cast<uint32_t>(limit);
                sum = sum_masses([&](float (&x)[W], uint32_t i) {
                    bool some = false;
#pragma unroll
                    for (int j = 0; j < W; ++j) {
                        const bool keep = x[j] > least_kept || (x[j] == least_kept && i + j <= last_kept);
                        some |= keep;
                        x[j] = keep ? x[j] : -INFINITY;
                    }
                    return some;
                });
            }
            sum = warp_total(sum);
            __syncthreads();
            if (lane == 0) shared().warp_mass[warp] = sum;
            __syncthreads();
        }
        if (warp == 0) {
            uint64_t none, x;
            over_warps(shared().warp_mass, &none, &x);
            tell(shared().kept, x);
        }
        cluster.sync();
        uint64_t before = 0, total = 0;
        for (int r = 0; r < C; ++r) {
            const uint64_t x = shared().kept[r];
            if (r < rank) before += x;
            total += x;
        }
        if (p.token) draw(at, limit, before, point_of(p.u[at], total));
        if (p.probs) write(at, limit, inverse(total));
    }
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleParams p) {
    cg::cluster_group cluster = cg::this_cluster();
    Sampler<T> s{p, cluster, static_cast<int>(cluster.num_blocks()), static_cast<int>(cluster.block_rank()), static_cast<int>(threadIdx.x >> 5),
                 static_cast<int>(threadIdx.x & 31)};
    s.run();
}

template <typename T>
kda_status launch_sample(SampleParams p, int N, cudaStream_t s) {
    constexpr int W = Elem<T>::kVec;
    const int sms = sm_count();
    if (sms <= 0) return KDA_ERR_CUDA;
    const int cols = static_cast<int>((static_cast<int64_t>(p.V) + 2 * W - 2) / W);  // at any alignment of the row
    // Two CTAs are resident on an SM.  A CTA alone has no cluster to wait for, but rows in fewer CTAs than that leave SMs idle:
    // clusters just large enough to fill them (128 rows of 131,072, fp32 with top-p: 183 us with one, 137 with two, 116 with
    // four, 142 with eight), as long as every thread has a column.  (Rows with top-k alone would like fewer, 128 of them 58 us
    // with two and 73 with four, but not where others are among them: 107 to 111 with four, 118 to 127 with two.)
    int C = 1;
    while (C < kMaxCluster && static_cast<int64_t>(N) * C < 2 * sms && cols / C >= 2 * kThreads) C *= 2;
    p.slice = (cols + C - 1) / C;
    // room for all of a CTA's tokens in one bin
    const int64_t tokens = static_cast<int64_t>(p.slice) * W;
    int count_bits = 1;
    while (tokens >> count_bits) ++count_bits;
    p.count_shift = 32 - count_bits;
    while (p.place_bits < 3 && (tokens * ((2 << p.place_bits) - 1)) >> p.count_shift == 0) ++p.place_bits;
    if (!smem_opt_in<sample_kernel<T>>(kSmemBytes)) return KDA_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(N) * C);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = s;
    cudaLaunchAttribute at[2];  // it may begin before the launch ahead of it has ended, and waits for that before it reads
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = static_cast<unsigned>(C);
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, sample_kernel<T>, p) != cudaSuccess) return KDA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace
}  // namespace kda

extern "C" {

kda_status kda_sample(const void *logits, kda_dtype dtype, const float *u, const float *temperature, const int32_t *top_k, const float *top_p,
                      const float *min_p, int N, int V, int64_t logits_stride, int32_t *token, void *probs, kda_dtype probs_dtype,
                      int64_t probs_stride, void *stream) {
    using namespace kda::spec;
    if (!dtype_ok(dtype) || (probs && !dtype_ok(probs_dtype))) return KDA_ERR_UNSUPPORTED;
    if (N < 0 || N > (1 << 24) || V <= 0 || V > (1 << 24)) return KDA_ERR_INVALID_ARGUMENT;
    if (!logits_stride) logits_stride = V;
    if (!probs_stride) probs_stride = V;
    if (logits_stride < V || probs_stride < V) return KDA_ERR_INVALID_ARGUMENT;
    if (N == 0) return KDA_OK;
    if (!token && !probs) return KDA_ERR_INVALID_ARGUMENT;
    if (!aligned_to(logits, elem_size(dtype)) || !aligned_to(u, 4) || !aligned_to(temperature, 4) || !aligned_to(top_k, 4) ||
        !aligned_to(top_p, 4) || !aligned_to(min_p, 4) || !aligned_to(token, 4) || (probs && !aligned_to(probs, elem_size(probs_dtype))))
        return KDA_ERR_INVALID_ARGUMENT;
    if (!logits || (token && !u)) return KDA_ERR_INVALID_ARGUMENT;
    kda::SampleParams p{};
    p.logits = logits; p.probs = probs; p.ls = logits_stride; p.ps = probs_stride; p.u = u; p.temperature = temperature; p.top_p = top_p;
    p.min_p = min_p; p.top_k = top_k; p.token = token; p.V = V; p.wide_probs = probs_dtype == KDA_F32;
    while (V > (1 << (19 + p.extra))) ++p.extra;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == KDA_BF16 ? kda::launch_sample<__nv_bfloat16>(p, N, s) : kda::launch_sample<float>(p, N, s);
}

}  // extern "C"
