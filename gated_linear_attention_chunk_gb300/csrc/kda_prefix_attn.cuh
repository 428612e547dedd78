// Shared by the kernels of attention over a shared prefix: parameters, how the work is cut, small device helpers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_spec.cuh"

namespace kda {
namespace prefix {

using namespace spec;

// One group as the plan leaves it.  Its units of work are (KV head, block of query rows); a unit's steps are its tiles of keys.
// The work is cut in one of two ways (entry N has it in `parts`):
//   0: the steps of all units, in the order of group, KV head, block, are cut into one run per CTA.  A unit begins with `blocks` steps (of entry
//      N) without keys: what beginning and ending a unit costs beside its tiles, so that CTAs with many short units do not come last.
//   1: every unit of a group into `parts` parts, numbered by KV head, part, block; CTA c takes the parts c, c + ctas, ..  So the
//      blocks of one KV head read the same keys at the same time, and these come from memory once.  (128 x 4 tokens of 32 heads over
//      131,072 keys of 8 KV heads: cut in runs 4.3 GB were read where there are 0.54 GB.)
struct __align__(16) GroupInfo {
    int64_t step0;            // steps (parts) before it (entry N: of all)
    int t0, tokens;           // its packed tokens
    int len, tiles;           // keys, and tiles of them
    int blocks, parts;        // blocks of query rows per KV head; see above
};
constexpr int kMostRounds = 4;  // parts per CTA at the most, unless each is a whole unit

struct PrefixParams {
    const void *q, *o_tail;
    const float *lse_tail;
    void *o;
    float *lse;
    Pages c;
    const int32_t *cu;
    int64_t T, qs;
    int N, Hq, Hkv, G;        // groups; heads; query heads per KV head
    float scale;
    bool wide;                // fp32
    uint32_t *status;
    GroupInfo *info;          // [N + 1]; entry N: errors of the lengths in `tokens`
    uint32_t *errors;         // [ctas] of what the CTA met
    bool planned;             // by a kernel before; otherwise every CTA makes the plan, and writes the same
    float *part_o;            // partial results: [slot][pitch][dv] sums, and their maximum (base 2) and weight sum; a negative sum marks a
                              // part with a bad page
    float2 *part_ml;
    int ctas, pitch;          // slots: two per CTA, or one per part; rows of a slot
    int rows;                 // query rows of a block
    int pages_per_tile, tiles_per_page, tile_keys;  // of a tile of keys (pages_per_tile 0: keys are counted across pages)
};

__host__ __device__ inline int tiles_of_len(const PrefixParams &p, int len) {
    const uint32_t n = static_cast<uint32_t>(len), keys = static_cast<uint32_t>(p.tile_keys);
    if (p.pages_per_tile > 0) {
        const uint32_t per = static_cast<uint32_t>(p.pages_per_tile * p.c.page_size);  // at most `keys`
        return static_cast<int>((n + per - 1) / per);
    }
    if (p.tiles_per_page > 0) {
        const uint32_t pages = n / p.c.page_size;
        return static_cast<int>(pages * p.tiles_per_page + (n - pages * p.c.page_size + keys - 1) / keys);
    }
    return static_cast<int>((n + keys - 1) / keys);
}

// Work is cut into parts where blocks share so many tiles of keys (64 KB each) that L2 does not keep them from one block to the
// next.
constexpr int64_t kShared = 1024;
constexpr int kPartCost = 4, kUnitCost = 4;  // tiles
// Up to so many groups the kernels plan themselves, which spares a launch: 65,536 keys of 8 heads, eight tokens per group, in 2
// to 16 groups 63 to 65 us and 69 with the launch, in 64 groups 90 and 94, in 256 173 and 191 (256 groups of two tokens and 128
// keys 116 and 108, of four and 1,000 296 and 290). Reading the plan from L2 is as fast as from shared memory (one group of
// 2,048 keys 22.4 us either way, 16 of 4,096 64.6).
constexpr int kPlanGroups = 256;

// What the plan of a CTA of whole warps, kPlanGroups threads at least, needs in shared memory.
struct PlanScratch {
    RunningMax tops;
    int64_t warp_sum[32], base;
    int64_t shared_tiles;         // tiles of keys that more than one block reads
    int64_t all_tiles;            // of all units
    uint64_t parts_at[32];        // parts of all units, for 32 sizes
    uint32_t errors;
    int longest;
    int tiles[kPlanGroups], blocks[kPlanGroups];
};

// Checks the lengths, numbers the steps and chooses the cut; by all threads of a CTA.  Each entry of p.info is written once, by
// every CTA that plans with the same.
__device__ inline void make_plan(const PrefixParams &p, PlanScratch &s) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, threads = blockDim.x;
    if (threadIdx.x == 0) {
        s.base = s.shared_tiles = s.all_tiles = 0;
        s.errors = 0;
        s.longest = 0;
    }
    if (threadIdx.x < 32) s.parts_at[threadIdx.x] = 0;
    s.tops.begin();
    bool by_parts = false;
    int lead = 0;
    for (int g0 = 0, round = 0; g0 < p.N; g0 += threads, ++round) {
        const int g = g0 + threadIdx.x;
        const int64_t a = g < p.N ? p.cu[g] : 0, b = g < p.N ? p.cu[g + 1] : 0, len = g < p.N ? p.c.ctx_len[g] : 0;
        const int before = s.tops.next(g < p.N ? static_cast<int>(a) : INT32_MIN, round);
        GroupInfo x{};
        if (g < p.N) {
            uint32_t err = 0;
            if (a < 0 || a > b || b > p.T || (g == 0 && a != 0) || a < before) err = DEV_ERR_SEQLENS;
            else if (len < 0 || len > static_cast<int64_t>(p.c.max_pages) * p.c.page_size) err = DEV_ERR_PAGE;
            x.t0 = before > a ? before : static_cast<int>(a);  // never falls, so that a token's group can be looked up
            if (err) {
                atomicOr(&s.errors, err);
            } else {
                x.tokens = static_cast<int>(b - a);
                x.len = static_cast<int>(len);
                x.tiles = tiles_of_len(p, x.len);
                x.blocks = static_cast<int>((static_cast<uint32_t>(x.tokens) * p.G + p.rows - 1) / p.rows);  // (T Hq is below 2^31)
            }
        }
        int64_t steps = static_cast<int64_t>(p.Hkv) * x.blocks * x.tiles;
        if (!p.wide && p.N <= kPlanGroups) {
            if (g < p.N) {
                s.tiles[g] = x.tiles;
                s.blocks[g] = x.blocks;
                if (x.blocks > 0) atomicMax(&s.longest, x.tiles);
                atomicAdd(reinterpret_cast<unsigned long long *>(&s.all_tiles), static_cast<unsigned long long>(steps));
                if (x.blocks > 1)
                    atomicAdd(reinterpret_cast<unsigned long long *>(&s.shared_tiles), static_cast<unsigned long long>(x.tiles) * p.Hkv);
            }
            __syncthreads();
            by_parts = s.shared_tiles >= kShared;
            const int64_t share = s.all_tiles / (4 * static_cast<int64_t>(p.ctas));  // (where a CTA has few tiles each counts more)
            lead = by_parts ? 0 : static_cast<int>(share < kUnitCost ? share : kUnitCost);
            if (x.tiles > 0) steps += static_cast<int64_t>(p.Hkv) * x.blocks * lead;
            if (by_parts) {
                // Parts of at most `size` tiles: of 32 sizes the one whose rounds take least, a part costing kPartCost tiles
                // beside its own.
                auto parts_of = [](int tiles, int size) { return tiles > 0 ? (tiles + size - 1) / size : 0; };
                // (a lane has a size, a warp some of the groups)
                const int size = (s.longest + lane) / (lane + 1);
                int64_t n = 0;
                for (int h = warp; h < p.N; h += threads / 32) n += static_cast<int64_t>(p.Hkv) * s.blocks[h] * parts_of(s.tiles[h], size);
                if (n > 0) atomicAdd(reinterpret_cast<unsigned long long *>(&s.parts_at[lane]), static_cast<unsigned long long>(n));
                __syncthreads();
                const uint64_t rounds = (s.parts_at[lane] + p.ctas - 1) / p.ctas;
                uint64_t best = lane == 0 || rounds <= kMostRounds ? rounds * static_cast<uint64_t>(size + kPartCost) << 5 | lane : ~0ull;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const uint64_t y = __shfl_xor_sync(0xffffffffu, best, o);
                    best = y < best ? y : best;
                }
                const int pick = static_cast<int>(best & 31u);
                x.parts = parts_of(x.tiles, (s.longest + pick) / (pick + 1));
                steps = static_cast<int64_t>(p.Hkv) * x.blocks * x.parts;
            }
        }
        int64_t upto = steps;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        if (lane == 31) s.warp_sum[warp] = upto;
        __syncthreads();
        int64_t off = s.base;
        for (int w = 0; w < warp; ++w) off += s.warp_sum[w];
        if (g < p.N) {
            x.step0 = off + upto - steps;
            p.info[g] = x;
        }
        __syncthreads();
        if (threadIdx.x == threads - 1) s.base = off + upto;
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        GroupInfo x{};
        x.tokens = static_cast<int>(s.errors);
        x.step0 = s.base;
        x.parts = by_parts ? 1 : 0;
        x.blocks = lead;
        p.info[p.N] = x;
    }
    __syncthreads();
}

// The steps of a CTA begin at first_step(c); cta_of is the CTA that has a step.
__device__ __forceinline__ int64_t first_step(int64_t total, int c, int ctas) { return total * c / ctas; }
__device__ __forceinline__ int cta_of(int64_t total, int64_t step, int ctas) {
    return static_cast<int>(((step + 1) * ctas + total - 1) / total) - 1;
}

// A CTA's walk over its segments: runs of steps within one unit, those with keys.
struct SegmentWalk {
    int64_t next_step, end, begin;
    int lead;                    // steps without keys at the beginning of a unit
    bool by_parts, is_live;
    int g, head, block, k0, k1;  // key tiles [k0, k1) of the unit
    int t0, tokens, len, tiles;
    bool whole;                  // all of the unit's tiles
    int slot;

    // Every lane of a converged warp.
    __device__ __forceinline__ void start(const PrefixParams &p) {
        const GroupInfo all = p.info[p.N];
        by_parts = all.parts != 0;
        lead = all.blocks;
        begin = next_step = by_parts ? blockIdx.x : first_step(all.step0, blockIdx.x, p.ctas);
        end = by_parts ? all.step0 : first_step(all.step0, blockIdx.x + 1, p.ctas);
        next(p);
    }
    __device__ __forceinline__ bool live() const { return is_live; }
    __device__ __forceinline__ void next(const PrefixParams &p) {
        for (is_live = next_step < end; next_step < end;) {
            enter(p);
            if (k0 < k1) return;
        }
        is_live = false;
    }
    __device__ __forceinline__ void enter(const PrefixParams &p) {
        const int64_t at = next_step;
        // (groups without steps begin where the next one does: the last of them has it)
        g = warp_find([&](int i) { return p.info[i].step0; }, p.N, at);
        const GroupInfo s = p.info[g];
        t0 = s.t0; tokens = s.tokens; len = s.len; tiles = s.tiles;
        if (by_parts) {
            const int off = static_cast<int>(at - s.step0), rest = off / s.blocks;
            block = off - rest * s.blocks;
            head = rest / s.parts;
            const int part = rest - head * s.parts;
            k0 = static_cast<int>(static_cast<int64_t>(s.tiles) * part / s.parts);
            k1 = static_cast<int>(static_cast<int64_t>(s.tiles) * (part + 1) / s.parts);
            whole = s.parts == 1;
            slot = static_cast<int>(at);
            next_step = at + p.ctas;
            return;
        }
        const int size = s.tiles + lead;
        const int64_t off = at - s.step0;
        const int u = static_cast<int>(off >> 32 ? off / size : static_cast<uint32_t>(off) / static_cast<uint32_t>(size));
        const int from = static_cast<int>(off - static_cast<int64_t>(u) * size);
        const int to = end - at < size - from ? from + static_cast<int>(end - at) : size;
        k0 = from > lead ? from - lead : 0;
        k1 = to > lead ? to - lead : 0;
        head = u / s.blocks;
        block = u - head * s.blocks;
        whole = k0 == 0 && k1 == s.tiles;
        slot = 2 * blockIdx.x + (at == begin ? 0 : 1);
        next_step = at + (to - from);
    }
};

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// The prefix's share and the tail's: with the prefix's maximum m (base 2) and weight sum l, the factors of its sums and of
// o_tail, and the log-sum of both.  A side without mass has the factor 0 (and is not to be read).
struct Join {
    float prefix, tail, lse;
};
__device__ __forceinline__ Join join_tail(float m, float l, bool has_tail, float lse_tail) {
    const bool some = l != 0.f;
    const float lse_p = some ? (m + log2f(l)) * kLn2 : -INFINITY;
    if (!has_tail || lse_tail == -INFINITY) return Join{some ? 1.f / l : 0.f, 0.f, lse_p};
    if (!some) return Join{0.f, 1.f, lse_tail};
    const float high = fmaxf(lse_p, lse_tail);
    const float a = exp2f((lse_p - high) * kLog2e), b = exp2f((lse_tail - high) * kLog2e), inv = 1.f / (a + b);
    return Join{a * inv / l, b * inv, high + logf(a + b)};
}

// kda_prefix_attn_tc.cu (bf16): blocks of up to 256 rows, one CTA per SM.
constexpr int kTcBlock = 256;
void tc_cut(PrefixParams *p);  // how keys are cut into tiles
cudaError_t launch_prefix_tc(const PrefixParams &p, int dk, int dv, cudaStream_t s);

}  // namespace prefix
}  // namespace kda
