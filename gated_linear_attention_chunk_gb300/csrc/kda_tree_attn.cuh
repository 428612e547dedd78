// Shared by the kernels of tree attention: parameters, how a sequence is cut, small device helpers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_spec.cuh"
#include "sm100_ptx.cuh"

namespace kda {
namespace attn {

using namespace spec;

constexpr int kTileRows = 64;    // query rows of a unit of the register kernels
constexpr int kTcLeast = 32;     // bf16 sequences of more rows per KV head go to the tcgen05 kernel
constexpr int kTcRows = 128;     // query rows of a tcgen05 tile
constexpr int kTcKeys = 128;     // keys of a tile there

// One sequence as the plan leaves it, once for the register kernels and once for the tcgen05 kernel (a
// sequence has units in one of the two lists).
struct __align__(16) SeqInfo {
    int ctx, nodes, t0, unit0;   // context, nodes, first packed node; units (tcgen05: row tiles) before it
    int nsplit, chunk, tiles;
    int part0;                   // its first row of partial results
};

struct AttnParams {
    const void *q, *k, *v;       // v: the drafted nodes' values, in a batch of trees the finite copy of them
    void *o;
    float *lse;
    Pages c;
    const int32_t *cu, *parent;
    int64_t T, qs, ks, vs;       // token strides in elements
    int N, Hq, Hkv, G, max_nodes;
    bool wide;                   // fp32
    int tc;                      // sequences of more than kTcLeast rows go to the tcgen05 kernel
    float scale;
    uint32_t *status;
    SeqInfo *info, *info_tc;     // [N + 1] each; entry N holds the total in unit0
    uint32_t *bad;               // [N] a page or a parent of the sequence is not valid
    int32_t *seq_of;             // [T] sequence of a packed node
    uint64_t *sees;              // [T] ancestors of a packed node, itself included
    // Trees of more than one node: a tile holds drafted values that some of its rows do not see, and a weight of zero does not take an
    // infinity or NaN out of a product.  So the tiles are made of a copy with zeros in the place of such values (v, vs), and
    // combine_kernel, the last one, adds them to the rows that do see them.
    const void *given_v;
    int64_t given_vs;
    int32_t *odd;                // [T] a packed node has such values; null in a batch of single nodes, which has no copy
    float *part_o;               // partial results, dv columns a row: [node, Hq, part] of a sequence, or tc_part's tiles
    float2 *part_ml;             // and their maximum (base 2) and sum
};

// How a sequence is cut, whatever else is in the batch: parts of at least least_chunk keys (a part's partial result, rows x dv
// fp32 written and read again, has to stay small beside its keys, and so have the few microseconds that a part takes to begin and
// end: with 256 keys in the place of 384 a batch of 128 contexts of 2048 took 238 us for 223, with 512 it took 219, but one
// context of 1025 took 1.5 us longer), as many as give the sequence alone about one unit per SM; long contexts in parts of at
// least 1024 keys up to three units per SM, one per resident CTA, which makes the units of a batch share out more evenly.
constexpr int kFillUnits = 152;
__host__ __device__ inline int most_splits(int Hkv, int tiles, int per_sm = 1) {
    const int per = Hkv * tiles;
    return per >= per_sm * kFillUnits ? 1 : (per_sm * kFillUnits + per - 1) / per;
}
// KV heads of a unit: in fp32 with at most 16 rows the four warps of a CTA take a head each, so that they have nothing to
// join (62 us to 42 for seven contexts of up to 4099); otherwise they share one (bf16 with a head per warp was slower: fewer and
// larger units).
__host__ __device__ inline int heads_of(int rows, int Hkv, bool wide) { return wide && rows <= 16 && Hkv % 4 == 0 ? 4 : 1; }
__host__ __device__ inline int least_chunk(int rows, bool wide, int heads) {
    if (heads == 4) return 128;
    if (wide) return rows <= 32 ? 128 : rows <= 64 ? 4 * rows : 256;
    return rows <= 16 ? 384 : 512;
}
__host__ __device__ inline int splits_of(int64_t ctx, int least, int Hkv, int tiles) {
    const int64_t some = (ctx + least - 1) / least, one = most_splits(Hkv, tiles);
    const int64_t many = (ctx + 1023) / 1024, three = most_splits(Hkv, tiles, 3);
    const int64_t s = some < one ? some : one, t = many < three ? many : three;
    return static_cast<int>(s > t ? (s < 1 ? 1 : s) : (t < 1 ? 1 : t));
}
// Keys of each of s parts, a multiple of `unit` (but for one part of a context that ends right below 2^31).
__host__ __device__ inline int chunk_of(int ctx, int s, int unit) {
    const int c = ctx > 0 ? (ctx - 1) / s + 1 : 1;
    return c > 0x7fffffff - unit ? 0x7fffffff : (c + unit - 1) / unit * unit;
}
__host__ __device__ inline void split_of(int ctx, int rows, int Hkv, int tiles, bool wide, int *nsplit, int *chunk) {
    const int heads = heads_of(rows, Hkv, wide);
    const int s = splits_of(ctx, least_chunk(rows, wide, heads), Hkv / heads, tiles);
    *chunk = chunk_of(ctx, s, 64);
    *nsplit = ctx > 0 ? (ctx - 1) / *chunk + 1 : 1;
}
__host__ __device__ inline int tiles_of(int rows) { return (rows + kTileRows - 1) / kTileRows; }

// The same for the tcgen05 kernel, whose units are pairs of row tiles (or one): the number that fills the GPU, or a
// multiple of it, so that the units of a batch of such sequences share out evenly (32 parts in the place of 19 for four
// sequences of 131,072 keys and 264 rows on 4 KV heads: 531 us against 430).
constexpr int kTcChunk = 16384, kTcShort = 1024;
__host__ __device__ inline int tc_tiles_of(int rows) { return (rows + kTcRows - 1) / kTcRows; }
__host__ __device__ inline int tc_groups_of(int tiles) { return (tiles + 1) / 2; }
__host__ __device__ inline int tc_splits_of(int64_t ctx, int Hkv, int groups) {
    const int64_t some = (ctx + kTcShort - 1) / kTcShort, most = most_splits(Hkv, groups);
    const int64_t s = some < most ? some : most * ((ctx + most * kTcChunk - 1) / (most * kTcChunk));
    return static_cast<int>(s < 1 ? 1 : s);
}
__host__ __device__ inline void tc_split_of(int ctx, int Hkv, int tiles, int *nsplit, int *chunk) {
    const int s = tc_splits_of(ctx, Hkv, tc_groups_of(tiles));
    *chunk = chunk_of(ctx, s, kTcKeys);
    *nsplit = ctx > 0 ? (ctx - 1) / *chunk + 1 : 1;
}

// Partial results are numbered by the plan: a sequence has as many rows of them as its own cut asks for.  The tcgen05 kernel's lie by
// KV head, row tile and part, [dv / 4][pitch] of 4 columns each; a tile alone leaves two per part, a pair of one part none.
__host__ __device__ inline int tc_pitch(int rows, int tile) {
    const int left = rows - tile * kTcRows;
    return left >= kTcRows ? kTcRows : (left + 7) / 8 * 8;
}
__host__ __device__ inline int tc_part_rows(int rows, int tiles, int nsplit) {  // of one KV head
    const int paired = nsplit > 1 ? nsplit : 0;
    return (tiles - 1) * kTcRows * paired + tc_pitch(rows, tiles - 1) * (tiles & 1 ? 2 * nsplit : paired);
}
__device__ __forceinline__ int64_t tc_part(int part0, int rows, int tiles, int nsplit, int head, int tile, int split, int stream) {
    const bool alone = (tile | 1) >= tiles;  // the last of an odd number: those before it are pairs
    return part0 + static_cast<int64_t>(head) * tc_part_rows(rows, tiles, nsplit) + tile * kTcRows * (nsplit > 1 ? nsplit : 0) +
           (alone ? 2 * split + stream : split) * tc_pitch(rows, tile);
}
// Rows of partial results of a sequence of `nodes` nodes in nsplit parts.
__host__ __device__ inline int64_t part_rows(bool tc, int nodes, int Hq, int Hkv, int nsplit) {
    const int rows = nodes * (Hq / Hkv);
    if (tc && rows > kTcLeast) return static_cast<int64_t>(Hkv) * tc_part_rows(rows, tc_tiles_of(rows), nsplit);
    return nsplit > 1 ? static_cast<int64_t>(nodes) * Hq * nsplit : 0;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool there) {
    const int n = there ? 16 : 0;  // 0: nothing is read and the 16 bytes become zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// 16 bytes of T without what is not finite; `odd` becomes true if there was such a value.
template <typename T>
__device__ __forceinline__ uint4 finite_only(uint4 x, bool &odd) {
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool high = (w[i] & 0x7f800000u) == 0x7f800000u, low = sizeof(T) == 2 && (w[i] & 0x7f80u) == 0x7f80u;
        odd |= high || low;
        if (high) w[i] = sizeof(T) == 2 ? w[i] & 0xffffu : 0u;
        if (low) w[i] &= 0xffff0000u;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// kda_tree_attn_tc.cu: the units of info_tc (bf16).
cudaError_t launch_attn_tc(const AttnParams &p, int dk, int dv, int sms, cudaStream_t s);

}  // namespace attn
}  // namespace kda
