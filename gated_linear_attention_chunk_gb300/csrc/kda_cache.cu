// Append of new rows to a paged cache: the keys and values of a prompt, or of the accepted nodes of a
// drafted tree (through their row indices), to the rows after each sequence's context.
//
// A pure copy, bounded by its bytes (each row read and written once).  A warp has a few consecutive tokens; their
// sequence is found by a 32-way search, their rows and pages looked up by a lane each, and
// then all lanes copy 16 bytes of a token's heads at a time, all loads of a step before the first store.
// 16,392 tokens of 8 heads, 2 KB of keys and of values each: 26.7 us, 5.0 TB/s.  The status word is cleared and the
// lengths are looked over by a kernel that this one overlaps: one call takes 8 to 9 us with its host side (10.7 behind a memset).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_spec.cuh"

namespace kda {
namespace {

// Words 0 and 1 become 0; word 2 says whether cu falls somewhere.  If it does, begins_low[n] (where given) says of each
// sequence whether it begins below an earlier entry, that is, shares packed rows with another one.
__global__ void check_kernel(uint32_t *words, const int32_t *cu, int N, uint64_t *begins_low) {
    spec::grid_go();
    bool falls = false;
    for (int i = threadIdx.x; i < N; i += blockDim.x) falls |= cu[i + 1] < cu[i];
    falls = __syncthreads_or(falls);
    if (threadIdx.x < 3) words[threadIdx.x] = threadIdx.x == 2 && falls ? 1u : 0u;
    if (!falls || !begins_low) return;
    __shared__ spec::RunningMax run;
    run.begin();
    for (int base = 0; base < N; base += blockDim.x) {
        const int n = base + threadIdx.x, first = n < N ? cu[n] : INT32_MIN;
        const int before = run.next(first, base / static_cast<int>(blockDim.x));
        if (n < N) begins_low[n] = first < before;
    }
}

}  // namespace

namespace spec {

bool check_lengths(void *workspace, const int32_t *cu, int N, uint64_t *begins_low, cudaStream_t s) {
    check_kernel<<<1, N > 2048 ? 1024 : 256, 0, s>>>(static_cast<uint32_t *>(workspace), cu, N, begins_low);
    return cudaGetLastError() == cudaSuccess;
}

}  // namespace spec

namespace {

using namespace spec;

constexpr int kAppendThreads = 256;
constexpr int kAppendWarps = kAppendThreads / 32;
constexpr int kAppendUnroll = 4;  // 16-byte loads in flight per lane

struct AppendParams {
    const char *k, *v;
    Pages c;
    const int32_t *cu, *rows;
    int32_t *new_len;
    int64_t A_total, T_src, ks, vs;  // token strides in 16-byte units
    int N, Hkv;
    int per;                         // tokens of a warp (at most 32)
    int kshift, vshift;              // log2 of a head's 16-byte units
    uint32_t *status;
};

__device__ __forceinline__ void raise(uint32_t *status, uint32_t err) {
    grid_wait();  // the status word has been cleared
    atomicOr(status, err);
}

// A sequence's place in the packed rows and its context, checked.
struct AppendSeq {
    int64_t first, last, ctx;
    uint32_t err;
};
__device__ __forceinline__ AppendSeq append_seq(const AppendParams &p, int n) {
    AppendSeq s{p.cu[n], p.cu[n + 1], p.c.ctx_len[n], 0u};
    if (s.first < 0 || s.first > s.last || s.last > p.A_total || (n == 0 && s.first != 0)) s.err = DEV_ERR_SEQLENS;
    else if (s.ctx < 0 || s.ctx + (s.last - s.first) > static_cast<int64_t>(p.c.max_pages) * p.c.page_size)
        s.err = DEV_ERR_PAGE;
    return s;
}

// The heads of a token's key and value rows, 16 bytes per lane and step, all loads of a step before its stores.
struct CopySide {
    const char *src;
    char *dst;
    int64_t head_bytes;
    int units, shift;
    __device__ __forceinline__ void load(uint4 (&x)[kAppendUnroll], int u0) const {
#pragma unroll
        for (int i = 0; i < kAppendUnroll; ++i)
            if (u0 + 32 * i < units) x[i] = __ldcs(reinterpret_cast<const uint4 *>(src) + u0 + 32 * i);
    }
    __device__ __forceinline__ void store(const uint4 (&x)[kAppendUnroll], int u0) const {
#pragma unroll
        for (int i = 0; i < kAppendUnroll; ++i) {
            const int u = u0 + 32 * i;
            if (u < units) *reinterpret_cast<uint4 *>(dst + (u >> shift) * head_bytes + ((u & ((1 << shift) - 1)) << 4)) = x[i];
        }
    }
};

__device__ __forceinline__ CopySide key_side(const AppendParams &p, int64_t row, int64_t place, int64_t es) {
    return CopySide{p.k + row * p.ks * 16, p.c.k + place, p.c.kh * es, p.Hkv << p.kshift, p.kshift};
}
__device__ __forceinline__ CopySide value_side(const AppendParams &p, int64_t row, int64_t place, int64_t es) {
    return CopySide{p.v + row * p.vs * 16, p.c.v + place, p.c.vh * es, p.Hkv << p.vshift, p.vshift};
}

// Source row and place of token j of sequence n (row -1: not to be written), from a sequence without errors.
__device__ __forceinline__ int64_t append_place(const AppendParams &p, const AppendSeq &s, int n, int64_t j, int64_t es, int64_t *place_k,
                                                int64_t *place_v) {
    const int64_t r = p.rows ? static_cast<int64_t>(p.rows[j]) : j, at = s.ctx + j - s.first;
    const int64_t page = p.c.table[static_cast<int64_t>(n) * p.c.table_stride + at / p.c.page_size];
    const int64_t slot = at % p.c.page_size;
    const bool row_ok = r >= 0 && r < p.T_src, page_ok = page >= 0 && page < p.c.num_pages;
    if (!row_ok || !page_ok) {
        raise(p.status, row_ok ? DEV_ERR_PAGE : DEV_ERR_SLOT);
        return -1;
    }
    *place_k = (page * p.c.kp + slot * p.c.kr) * es;
    *place_v = (page * p.c.vp + slot * p.c.vr) * es;
    return r;
}

// The whole call for a cu that falls somewhere: every CTA walks the sequences with the running maximum of cu and copies, a warp
// per sequence, those of its own number.  A sequence that begins below an earlier entry is a bad one.
__device__ __noinline__ void append_malformed(const AppendParams &p, int64_t es) {
    __shared__ RunningMax run;
    const int lane = threadIdx.x & 31;
    run.begin();
    for (int base = 0; base < p.N; base += kAppendThreads) {
        const int n = base + threadIdx.x;
        const int before = run.next(n < p.N ? p.cu[n] : INT32_MIN, base / kAppendThreads);
        AppendSeq mine{0, 0, 0, DEV_ERR_SEQLENS};
        if (n < p.N) {
            mine = append_seq(p, n);
            if (mine.first < before) mine.err = DEV_ERR_SEQLENS;
            if (blockIdx.x == 0) {
                if (mine.err) raise(p.status, mine.err);
                if (p.new_len) p.new_len[n] = static_cast<int32_t>(mine.err ? mine.ctx : mine.ctx + mine.last - mine.first);
            }
        }
        const int n0 = base + static_cast<int>(threadIdx.x) - lane;
        for (int l = 0; l < 32 && n0 + l < p.N; ++l) {
            const AppendSeq s{__shfl_sync(0xffffffffu, mine.first, l), __shfl_sync(0xffffffffu, mine.last, l),
                              __shfl_sync(0xffffffffu, mine.ctx, l), __shfl_sync(0xffffffffu, mine.err, l)};
            if (s.err || (n0 + l) % gridDim.x != blockIdx.x) continue;
            for (int64_t j = s.first; j < s.last; ++j) {
                int64_t place_k = 0, place_v = 0;
                const int64_t r = append_place(p, s, n0 + l, j, es, &place_k, &place_v);
                if (r < 0) continue;
                const CopySide k = key_side(p, r, place_k, es), v = value_side(p, r, place_v, es);
                for (int u0 = lane; u0 < k.units || u0 < v.units; u0 += 32 * kAppendUnroll) {
                    uint4 x[kAppendUnroll];
                    k.load(x, u0);
                    k.store(x, u0);
                    v.load(x, u0);
                    v.store(x, u0);
                }
            }
        }
    }
}

__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendParams p, int64_t es) {
    // A few lengths are looked over here, more of them by the kernel ahead.
    bool falls;
    if (p.N <= kAppendThreads) {
        const int i = threadIdx.x;
        falls = __syncthreads_or(i < p.N && p.cu[i + 1] < p.cu[i]);
    } else {
        grid_wait();
        falls = __ldcg(p.status + 2) != 0;
    }
    if (falls) {
        append_malformed(p, es);
        grid_wait();
        return;
    }
    // new lengths, one thread per sequence
    const int64_t gid = static_cast<int64_t>(blockIdx.x) * kAppendThreads + threadIdx.x;
    for (int64_t n = gid; n < p.N; n += static_cast<int64_t>(gridDim.x) * kAppendThreads) {
        const AppendSeq s = append_seq(p, static_cast<int>(n));
        if (s.err) raise(p.status, s.err);
        if (p.new_len) p.new_len[n] = static_cast<int32_t>(s.err ? s.ctx : s.ctx + s.last - s.first);
    }
    const int lane = threadIdx.x & 31;
    const int64_t most = p.cu[p.N];
    const int64_t total = most < p.A_total ? most : p.A_total;
    for (int64_t j0 = (static_cast<int64_t>(blockIdx.x) * kAppendWarps + (threadIdx.x >> 5)) * p.per; j0 < total;
         j0 += static_cast<int64_t>(gridDim.x) * kAppendWarps * p.per) {
        // lane i looks up token j0 + i: one chain of dependent loads for all of the warp's tokens
        const int n0 = warp_find([&](int i) { return p.cu[i]; }, p.N, j0);
        const int64_t j = j0 + lane;
        int64_t row = -1, place_k = 0, place_v = 0;
        if (lane < p.per && j < total) {
            int n = n0;
            while (n + 1 < p.N && p.cu[n + 1] <= j) ++n;
            const AppendSeq s = append_seq(p, n);
            if (s.err || j < s.first || j >= s.last) {
                if (!s.err) raise(p.status, DEV_ERR_SEQLENS);
            } else {
                row = append_place(p, s, n, j, es, &place_k, &place_v);
            }
        }
        __syncwarp();
        for (int i = 0; i < p.per; ++i) {
            const int64_t r = __shfl_sync(0xffffffffu, row, i);
            const int64_t pk = __shfl_sync(0xffffffffu, place_k, i), pv = __shfl_sync(0xffffffffu, place_v, i);
            if (r < 0) continue;
            const CopySide k = key_side(p, r, pk, es), v = value_side(p, r, pv, es);
            for (int u0 = lane; u0 < k.units || u0 < v.units; u0 += 32 * kAppendUnroll) {
                uint4 x[kAppendUnroll], y[kAppendUnroll];
                k.load(x, u0);
                v.load(y, u0);
                k.store(x, u0);
                v.store(y, u0);
            }
        }
    }
    grid_wait();
}

}  // namespace
}  // namespace kda

extern "C" {

kda_status kda_cache_append(const void *k, const void *v, kda_dtype dtype, const kda_paged_kv *cache,
                            const int32_t *cu, const int32_t *rows, int N, int64_t A_total, int64_t T_src, int Hkv,
                            int dk, int dv, int64_t k_stride, int64_t v_stride, int32_t *new_len, void *workspace,
                            size_t ws_bytes, void *stream) {
    using namespace kda::spec;
    if (!dtype_ok(dtype) || !dim_ok(dk) || !dim_ok(dv)) return KDA_ERR_UNSUPPORTED;
    if (N < 0 || N > 0x7fffffff - 1024 || A_total < 0 || T_src < 0 || Hkv <= 0 || Hkv > 4096) return KDA_ERR_INVALID_ARGUMENT;
    if (!workspace || !aligned_to(workspace, 16) || ws_bytes < KDA_WS_HEADER_BYTES) return KDA_ERR_WORKSPACE;
    Pages c;
    kda_status st = check_pages(cache, dtype, N, &c);
    if (st != KDA_OK) return st;
    const int es = static_cast<int>(elem_size(dtype)), vec = 16 / es;
    if (!k_stride) k_stride = static_cast<int64_t>(Hkv) * dk;
    if (!v_stride) v_stride = static_cast<int64_t>(Hkv) * dv;
    if (k_stride < static_cast<int64_t>(Hkv) * dk || v_stride < static_cast<int64_t>(Hkv) * dv || k_stride % vec ||
        v_stride % vec)
        return KDA_ERR_INVALID_ARGUMENT;
    if (N > 0 && (!cu || !aligned_to(cu, 4))) return KDA_ERR_INVALID_ARGUMENT;
    if (A_total > 0 && T_src > 0 && (!k || !v)) return KDA_ERR_INVALID_ARGUMENT;
    if (!rows && A_total > T_src) return KDA_ERR_INVALID_ARGUMENT;
    if (!aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(rows, 4) || !aligned_to(new_len, 4))
        return KDA_ERR_INVALID_ARGUMENT;
    if (new_len && new_len == cache->ctx_len) return KDA_ERR_INVALID_ARGUMENT;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!check_lengths(workspace, cu, N, nullptr, s)) return KDA_ERR_CUDA;
    if (N == 0) return KDA_OK;
    auto shift = [&](int d) { int b = 0; for (int u = d / vec; u > 1; u >>= 1) ++b; return b; };
    kda::AppendParams p{static_cast<const char *>(k), static_cast<const char *>(v), c, cu, rows, new_len, A_total, T_src,
                        k_stride / vec, v_stride / vec, N, Hkv, 1, shift(dk), shift(dv), static_cast<uint32_t *>(workspace)};
    const int64_t most = static_cast<int64_t>(sm_count()) * 8;
    if (most <= 0) return KDA_ERR_CUDA;
    // few tokens: a warp each; many: up to 4 per warp, whose look-ups then wait for memory together
    const int64_t share = A_total / (most * 4);
    p.per = static_cast<int>(share < 1 ? 1 : share > 4 ? 4 : share);
    const int64_t work = A_total / p.per + 1 > N / 32 ? A_total / p.per + 1 : N / 32 + 1;
    const int64_t want = (work + kda::kAppendWarps - 1) / kda::kAppendWarps;
    const dim3 grid(static_cast<unsigned>(want < most ? want : most));
    return launch_after(kda::append_kernel, grid, kda::kAppendThreads, 0, s, p, static_cast<int64_t>(es)) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
