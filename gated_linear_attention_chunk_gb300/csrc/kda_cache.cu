// Append of new rows to a paged cache: the keys and values of a prompt, or of the accepted nodes of a
// drafted tree (through their row indices), to the rows after each sequence's context.
//
// A pure copy, bounded by its bytes (each row read and written once).  A warp has a few consecutive tokens; their
// sequence is found by a 32-way search, their rows and pages looked up by a lane each, and
// then all lanes copy 16 bytes of a token's heads at a time, all loads of a step before the first store.
// 16,392 tokens of 8 heads, 2 KB of keys and of values each: 26.7 us, 5.0 TB/s.  The status word is cleared by a kernel that
// this one overlaps: one call takes 8.3 us with its host side (10.7 behind a memset).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_spec.cuh"

namespace kda {
namespace {

__global__ void clear_kernel(uint32_t *words) {
    spec::grid_go();
    if (threadIdx.x < 2) words[threadIdx.x] = 0;
}

}  // namespace

namespace spec {

bool clear_words(void *workspace, cudaStream_t s) {
    clear_kernel<<<1, 32, 0, s>>>(static_cast<uint32_t *>(workspace));
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

__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendParams p, int64_t es) {
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
                const int64_t r = p.rows ? static_cast<int64_t>(p.rows[j]) : j, at = s.ctx + j - s.first;
                const int64_t page = p.c.table[static_cast<int64_t>(n) * p.c.table_stride + at / p.c.page_size];
                const int64_t slot = at % p.c.page_size;
                const bool row_ok = r >= 0 && r < p.T_src, page_ok = page >= 0 && page < p.c.num_pages;
                if (row_ok && page_ok) {
                    row = r;
                    place_k = (page * p.c.kp + slot * p.c.kr) * es;
                    place_v = (page * p.c.vp + slot * p.c.vr) * es;
                } else {
                    raise(p.status, row_ok ? DEV_ERR_PAGE : DEV_ERR_SLOT);
                }
            }
        }
        __syncwarp();
        for (int i = 0; i < p.per; ++i) {
            const int64_t r = __shfl_sync(0xffffffffu, row, i);
            const int64_t pk = __shfl_sync(0xffffffffu, place_k, i), pv = __shfl_sync(0xffffffffu, place_v, i);
            if (r < 0) continue;
            const CopySide k{p.k + r * p.ks * 16, p.c.k + pk, p.c.kh * es, p.Hkv << p.kshift, p.kshift};
            const CopySide v{p.v + r * p.vs * 16, p.c.v + pv, p.c.vh * es, p.Hkv << p.vshift, p.vshift};
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
    if (N < 0 || A_total < 0 || T_src < 0 || Hkv <= 0 || Hkv > 4096) return KDA_ERR_INVALID_ARGUMENT;
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
    if (!clear_words(workspace, s)) return KDA_ERR_CUDA;
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
