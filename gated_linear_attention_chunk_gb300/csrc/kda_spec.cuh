// Shared by the kernels of a speculative step (rotary positions, tree attention, cache append,
// draft verification): element types, the search for a packed row's sequence, host checks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/kda.h"
#include "kda_internal.h"

namespace kda {
namespace spec {

template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
    static constexpr int kVec = 8;  // elements in 16 bytes
    static __device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
    static __device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16_rn(x); }
};
template <>
struct Elem<float> {
    static constexpr int kVec = 4;
    static __device__ __forceinline__ float to_f(float x) { return x; }
    static __device__ __forceinline__ float from_f(float x) { return x; }
};

// 16 bytes as floats and back.
__device__ __forceinline__ void unpack16(uint4 u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack16(uint4 u, float (&f)[4]) {
    f[0] = __uint_as_float(u.x);
    f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z);
    f[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ uint4 pack16(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<uint32_t *>(&v);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 pack16(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}

// The largest n in [0, N) with first(n) <= x, for non-decreasing `first` with first(0) <= x: 32 probes a
// round by a converged warp.  Any other array gives some n in range; callers check what they found.
template <typename F>
__device__ __forceinline__ int warp_find(F first, int N, int64_t x) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = N;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int64_t at = static_cast<int64_t>(lo) + static_cast<int64_t>(lane) * step;
        const bool le = at < hi && static_cast<int64_t>(first(static_cast<int>(at))) <= x;
        const int c = __popc(__ballot_sync(0xffffffffu, le));
        lo += (c > 0 ? c - 1 : 0) * step;
        hi = hi < lo + step ? hi : lo + step;
    }
    return lo;
}

inline bool dtype_ok(kda_dtype t) { return t == KDA_BF16 || t == KDA_F32; }
inline size_t elem_size(kda_dtype t) { return t == KDA_BF16 ? 2 : 4; }
inline bool aligned_to(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool dim_ok(int d) { return d == 64 || d == 128; }

// SMs of the current device (0 on failure).  A device attribute does not change: looked up once per device.
int sm_count();

// Opts a kernel into `bytes` of dynamic shared memory, once per device (devices past the 64th: in every call).
template <auto kKernel>
inline bool smem_opt_in(int bytes) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
    if (done.load(std::memory_order_relaxed) & bit) return true;
    if (cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
    done.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

// A launch that may begin before the one ahead of it in the stream has ended: the kernel calls grid_wait() before it touches what
// that one writes, and in any case before it ends.
template <typename... P, typename... A>
inline cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, const A &...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
// Ends when every grid before this one has ended and its writes are visible.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the next grid in the stream begin (it waits for this one's end all the same).
__device__ __forceinline__ void grid_go() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Clears the status word and the word behind it, and looks cu over: word 2 becomes 1 if it falls somewhere, else 0.  If it falls,
// begins_low[n] (N entries, or null) says whether sequence n begins below an earlier entry.  A kernel launched after it with the
// programmatic attribute begins once everything before this call has ended; it waits (grid_wait) before it touches these words,
// and before it ends.
bool check_lengths(void *workspace, const int32_t *cu, int N, uint64_t *begins_low, cudaStream_t s);

// In shared memory: the maximum of all values that lower-numbered threads gave, and that all threads gave in earlier rounds.  For
// whole CTAs of whole warps.
struct RunningMax {
    int warp_top[2][32], base[2];
    __device__ __forceinline__ void begin() {
        if (threadIdx.x == 0) base[0] = INT32_MIN;
        __syncthreads();
    }
    __device__ __forceinline__ int next(int x, int round) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = round & 1;
        int top = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, top, o);
            if (lane >= o) top = max(top, y);
        }
        if (lane == 31) warp_top[b][warp] = top;
        int before = __shfl_up_sync(0xffffffffu, top, 1);
        __syncthreads();
        before = lane == 0 ? base[b] : max(before, base[b]);
        for (int w = 0; w < warp; ++w) before = max(before, warp_top[b][w]);
        if (threadIdx.x == blockDim.x - 1) base[b ^ 1] = max(before, x);
        return before;
    }
};

// A page pool as the kernels see it (strides in elements).
struct Pages {
    char *k, *v;
    int64_t kp, kr, kh, vp, vr, vh;
    int64_t num_pages, table_stride;
    const int32_t *table, *ctx_len;
    int page_size, max_pages;
};

// Host checks of a kda_paged_kv: 16-byte aligned pools and strides, sane sizes.
inline kda_status check_pages(const kda_paged_kv *c, kda_dtype dtype, int N, Pages *out) {
    if (!c) return KDA_ERR_INVALID_ARGUMENT;
    const int64_t vec = 16 / static_cast<int64_t>(elem_size(dtype));
    if (c->page_size <= 0 || c->max_pages < 0 || c->num_pages < 0) return KDA_ERR_INVALID_ARGUMENT;
    if (static_cast<int64_t>(c->page_size) * c->max_pages > 0x7fffffffLL) return KDA_ERR_INVALID_ARGUMENT;
    if (c->table_stride < c->max_pages && N > 1) return KDA_ERR_INVALID_ARGUMENT;
    for (int64_t s : {c->k_page_stride, c->k_row_stride, c->k_head_stride, c->v_page_stride, c->v_row_stride,
                      c->v_head_stride})
        if (s < 0 || s % vec != 0) return KDA_ERR_INVALID_ARGUMENT;
    if (N > 0 && (!c->ctx_len || !aligned_to(c->ctx_len, 4))) return KDA_ERR_INVALID_ARGUMENT;
    if (N > 0 && c->max_pages > 0 && (!c->block_table || !aligned_to(c->block_table, 4))) return KDA_ERR_INVALID_ARGUMENT;
    if (c->num_pages > 0 && (!c->k || !c->v)) return KDA_ERR_INVALID_ARGUMENT;
    if (!aligned_to(c->k, 16) || !aligned_to(c->v, 16)) return KDA_ERR_INVALID_ARGUMENT;
    *out = Pages{static_cast<char *>(c->k), static_cast<char *>(c->v), c->k_page_stride, c->k_row_stride,
                 c->k_head_stride, c->v_page_stride, c->v_row_stride, c->v_head_stride, c->num_pages,
                 c->table_stride, c->block_table, c->ctx_len, c->page_size, c->max_pages};
    return KDA_OK;
}

}  // namespace spec
}  // namespace kda
