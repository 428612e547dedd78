// Rotary positions of q and k, and their gradient.
//
// Pair j of a head at position p turns by t = p w_j:
//     (a, b) -> m (a cos t - b sin t, a sin t + b cos t),
// and the gradient is the transposed map, the same with -t.
//
// The angle is reduced exactly: w_j / 2 pi is kept as a 64-bit fixed-point fraction of a turn
// (rounded once, 2^-53 relative), so p times it modulo one turn is the low 64 bits of an integer
// product, with no error that grows beyond |p| 2^-54 turns.  Its signed top 32 bits then go
// through sincospif.
//
// The bytes of q and k, read and written once, bound it.  A CTA takes kTokens tokens at a time: one
// sine and cosine per (token, pair) into shared memory, used by every head of that token; a thread
// keeps one 16-byte column of a head (half layout: the two 16-byte halves of its pairs) and
// walks the (token, head) rows.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "kda_spec.cuh"

namespace kda {
namespace spec {

int sm_count() {
    static std::atomic<int> count[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev >= 0 && dev < 64 && (n = count[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (dev >= 0 && dev < 64) count[dev].store(n, std::memory_order_relaxed);
    return n;
}

}  // namespace spec

namespace {

using namespace spec;

constexpr int kRopeThreads = 256;
constexpr int kTokens = 4;  // tokens whose sines and cosines a CTA holds at a time

struct RopeParams {
    const void *q, *k;
    void *q_out, *k_out;
    const int32_t *positions;
    const double *inv_freq;
    int64_t T, qs, ks, qos, kos;  // token strides in elements
    int Hq, Hk, d, rot;
    int cols;        // columns of a head: kVec-wide rotated ones (pairs of them in the half layout), then copied ones
    int rot_cols;
    int lanes;       // columns taken side by side: min(cols, threads)
    int rows;        // (token, head) rows taken side by side: threads / lanes
    float mscale, sign;
};

// kVector: a column is 16 bytes; otherwise a single pair (rotated) or channel (copied).
template <typename T, bool kInterleaved, bool kVector>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
    extern __shared__ char smem[];
    constexpr int V = kVector ? Elem<T>::kVec : 1;
    const int half = p.rot / 2;
    uint64_t *turn = reinterpret_cast<uint64_t *>(smem);                // [half]
    float *cs = reinterpret_cast<float *>(smem + ((static_cast<size_t>(half) * 8 + 15) & ~static_cast<size_t>(15)));
    float *sn = cs + kTokens * half;                                    // [kTokens][half] each
    for (int j = threadIdx.x; j < half; j += kRopeThreads) {
        const double f = p.inv_freq[j] * 0.15915494309189533577;        // 1 / (2 pi)
        turn[j] = __double2ull_rz((f - floor(f)) * 18446744073709551616.0);
    }
    const int H = p.Hq + p.Hk;
    const int col0 = threadIdx.x % p.lanes;
    const int row0 = threadIdx.x / p.lanes;
    const bool live = row0 < p.rows;
    __syncthreads();
    for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTokens; t0 < p.T; t0 += static_cast<int64_t>(gridDim.x) * kTokens) {
        const int nt = static_cast<int>(p.T - t0 < kTokens ? p.T - t0 : kTokens);
        for (int e = threadIdx.x; e < nt * half; e += kRopeThreads) {
            const int t = e / half, j = e - t * half;
            const uint64_t a = static_cast<uint64_t>(static_cast<int64_t>(p.positions[t0 + t])) * turn[j];
            const float x = static_cast<float>(static_cast<int32_t>(a >> 32)) * 4.656612873077392578e-10f;  // half turns
            float s, c;
            sincospif(x, &s, &c);
            cs[e] = c * p.mscale;
            sn[e] = s * p.mscale * p.sign;
        }
        __syncthreads();
        if (live) {
            for (int r = row0 + static_cast<int>(blockIdx.y) * p.rows; r < nt * H; r += p.rows * gridDim.y) {
                const int t = r / H, h = r - t * H;
                const bool is_q = h < p.Hq;
                const int64_t tok = t0 + t;
                const T *x = is_q ? static_cast<const T *>(p.q) + tok * p.qs + static_cast<int64_t>(h) * p.d
                                  : static_cast<const T *>(p.k) + tok * p.ks + static_cast<int64_t>(h - p.Hq) * p.d;
                T *y = is_q ? static_cast<T *>(p.q_out) + tok * p.qos + static_cast<int64_t>(h) * p.d
                            : static_cast<T *>(p.k_out) + tok * p.kos + static_cast<int64_t>(h - p.Hq) * p.d;
                const float *c = cs + t * half, *s = sn + t * half;
                for (int col = col0; col < p.cols; col += p.lanes) {
                    if (col >= p.rot_cols) {
                        const int i = p.rot + (col - p.rot_cols) * V;
                        if constexpr (kVector)
                            *reinterpret_cast<uint4 *>(y + i) = *reinterpret_cast<const uint4 *>(x + i);
                        else
                            y[i] = x[i];
                    } else if constexpr (!kVector) {
                        const int ia = kInterleaved ? 2 * col : col, ib = kInterleaved ? 2 * col + 1 : col + half;
                        const float a = Elem<T>::to_f(x[ia]), b = Elem<T>::to_f(x[ib]);
                        y[ia] = Elem<T>::from_f(a * c[col] - b * s[col]);
                        y[ib] = Elem<T>::from_f(a * s[col] + b * c[col]);
                    } else if constexpr (kInterleaved) {
                        float f[V], g[V];
                        unpack16(*reinterpret_cast<const uint4 *>(x + col * V), f);
    #pragma unroll
                        for (int i = 0; i < V / 2; ++i) {
                            const float cc = c[col * (V / 2) + i], ss = s[col * (V / 2) + i];
                            g[2 * i] = f[2 * i] * cc - f[2 * i + 1] * ss;
                            g[2 * i + 1] = f[2 * i] * ss + f[2 * i + 1] * cc;
                        }
                        *reinterpret_cast<uint4 *>(y + col * V) = pack16(g);
                    } else {
                        float a[V], b[V], ya[V], yb[V];
                        unpack16(*reinterpret_cast<const uint4 *>(x + col * V), a);
                        unpack16(*reinterpret_cast<const uint4 *>(x + half + col * V), b);
    #pragma unroll
                        for (int i = 0; i < V; ++i) {
                            const float cc = c[col * V + i], ss = s[col * V + i];
                            ya[i] = a[i] * cc - b[i] * ss;
                            yb[i] = a[i] * ss + b[i] * cc;
                        }
                        *reinterpret_cast<uint4 *>(y + col * V) = pack16(ya);
                        *reinterpret_cast<uint4 *>(y + half + col * V) = pack16(yb);
                    }
                }
            }
        }
        __syncthreads();
    }
}

template <typename T>
kda_status launch_rope(RopeParams p, bool interleaved, bool vector, cudaStream_t s) {
    const int V = vector ? Elem<T>::kVec : 1;
    p.rot_cols = vector ? (interleaved ? p.rot / V : p.rot / 2 / V) : p.rot / 2;
    p.cols = p.rot_cols + (p.d - p.rot) / V;
    p.lanes = p.cols < kRopeThreads ? p.cols : kRopeThreads;
    p.rows = kRopeThreads / p.lanes;
    const size_t smem = ((static_cast<size_t>(p.rot / 2) * 8 + 15) & ~static_cast<size_t>(15)) +
                        static_cast<size_t>(kTokens) * p.rot * sizeof(float);
    const int64_t groups = (p.T + kTokens - 1) / kTokens;
    const int64_t most = static_cast<int64_t>(spec::sm_count()) * 8;
    if (most <= 0) return KDA_ERR_CUDA;
    const int64_t gx = groups < most ? groups : most;
    // few tokens: their heads are spread over several CTAs
    const int64_t steps = (static_cast<int64_t>(kTokens) * (p.Hq + p.Hk) + p.rows - 1) / p.rows;
    int64_t gy = most / gx < steps ? most / gx : steps;
    gy = gy < 1 ? 1 : gy > 64 ? 64 : gy;
    const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy));
    if (interleaved) {
        if (vector) rope_kernel<T, true, true><<<grid, kRopeThreads, smem, s>>>(p);
        else rope_kernel<T, true, false><<<grid, kRopeThreads, smem, s>>>(p);
    } else {
        if (vector) rope_kernel<T, false, true><<<grid, kRopeThreads, smem, s>>>(p);
        else rope_kernel<T, false, false><<<grid, kRopeThreads, smem, s>>>(p);
    }
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status rope(const void *q, const void *k, kda_dtype dtype, const int32_t *positions, const double *inv_freq,
                int64_t T, int Hq, int Hk, int d, int rot, int64_t qs, int64_t ks, int interleaved, float mscale,
                float sign, void *q_out, void *k_out, int64_t qos, int64_t kos, void *stream) {
    if (!dtype_ok(dtype)) return KDA_ERR_UNSUPPORTED;
    if (d <= 0 || d % 8 != 0 || d > 1024) return KDA_ERR_UNSUPPORTED;
    if (rot < 0 || rot > d || rot % 2 != 0 || T < 0 || Hq <= 0 || Hk < 0) return KDA_ERR_INVALID_ARGUMENT;
    if (Hk > 0 && !k) Hk = 0;
    if (!qs) qs = static_cast<int64_t>(Hq) * d;
    if (!ks) ks = static_cast<int64_t>(Hk) * d;
    if (!qos) qos = static_cast<int64_t>(Hq) * d;
    if (!kos) kos = static_cast<int64_t>(Hk) * d;
    const int64_t wide = static_cast<int64_t>(Hq) * d, widek = static_cast<int64_t>(Hk) * d;
    if (qs < wide || qos < wide || ks < widek || kos < widek) return KDA_ERR_INVALID_ARGUMENT;
    if (T == 0) return KDA_OK;
    const size_t es = elem_size(dtype);
    if (!q || !q_out || !positions || (rot > 0 && !inv_freq) || (Hk > 0 && !k_out)) return KDA_ERR_INVALID_ARGUMENT;
    if (!aligned_to(q, es) || !aligned_to(q_out, es) || !aligned_to(k, es) || !aligned_to(k_out, es) ||
        !aligned_to(positions, 4) || !aligned_to(inv_freq, 8))
        return KDA_ERR_INVALID_ARGUMENT;
    const int V = dtype == KDA_BF16 ? 8 : 4;
    bool vector = aligned_to(q, 16) && aligned_to(q_out, 16) && qs % V == 0 && qos % V == 0 && rot % V == 0 &&
                  (interleaved || (rot / 2) % V == 0);
    if (Hk > 0) vector = vector && aligned_to(k, 16) && aligned_to(k_out, 16) && ks % V == 0 && kos % V == 0;
    RopeParams p{q, k, q_out, k_out, positions, inv_freq, T, qs, ks, qos, kos, Hq, Hk, d, rot, 0, 0, 0, 0, mscale, sign};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == KDA_BF16 ? launch_rope<__nv_bfloat16>(p, interleaved != 0, vector, s)
                             : launch_rope<float>(p, interleaved != 0, vector, s);
}

}  // namespace
}  // namespace kda

extern "C" {

kda_status kda_rope(const void *q, const void *k, kda_dtype dtype, const int32_t *positions, const double *inv_freq,
                    int64_t T, int Hq, int Hk, int d, int rot, int64_t q_stride, int64_t k_stride, int interleaved,
                    float mscale, void *q_out, void *k_out, int64_t q_out_stride, int64_t k_out_stride, void *stream) {
    return kda::rope(q, k, dtype, positions, inv_freq, T, Hq, Hk, d, rot, q_stride, k_stride, interleaved, mscale, 1.f,
                     q_out, k_out, q_out_stride, k_out_stride, stream);
}

kda_status kda_rope_bwd(const void *d_q_out, const void *d_k_out, kda_dtype dtype, const int32_t *positions,
                        const double *inv_freq, int64_t T, int Hq, int Hk, int d, int rot, int64_t q_stride,
                        int64_t k_stride, int interleaved, float mscale, void *d_q, void *d_k, int64_t q_out_stride,
                        int64_t k_out_stride, void *stream) {
    return kda::rope(d_q_out, d_k_out, dtype, positions, inv_freq, T, Hq, Hk, d, rot, q_stride, k_stride, interleaved,
                     mscale, -1.f, d_q, d_k, q_out_stride, k_out_stride, stream);
}

}  // extern "C"
