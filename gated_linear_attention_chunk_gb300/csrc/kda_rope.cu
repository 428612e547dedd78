// Rotary positions of q and k, and their gradient.
//
// Pair j of a head at position p turns by t = p w_j:
//     (a, b) -> m (a cos t - b sin t, a sin t + b cos t),
// and the gradient is the transposed map, the same with -t.
//
// The angle is reduced without a loss of its own: w_j / 2 pi is kept as a 64-bit fixed-point fraction of a
// turn (two fp64 roundings, 2^-52 relative, and 2^-64), so p times it modulo one turn is the low 64 bits of an integer product,
// and the angle is off by |p w_j| 2^-52 radians and |p| 2^-64 turns at most: less than the rounding that follows up to
// |p w_j| of about 2^27.  Its signed top 32 bits go through sincospif as an fp32 number (2^-24 of a half turn: the
// products after it are fp32 as well).
//
// The bytes of q and k, read and written once, bound it.  A CTA takes up to kTokens tokens at a time: one
// sine and cosine per (token, pair) into shared memory, used by every head of that token; a thread
// keeps one 16-byte column of a head (half layout: the two 16-byte halves of its pairs) and
// walks the (token, head) rows, two in flight.  16,384 tokens of 32 + 8 heads of 128, bf16: 57.5 us, 5.8 TB/s (a persistent grid
// 62.6 us; four rows in flight, at fewer CTAs per SM, 64.1; eight tokens per CTA 58.4 to 68.5).  Rows or rotated widths that are no
// multiple of 16 bytes go by single elements: 231 us for the same tokens with 126 rotated channels.
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
constexpr int kTokens = 4;  // at most so many tokens' sines and cosines are held at a time
constexpr int kUnroll = 2;  // rows in flight per thread

struct RopeParams {
    const void *q, *k;
    void *q_out, *k_out;
    const int32_t *positions;
    const double *inv_freq;
    int64_t T, qs, ks, qos, kos;  // token strides in elements
    int Hq, Hk, d, rot;
    int tokens;      // tokens of a CTA at a time
    int cols;        // columns of a head: kVec-wide rotated ones (pairs of them in the half layout), then copied ones
    int rot_cols;
    int lanes;       // columns taken side by side: min(cols, threads)
    int rows;        // (token, head) rows taken side by side: threads / lanes
    float mscale, sign;
};

// What a thread holds of one row: kVector: a 16-byte column, or in the half layout the two columns of its pairs;
// otherwise a single pair (rotated) or channel (copied).
template <typename T, bool kInterleaved, bool kVector>
struct Piece {
    static constexpr int V = kVector ? Elem<T>::kVec : 1;
    uint4 a, b;  // kVector
    T x, y;      // not kVector

    __device__ __forceinline__ void load(const RopeParams &p, const T *row, int col) {
        const int half = p.rot / 2;
        if (col >= p.rot_cols) {
            const int i = p.rot + (col - p.rot_cols) * V;
            if constexpr (kVector) a = *reinterpret_cast<const uint4 *>(row + i);
            else x = row[i];
        } else if constexpr (kVector) {
            a = *reinterpret_cast<const uint4 *>(row + col * V);
            if constexpr (!kInterleaved) b = *reinterpret_cast<const uint4 *>(row + half + col * V);
        } else {
            x = row[kInterleaved ? 2 * col : col];
            y = row[kInterleaved ? 2 * col + 1 : col + half];
        }
    }
    // c, s: the token's cosines and sines
    __device__ __forceinline__ void store(const RopeParams &p, T *row, int col, const float *c, const float *s) const {
        const int half = p.rot / 2;
        if (col >= p.rot_cols) {
            const int i = p.rot + (col - p.rot_cols) * V;
            if constexpr (kVector) *reinterpret_cast<uint4 *>(row + i) = a;
            else row[i] = x;
        } else if constexpr (!kVector) {
            const float u = Elem<T>::to_f(x), v = Elem<T>::to_f(y);
            row[kInterleaved ? 2 * col : col] = Elem<T>::from_f(u * c[col] - v * s[col]);
            row[kInterleaved ? 2 * col + 1 : col + half] = Elem<T>::from_f(u * s[col] + v * c[col]);
        } else if constexpr (kInterleaved) {
            float f[V], g[V];
            unpack16(a, f);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const float cc = c[col * (V / 2) + i], ss = s[col * (V / 2) + i];
                g[2 * i] = f[2 * i] * cc - f[2 * i + 1] * ss;
                g[2 * i + 1] = f[2 * i] * ss + f[2 * i + 1] * cc;
            }
            *reinterpret_cast<uint4 *>(row + col * V) = pack16(g);
        } else {
            float u[V], v[V], yu[V], yv[V];
            unpack16(a, u);
            unpack16(b, v);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float cc = c[col * V + i], ss = s[col * V + i];
                yu[i] = u[i] * cc - v[i] * ss;
                yv[i] = u[i] * ss + v[i] * cc;
            }
            *reinterpret_cast<uint4 *>(row + col * V) = pack16(yu);
            *reinterpret_cast<uint4 *>(row + half + col * V) = pack16(yv);
        }
    }
};

template <typename T, bool kInterleaved, bool kVector>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
    extern __shared__ char smem[];
    const int half = p.rot / 2;
    uint64_t *turn = reinterpret_cast<uint64_t *>(smem);                // [half]
    float *cs = reinterpret_cast<float *>(smem + ((static_cast<size_t>(half) * 8 + 15) & ~static_cast<size_t>(15)));
    float *sn = cs + p.tokens * half;                                   // [tokens][half] each
    for (int j = threadIdx.x; j < half; j += kRopeThreads) {
        const double f = p.inv_freq[j] * 0.15915494309189533577;        // 1 / (2 pi)
        turn[j] = __double2ull_rz((f - floor(f)) * 18446744073709551616.0);
    }
    const int H = p.Hq + p.Hk;
    const int col0 = threadIdx.x % p.lanes, row0 = threadIdx.x / p.lanes + static_cast<int>(blockIdx.y) * p.rows;
    const int step = p.rows * gridDim.y;
    const bool live = threadIdx.x / p.lanes < p.rows;
    __syncthreads();
    for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.tokens; t0 < p.T; t0 += static_cast<int64_t>(gridDim.x) * p.tokens) {
        const int nt = static_cast<int>(p.T - t0 < p.tokens ? p.T - t0 : p.tokens);
        const int rows = live ? nt * H : 0;
        // the i-th row from r on: its source, destination and token
        auto src = [&](int r) -> const T * {
            const int t = r / H, h = r - t * H;
            return h < p.Hq ? static_cast<const T *>(p.q) + (t0 + t) * p.qs + static_cast<int64_t>(h) * p.d
                            : static_cast<const T *>(p.k) + (t0 + t) * p.ks + static_cast<int64_t>(h - p.Hq) * p.d;
        };
        auto dst = [&](int r) -> T * {
            const int t = r / H, h = r - t * H;
            return h < p.Hq ? static_cast<T *>(p.q_out) + (t0 + t) * p.qos + static_cast<int64_t>(h) * p.d
                            : static_cast<T *>(p.k_out) + (t0 + t) * p.kos + static_cast<int64_t>(h - p.Hq) * p.d;
        };
        Piece<T, kInterleaved, kVector> x[kUnroll];
        auto load = [&](int r, int col) {
#pragma unroll
            for (int i = 0; i < kUnroll; ++i)
                if (r + i * step < rows) x[i].load(p, src(r + i * step), col);
        };
        load(row0, col0);  // on its way while the sines are computed
        for (int e = threadIdx.x; e < nt * half; e += kRopeThreads) {
            const int t = e / half, j = e - t * half;
            const uint64_t a = static_cast<uint64_t>(static_cast<int64_t>(p.positions[t0 + t])) * turn[j];
            const float h = static_cast<float>(static_cast<int32_t>(a >> 32)) * 4.656612873077392578e-10f;  // half turns
            float s, c;
            sincospif(h, &s, &c);
            cs[e] = c * p.mscale;
            sn[e] = s * p.mscale * p.sign;
        }
        __syncthreads();
        for (int col = col0; col < p.cols; col += p.lanes)
            for (int r = row0; r < rows; r += kUnroll * step) {
                if (col != col0 || r != row0) load(r, col);
#pragma unroll
                for (int i = 0; i < kUnroll; ++i) {
                    const int at = r + i * step;
                    if (at < rows) x[i].store(p, dst(at), col, cs + at / H * half, sn + at / H * half);
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
    const int64_t most = static_cast<int64_t>(spec::sm_count()) * 8;
    if (most <= 0) return KDA_ERR_CUDA;
    // few tokens: fewer per CTA, and their heads spread over several CTAs
    const int64_t share = p.T / most;
    p.tokens = static_cast<int>(share < 1 ? 1 : share > kTokens ? kTokens : share);
    const size_t smem = ((static_cast<size_t>(p.rot / 2) * 8 + 15) & ~static_cast<size_t>(15)) +
                        static_cast<size_t>(p.tokens) * p.rot * sizeof(float);
    const int64_t groups = (p.T + p.tokens - 1) / p.tokens;
    const int64_t gx = groups < 0x7fffffffLL ? groups : 0x7fffffffLL;
    const int64_t steps = (static_cast<int64_t>(p.tokens) * (p.Hq + p.Hk) + p.rows - 1) / p.rows;
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
    RopeParams p{q, k, q_out, k_out, positions, inv_freq, T, qs, ks, qos, kos, Hq, Hk, d, rot, 0, 0, 0, 0, 0, mscale, sign};
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
