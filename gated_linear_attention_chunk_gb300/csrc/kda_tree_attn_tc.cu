// Tree attention on the tcgen05 tensor cores, for sequences of more than 32 query rows per KV head (bf16).
//
// The same one-pass softmax as the register kernels.  With R rows per KV head a key costs 2 (dk + dv) R operations against
// 2 (dk + dv) bytes, so from about 280 rows on the tensor cores bound it, and mma.sync reaches less than half of
// their rate.  One CTA per SM works on two streams of 128 rows x 128 keys:
//   a pair of row tiles: stream s has the rows of tile s, both take every key tile;
//   a row tile alone:    both streams have its rows, stream s takes the key tiles of parity s, and
//                        each leaves its own partial result.
// Per step of a stream S = Q K^T (128 x 128, fp32, TMEM), the softmax warps turn S into weights P (bf16, written over S in
// TMEM), O += P V (P from TMEM, V as an MN-major operand).  While one stream's softmax runs, the tensor cores work
// for the other.  The running maximum a row's weights refer to is raised only when the true one has grown by more than
// 2^8 beyond it, so O is seldom rescaled (fp32 and bf16 have the range for weights up to 2^8).  P is bf16 because both
// operands of a product have one type and V is bf16; that rounds a weight by at most 2^-8 of it (a second product with the
// remainders would add half of the tensor work).  The row's sum is fp32, of the weights before that rounding.
//
// Warps:  0-3 and 4-7 softmax of stream 0 and 1 (a thread per row), 8-11 fill the ring, 12 issues the MMAs.
// TMEM:   S0 0..127, S1 128..255, O0 256.., O1 384.. (512 columns).
// Shared memory: two Q tiles and a ring of 128-row K or V tiles, all with the 128-byte swizzle (two 64-channel
// halves), filled by 16-byte asynchronous copies: cache rows lie anywhere, a page may have any size, and rows past the end are
// filled with zeros.  The ring holds the tiles in the order in which they are consumed:
// K_0 .. K_{L-1}, V_0, K_L, V_1, K_{L+1}, .. with L = 1 for a pair and 2 for a tile alone.
//
// Four sequences of 32 nodes over 131,072 keys (8 heads on each of 4 KV heads: a pair of tiles): 275 us, 1.0 PFLOP/s.  A pair's
// step of 2 x 128 x 128 scores takes 3.4k clocks, the chain of one stream: maximum 0.6k, exponentials 1.0k (16 per clock and
// SM), PV 0.45k, QK 0.5k and the hand-offs.  A tile alone is bound by the loads, of which
// the ring keeps two or so in flight: 64 rows 235 us, 4.6 TB/s; 128 rows 247.  The compiler, which is held to 128 registers for all
// warps, spills 200 (dk = 64) to 260 bytes a thread.
//
// Every wait is bounded (2 s): a role that gives up raises the abort flag, which ends all the others' waits; the MMAs
// issued so far are drained and the TMEM is freed.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_tree_attn.cuh"

namespace kda {
namespace attn {
namespace {

using namespace ptx;

constexpr int kSoftmaxWarps = 8, kLoadWarps = 4;
constexpr int kTcThreads = 512;  // four warpgroups; the last one's other three warps have no role
constexpr float kRaise = 8.f;  // growth (log2) of a row's maximum before its reference follows

template <int DK, int DV>
struct Smem {
    static constexpr int kHalf = 128 * 128;                     // bytes of 128 rows x 64 channels
    static constexpr int kQ = DK / 64 * kHalf;
    static constexpr int kSlot = (DK > DV ? DK : DV) / 64 * kHalf;
    static constexpr int kSlots = kSlot == 2 * kHalf ? 5 : 8;
    static constexpr int kBytes = 2 * kQ + kSlots * kSlot + 1024;  // plus alignment
};

struct Control {
    uint64_t full[8], empty[8], q_full[2], q_empty[2], s_full[2], p_full[2], o_full[2], o_empty[2], drained;
    uint32_t tmem;
    int abort, bad_seen;
};

// Registers, launched with 128 for each of 512 threads: a softmax thread holds a row's 128 scores and takes 168, the
// others 88 (168 + 168 + 88 + 88 = 4 x 128).
__device__ __forceinline__ void regs_more() { asm volatile("setmaxnreg.inc.sync.aligned.u32 168;" ::: "memory"); }
__device__ __forceinline__ void regs_less() { asm volatile("setmaxnreg.dec.sync.aligned.u32 88;" ::: "memory"); }

// Two floats at a time (each rounded as by the scalar instruction).
__device__ __forceinline__ uint64_t pair2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpair2(uint64_t x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// A wait that ends after about 2 s (4e9 clocks, counted from the 64th look), or once another role has given up.  By a converged
// warp, whose lanes stay together also where it gives up: instructions of whole warps follow.
constexpr long long kPatience = 4000000000ll;
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, Control &c, uint32_t *status) {
    long long t0 = 0;
    for (uint32_t spins = 1; !__all_sync(0xffffffffu, mbar_try_wait(bar, parity)); ++spins) {
        if (spins & 63u) continue;
        if (__any_sync(0xffffffffu, *reinterpret_cast<volatile int *>(&c.abort))) return false;
        const long long now = clock64();
        if (t0 == 0) t0 = now;
        if (__any_sync(0xffffffffu, now - t0 > kPatience)) {
            *reinterpret_cast<volatile int *>(&c.abort) = 1;
            atomicOr(status, static_cast<uint32_t>(DEV_ERR_TIMEOUT));
            return false;
        }
    }
    return true;
}

// The units of a CTA: every role walks them alike.  A unit is (sequence, KV head, part, group of two row tiles),
// the group running fastest; a CTA's share is a range of the row tiles counted in that order.
struct TcWalk {
    int n, u, en, eu;                                // at unit u of sequence n; end
    int ctx, nodes, t0, nsplit, chunk, tiles, units, first;  // of the sequence; first: row tiles before it
    int head, split, group;
    bool pair;
    int key0, nctx, keys, node_end;                  // context keys, their tiles and count; drafted keys
    int ntiles;

    static __device__ __forceinline__ void boundary(const AttnParams &p, int64_t c, int total, int *n, int *u) {
        if (c >= total) {
            *n = p.N;
            *u = 0;
            return;
        }
        const int at = warp_find([&](int i) { return __ldg(&p.info_tc[i].unit0); }, p.N, c);
        const int4 a = __ldg(reinterpret_cast<const int4 *>(p.info_tc + at) + 1);
        const int off = static_cast<int>(c) - __ldg(&p.info_tc[at].unit0), tiles = a.z;
        *n = at;
        *u = off / tiles * tc_groups_of(tiles) + (off % tiles + 1) / 2;
    }
    __device__ __forceinline__ bool live() const { return n < en || (n == en && u < eu); }
    __device__ __forceinline__ void enter(const AttnParams &p) {
        // to the next unit at or after (n, u) that exists
        while (live()) {
            const int4 a = __ldg(reinterpret_cast<const int4 *>(p.info_tc + n));
            const int4 b = __ldg(reinterpret_cast<const int4 *>(p.info_tc + n) + 1);
            const int next = __ldg(&p.info_tc[n + 1].unit0);
            ctx = a.x; nodes = a.y; t0 = a.z; first = a.w; nsplit = b.x; chunk = b.y; tiles = b.z;
            units = next > a.w ? p.Hkv * nsplit * tc_groups_of(tiles) : 0;
            if (u < units) break;
            ++n;
            u = 0;
        }
        if (live()) unit();
    }
    __device__ __forceinline__ void unit() {
        const int groups = tc_groups_of(tiles), hs = u / groups;
        group = u - hs * groups;
        head = hs / nsplit;
        split = hs - head * nsplit;
        pair = 2 * group + 1 < tiles;
        key0 = split * chunk;
        keys = ctx - key0 < chunk ? ctx - key0 : chunk;
        if (keys < 0) keys = 0;
        nctx = (keys + kTcKeys - 1) / kTcKeys;
        node_end = split == nsplit - 1 ? nodes : 0;
        ntiles = nctx + (node_end > 0 ? 1 : 0);
    }
    __device__ __forceinline__ void start(const AttnParams &p) {
        const int total = __ldg(&p.info_tc[p.N].unit0);
        boundary(p, static_cast<int64_t>(total) * blockIdx.x / gridDim.x, total, &n, &u);
        boundary(p, static_cast<int64_t>(total) * (blockIdx.x + 1) / gridDim.x, total, &en, &eu);
        enter(p);
    }
    __device__ __forceinline__ void next(const AttnParams &p) {
        if (++u < units) {
            if (live()) unit();
            return;
        }
        ++n;
        u = 0;
        enter(p);
    }
};

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]) : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]) : "memory");
}

// ---- filling side -------------------------------------------------------------------------------------------
// 128 rows of `channels` x 2 bytes: half a warp takes a row, its address from the lane that looked it up (0: zeros).
template <int kChannels>
__device__ __forceinline__ void copy_rows(uint32_t dst, uint64_t row_addr, int warp, int lane, const void *any) {
    constexpr int kUnits = kChannels / 8, kSide = 32 / kUnits;  // 16-byte units of a row; rows side by side
    const int u = lane % kUnits;
    const uint32_t to = dst + (u >> 3) * (128 * 128);
#pragma unroll
    for (int i = 0; i < 32 / kSide; ++i) {
        const int at = i * kSide + lane / kUnits, r = warp * 32 + at;
        const uint64_t a = __shfl_sync(0xffffffffu, row_addr, at);
        cp16(to + r * 128 + (((u & 7) ^ (r & 7)) << 4), a ? reinterpret_cast<const char *>(a) + u * 16 : any, a != 0);
    }
}

// Arrives on a barrier once this thread's copies so far have landed (the barrier counts every thread once).
__device__ __forceinline__ void arrive_landed(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

template <int DK, int DV>
__device__ void fill(const AttnParams &p, Control &c, uint32_t q_smem, uint32_t ring) {
    using S = Smem<DK, DV>;
    const int warp = (threadIdx.x >> 5) - kSoftmaxWarps, lane = threadIdx.x & 31;
    const int mine = warp * 32 + lane;  // this thread's row of a tile
    TcWalk w;
    w.start(p);
    uint32_t item = 0;                  // ring tiles issued
    uint32_t q_uses[2] = {0, 0};
    int alone = 0;
    while (w.live()) {
        // the page of this thread's row in key tile t: loaded a tile ahead of its use
        auto page_of = [&](int t) {
            const int j = t * kTcKeys + mine;
            return t < w.nctx && j < w.keys ? __ldg(p.c.table + static_cast<int64_t>(w.n) * p.c.table_stride + (w.key0 + j) / p.c.page_size) : 0;
        };
        int page = page_of(0);
        // the query rows
        for (int s = 0; s < (w.pair ? 2 : 1); ++s) {
            const int b = w.pair ? s : (alone & 1);
            if (!wait_warp(&c.q_empty[b], (q_uses[b] & 1) ^ 1, c, p.status)) return;
            ++q_uses[b];
            const int r = (2 * w.group + s) * kTcRows + mine;
            uint64_t a = 0;
            if (r < w.nodes * p.G) {
                const int node = r / p.G;
                a = reinterpret_cast<uint64_t>(static_cast<const __nv_bfloat16 *>(p.q) + (w.t0 + node) * p.qs +
                                               static_cast<int64_t>(w.head * p.G + r - node * p.G) * DK);
            }
            copy_rows<DK>(q_smem + b * S::kQ, a, warp, lane, p.q);
            arrive_landed(&c.q_full[b]);
        }
        // the keys and values
        const int lead = w.pair ? 1 : 2;
        uint64_t k_row = 0, v_row = 0, v_wait[2] = {0, 0};  // v_wait: value rows of the last tiles whose keys were issued
        for (int t = 0; t < w.ntiles + lead; ++t) {
            k_row = v_row = 0;
            if (t < w.nctx) {
                const int j = t * kTcKeys + mine;
                if (j < w.keys) {
                    const int64_t slot = (w.key0 + j) % p.c.page_size;
                    if (page >= 0 && page < p.c.num_pages) {
                        k_row = reinterpret_cast<uint64_t>(p.c.k) + 2 * (page * p.c.kp + slot * p.c.kr + w.head * p.c.kh);
                        v_row = reinterpret_cast<uint64_t>(p.c.v) + 2 * (page * p.c.vp + slot * p.c.vr + w.head * p.c.vh);
                    } else {
                        atomicOr(p.bad + w.n, static_cast<uint32_t>(DEV_ERR_PAGE));
                        atomicOr(p.status, static_cast<uint32_t>(DEV_ERR_PAGE));
                        *reinterpret_cast<volatile int *>(&c.bad_seen) = 1;
                    }
                }
                page = page_of(t + 1);
            } else if (t < w.ntiles && mine < w.node_end) {
                const int64_t row = w.t0 + mine;
                k_row = reinterpret_cast<uint64_t>(static_cast<const __nv_bfloat16 *>(p.k) + row * p.ks + static_cast<int64_t>(w.head) * DK);
                v_row = reinterpret_cast<uint64_t>(static_cast<const __nv_bfloat16 *>(p.v) + row * p.vs + static_cast<int64_t>(w.head) * DV);
            }
            // V of tile t - lead, then K of tile t
            if (t >= lead) {
                const uint32_t slot = item % S::kSlots;
                if (!wait_warp(&c.empty[slot], ((item / S::kSlots) & 1) ^ 1, c, p.status)) return;
                copy_rows<DV>(ring + slot * S::kSlot, lead == 1 ? v_wait[0] : v_wait[1], warp, lane, p.q);
                arrive_landed(&c.full[slot]);
                ++item;
            }
            if (t < w.ntiles) {
                const uint32_t slot = item % S::kSlots;
                if (!wait_warp(&c.empty[slot], ((item / S::kSlots) & 1) ^ 1, c, p.status)) return;
                copy_rows<DK>(ring + slot * S::kSlot, k_row, warp, lane, p.q);
                arrive_landed(&c.full[slot]);
                ++item;
            }
            v_wait[1] = v_wait[0];
            v_wait[0] = v_row;
        }
        if (!w.pair) ++alone;
        w.next(p);
    }
}

// ---- issuing side (one warp) ----------------------------------------------------------------------------------
// Every lane runs this code and one is elected inside each instruction: issued that way a TMEM-operand product of this
// shape takes about half the clocks that it takes from a single thread in a branch.
__device__ __forceinline__ void mma_bf16_ss_warp(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate));
}
template <int DK, int DV>
__device__ void issue(const AttnParams &p, Control &c, uint32_t q_smem, uint32_t ring, uint32_t tmem) {
    using S = Smem<DK, DV>;
    constexpr uint32_t id_s = idesc_bf16(128, kTcKeys, false, false);  // K-major keys
    constexpr uint32_t id_o = idesc_bf16(128, DV, false, true);        // values: MN-major
    uint32_t item = 0, q_uses[2] = {0, 0}, p_uses[2] = {0, 0}, o_uses[2] = {0, 0};
    int alone = 0;
    TcWalk w;
    w.start(p);
    auto scores = [&](int s, int b, uint32_t slot) {
        const uint64_t dq = sdesc_sw128(q_smem + b * S::kQ, 16, 1024), dk = sdesc_sw128(ring + slot * S::kSlot, 16, 1024);
#pragma unroll
        for (int k = 0; k < DK / 16; ++k) {
            const uint32_t at = ((k >> 2) * S::kHalf + (k & 3) * 32) >> 4;
            mma_bf16_ss_warp(tmem + s * 128, dq + at, dk + at, id_s, k > 0 ? 1u : 0u);
        }
        mma_commit_warp(&c.s_full[s]);
    };
    auto values = [&](int s, uint32_t slot, bool first) {
        const uint64_t dv = sdesc_sw128(ring + slot * S::kSlot, S::kHalf, 1024);
#pragma unroll
        for (int k = 0; k < kTcKeys / 16; ++k)
            mma_bf16_ts_warp(tmem + 256 + s * 128, tmem + s * 128 + 8 * k, dv + ((k * 2048) >> 4), id_o, (!first || k > 0) ? 1u : 0u);
    };
    auto have = [&](uint32_t i) {  // ring tile i has landed
        const bool ok = wait_warp(&c.full[i % S::kSlots], (i / S::kSlots) & 1, c, p.status);
        return ok;
    };
    auto landed = [&] {  // the copies' writes become visible to the MMAs that follow
        fence_proxy_async_smem();
        tc_fence_after();
    };
    auto weights = [&](int s, bool first) {  // the stream's weights are there (and its O has been read)
        if (!wait_warp(&c.p_full[s], p_uses[s]++ & 1, c, p.status)) return false;
        if (first && !wait_warp(&c.o_empty[s], (o_uses[s]++ & 1) ^ 1, c, p.status)) return false;
        tc_fence_after();
        return true;
    };
    while (w.live()) {
        const int nt = w.ntiles;
        if (w.pair) {
            for (int b = 0; b < 2; ++b)
                if (!wait_warp(&c.q_full[b], q_uses[b]++ & 1, c, p.status)) return;
            if (!have(item)) return;
            landed();
            scores(0, 0, item % S::kSlots);
            scores(1, 1, item % S::kSlots);
            mma_commit_warp(&c.empty[item % S::kSlots]);
            ++item;
            for (int t = 0; t < nt; ++t) {
                const uint32_t v = item, k = item + 1;
                for (int s = 0; s < 2; ++s) {
                    if (s == 0) {  // while the softmax works
                        if (!have(v) || (t + 1 < nt && !have(k))) return;
                        landed();
                    }
                    if (!weights(s, t == 0)) return;
                    values(s, v % S::kSlots, t == 0);
                    if (s == 1) mma_commit_warp(&c.empty[v % S::kSlots]);
                    if (t + 1 < nt) {
                        scores(s, s, k % S::kSlots);
                        if (s == 1) mma_commit_warp(&c.empty[k % S::kSlots]);
                    } else {
                        mma_commit_warp(&c.o_full[s]);
                    }
                }
                item += t + 1 < nt ? 2 : 1;
            }
            mma_commit_warp(&c.q_empty[0]);
            mma_commit_warp(&c.q_empty[1]);
        } else {
            const int b = alone & 1;
            if (!wait_warp(&c.q_full[b], q_uses[b]++ & 1, c, p.status)) return;
            for (int t = 0; t < (nt < 2 ? nt : 2); ++t, ++item) {
                if (!have(item)) return;
                landed();
                scores(t, b, item % S::kSlots);
                mma_commit_warp(&c.empty[item % S::kSlots]);
            }
            for (int t = 0; t < nt; ++t) {
                const int s = t & 1;
                if (!have(item) || (t + 2 < nt && !have(item + 1))) return;  // while the softmax works
                landed();
                if (!weights(s, t < 2)) return;
                values(s, item % S::kSlots, t < 2);
                mma_commit_warp(&c.empty[item % S::kSlots]);
                ++item;
                if (t + 2 < nt) {
                    scores(s, b, item % S::kSlots);
                    mma_commit_warp(&c.empty[item % S::kSlots]);
                    ++item;
                } else {
                    mma_commit_warp(&c.o_full[s]);
                }
            }
            mma_commit_warp(&c.q_empty[b]);
            ++alone;
        }
        w.next(p);
    }
}

// ---- softmax side (a thread per row of its stream) ---------------------------------------------------------------
template <int DK, int DV>
__device__ void softmax(const AttnParams &p, Control &c, uint32_t tmem) {
    const int s = threadIdx.x >> 7, row = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>(row & 96) << 16;
    const uint32_t ts = tmem + lanes + s * 128, to = tmem + lanes + 256 + s * 128;
    // a masked score is the one that the scale takes to -inf; a scale of zero has no such score, nor has it a row whose
    // weights differ: it becomes the smallest one that has
    const float given = p.scale * kLog2e;
    const float scale = given == 0.f ? 1e-37f : given;
    const uint32_t hidden = __float_as_uint(scale > 0.f ? -INFINITY : INFINITY);
    uint32_t s_uses = 0, o_uses = 0;
    TcWalk w;
    w.start(p);
    while (w.live()) {
        const int tile = 2 * w.group + (w.pair ? s : 0);
        const int r = tile * kTcRows + row, rows = w.nodes * p.G;
        const bool live = r < rows;
        const int node = live ? r / p.G : 0, hq = w.head * p.G + (live ? r - node * p.G : 0);
        const uint32_t flag = __ldcg(p.bad + w.n);
        const int step = w.pair ? 1 : 2, t_first = w.pair ? 0 : s;
        float ref = -INFINITY, top = -INFINITY, sum = 0.f;
        for (int t = t_first; t < w.ntiles; t += step) {
            const bool drafted = t >= w.nctx;
            const int count = drafted ? w.node_end : (w.keys - t * kTcKeys < kTcKeys ? w.keys - t * kTcKeys : kTcKeys);
            const bool ragged = drafted || count < kTcKeys;
            uint64_t sees = ~0ull;
            if (drafted) sees = __ldg(p.sees + w.t0 + node);
            if (!wait_warp(&c.s_full[s], s_uses++ & 1, c, p.status)) return;
            tc_fence_after();
            // the row's scores, all in registers
            uint32_t v[kTcKeys];
#pragma unroll
            for (int x = 0; x < kTcKeys; x += 32) tmem_ld32(ts + x, *reinterpret_cast<uint32_t(*)[32]>(&v[x]));
            tmem_ld_wait();
            if (ragged) {
                // key j counts for this row: below `count`, and among the drafted nodes (at most 64) an ancestor
#pragma unroll
                for (int x = 0; x < kTcKeys; x += 32) {
                    const int here = count - x;
                    uint32_t bits = here >= 32 ? 0xffffffffu : here > 0 ? (1u << here) - 1u : 0u;
                    if (drafted) bits &= x == 0 ? static_cast<uint32_t>(sees) : static_cast<uint32_t>(sees >> 32);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (!((bits >> i) & 1u)) v[x + i] = hidden;
                }
            }
            float m4[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) m4[j] = __uint_as_float(v[j]);
            if (scale > 0.f) {
#pragma unroll
                for (int i = 4; i < kTcKeys; i += 4)
#pragma unroll
                    for (int j = 0; j < 4; ++j) m4[j] = fmaxf(m4[j], __uint_as_float(v[i + j]));
                m4[0] = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
            } else {
#pragma unroll
                for (int i = 4; i < kTcKeys; i += 4)
#pragma unroll
                    for (int j = 0; j < 4; ++j) m4[j] = fminf(m4[j], __uint_as_float(v[i + j]));
                m4[0] = fminf(fminf(m4[0], m4[1]), fminf(m4[2], m4[3]));
            }
            top = fmaxf(top, m4[0] * scale);
            // the reference follows the maximum when that has left it behind (at the first keys, always)
            const bool raise = top > ref + kRaise || (ref == -INFINITY && top > -INFINITY);
            if (__any_sync(0xffffffffu, raise)) {
                const float f = raise ? ex2(ref - top) : 1.f;
                if (raise) ref = top;
                sum *= f;
                if (t > t_first) {  // O holds sums: the scores being there, the products before them are done
#pragma unroll 1
                    for (int x = 0; x < DV; x += 8) {
                        uint32_t o[8];
                        tmem_ld8(to + x, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                        tmem_st8(to + x, o);
                    }
                }
            }
            const float base = ref == -INFINITY ? 0.f : ref;
            const uint64_t scale2 = pair2(scale, scale), base2 = pair2(-base, -base);
            uint64_t s2[2] = {0ull, 0ull};
#pragma unroll
            for (int x = 0; x < kTcKeys; x += 32) {
                uint32_t pk[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 e = unpair2(fma2(pair2(__uint_as_float(v[x + 2 * i]), __uint_as_float(v[x + 2 * i + 1])), scale2, base2));
                    const float e0 = ex2(e.x), e1 = ex2(e.y);
                    s2[i & 1] = add2(s2[i & 1], pair2(e0, e1));
                    pk[i] = pack_bf16x2(e0, e1);
                }
                tmem_st16(ts + x / 2, pk);  // over scores that have been read
            }
            const float2 sa = unpair2(s2[0]), sb = unpair2(s2[1]);
            sum += (sa.x + sa.y) + (sb.x + sb.y);
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&c.p_full[s]);
        }
        const bool any = t_first < w.ntiles;
        if (any) {
            if (!wait_warp(&c.o_full[s], o_uses++ & 1, c, p.status)) return;
            tc_fence_after();
        }
        uint32_t err = flag;
        if (*reinterpret_cast<volatile int *>(&c.bad_seen)) err |= __ldcg(p.bad + w.n);
        if (flag && row == 0) atomicOr(p.status, flag);
        const bool ok = live && !err;
        const int64_t out = static_cast<int64_t>(w.t0 + node) * p.Hq + hq;
        const bool whole = w.pair && w.nsplit == 1;
        const int64_t part = whole ? 0 : tc_part(__ldg(&p.info_tc[w.n].part0), rows, w.tiles, w.nsplit, w.head, tile, w.split, s);
        const int pitch = tc_pitch(rows, tile);
        if (any) {
            const float f = whole ? 1.f / sum : 1.f;
#pragma unroll
            for (int x = 0; x < DV; x += 32) {
                uint32_t v[32];
                tmem_ld32(to + x, v);
                tmem_ld_wait();
                if (ok && whole) {
                    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.o) + out * DV + x);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t k[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            k[j] = pack_bf16x2(__uint_as_float(v[8 * i + 2 * j]) * f, __uint_as_float(v[8 * i + 2 * j + 1]) * f);
                        dst[i] = make_uint4(k[0], k[1], k[2], k[3]);
                    }
                } else if (live && !whole) {  // [DV / 4][row]: a warp's stores are consecutive
                    uint4 *dst = reinterpret_cast<uint4 *>(p.part_o) + part * (DV / 4) + (x / 4) * pitch + row;
#pragma unroll
                    for (int i = 0; i < 8; ++i) dst[i * pitch] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                }
            }
            tc_fence_before();
            mbar_arrive(&c.o_empty[s]);
        }
        if (live && !whole) p.part_ml[part + row] = make_float2(ref, sum);
        else if (ok && p.lse) p.lse[out] = (ref + log2f(sum)) * kLn2;
        w.next(p);
    }
}

template <int DK, int DV>
__global__ void __launch_bounds__(kTcThreads, 1) attn_tc_kernel(const AttnParams p) {
    using S = Smem<DK, DV>;
    extern __shared__ char raw[];
    __shared__ Control c;
    const int warp = threadIdx.x >> 5;
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    const uint32_t q_smem = base, ring = base + 2 * S::kQ;
    grid_wait();
    grid_go();
    if (__ldg(&p.info_tc[p.N].unit0) == 0) return;  // no such sequence in the batch
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kSlots; ++i) {
            mbar_init(&c.full[i], kLoadWarps * 32);
            mbar_init(&c.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&c.q_full[i], kLoadWarps * 32);
            mbar_init(&c.q_empty[i], 1);
            mbar_init(&c.s_full[i], 1);
            mbar_init(&c.p_full[i], 128);
            mbar_init(&c.o_full[i], 1);
            mbar_init(&c.o_empty[i], 128);
        }
        mbar_init(&c.drained, 1);
        c.abort = c.bad_seen = 0;
        fence_mbar_init();
    }
    if (warp == kSoftmaxWarps + kLoadWarps) {
        tmem_alloc(&c.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = c.tmem;
    if (warp < kSoftmaxWarps) {
        regs_more();
        softmax<DK, DV>(p, c, tmem);
    } else if (warp < kSoftmaxWarps + kLoadWarps) {
        regs_less();
        fill<DK, DV>(p, c, q_smem, ring);
        cp_wait<0>();  // (after a wait that gave up, too)
    } else {
        regs_less();
    }
    if (warp == kSoftmaxWarps + kLoadWarps) {
        issue<DK, DV>(p, c, q_smem, ring, tmem);
        __syncwarp();
        mma_commit_warp(&c.drained);  // everything issued so far ends before the TMEM goes
        const long long t0 = clock64();
        while (!mbar_try_wait(&c.drained, 0) && clock64() - t0 < kPatience) {}
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kSoftmaxWarps + kLoadWarps) tmem_dealloc(tmem, 512);
}

// The parts of a row tile joined, kCombCols columns of it: four sums of every fourth part, added in order.  kWays = 4: a
// thread for each of them, where there are few tiles; 1: one thread for all.
constexpr int kCombCols = 8;

template <int DV, int kWays>
__global__ void __launch_bounds__(kWays * kTcRows) combine_tc_kernel(const AttnParams p) {
    constexpr int kSums = 4 / kWays;
    __shared__ float share[kWays == 4 ? 3 : 1][kCombCols + 1][kWays == 4 ? kTcRows : 1];
    grid_wait();
    const int n = blockIdx.x, max_tiles = gridDim.y / p.Hkv;
    const int head = blockIdx.y / max_tiles, tile = blockIdx.y - head * max_tiles, c0 = blockIdx.z * kCombCols;
    const SeqInfo s = p.info_tc[n];
    if (p.info_tc[n + 1].unit0 == s.unit0 || tile >= s.tiles) return;
    const bool alone = (tile | 1) >= s.tiles;
    if ((!alone && s.nsplit == 1) || p.bad[n]) return;
    const int row = threadIdx.x % kTcRows, chain = threadIdx.x / kTcRows, r = tile * kTcRows + row;
    const int parts = alone ? 2 * s.nsplit : s.nsplit;
    const bool live = r < s.nodes * p.G;
    const int rows = s.nodes * p.G, pitch = tc_pitch(rows, tile);
    const int64_t part0 = tc_part(s.part0, rows, s.tiles, s.nsplit, head, tile, 0, 0);
    const float2 *all_ml = p.part_ml + part0 + row;
    const float4 *all_o = reinterpret_cast<const float4 *>(p.part_o) + part0 * (DV / 4) + c0 / 4 * pitch + row;
    float m = -INFINITY;
    if (live) {
#pragma unroll 8
        for (int i = 0; i < parts; ++i) m = fmaxf(m, all_ml[static_cast<int64_t>(i) * pitch].x);
    }
    const float base = m == -INFINITY ? 0.f : m;
    float l[kSums] = {}, o[kSums][kCombCols] = {};
    if (live) {
#pragma unroll(kWays == 4 ? 8 : 2)
        for (int i0 = chain; i0 < parts; i0 += 4)
#pragma unroll
            for (int y = 0; y < kSums; ++y) {
                const int i = i0 + y;
                if (i >= parts) break;
                const float2 ml = all_ml[static_cast<int64_t>(i) * pitch];
                const float4 *src = all_o + static_cast<int64_t>(i) * pitch * (DV / 4);
                const bool empty = ml.y == 0.f;  // no keys: its sums were not written
                const float f = exp2f(ml.x - base);
                l[y] = fmaf(f, ml.y, l[y]);
#pragma unroll
                for (int j = 0; j < kCombCols / 4; ++j) {
                    const float4 v = src[j * pitch];
                    o[y][4 * j] = fmaf(f, empty ? 0.f : v.x, o[y][4 * j]);
                    o[y][4 * j + 1] = fmaf(f, empty ? 0.f : v.y, o[y][4 * j + 1]);
                    o[y][4 * j + 2] = fmaf(f, empty ? 0.f : v.z, o[y][4 * j + 2]);
                    o[y][4 * j + 3] = fmaf(f, empty ? 0.f : v.w, o[y][4 * j + 3]);
                }
            }
    }
    float sum, out_o[kCombCols];
    if constexpr (kWays == 4) {
        if (chain > 0) {
#pragma unroll
            for (int x = 0; x < kCombCols; ++x) share[chain - 1][x][row] = o[0][x];
            share[chain - 1][kCombCols][row] = l[0];
        }
        __syncthreads();
        if (chain > 0) return;
#pragma unroll
        for (int x = 0; x < kCombCols; ++x) out_o[x] = (o[0][x] + share[0][x][row]) + (share[1][x][row] + share[2][x][row]);
        sum = (l[0] + share[0][kCombCols][row]) + (share[1][kCombCols][row] + share[2][kCombCols][row]);
    } else {
#pragma unroll
        for (int x = 0; x < kCombCols; ++x) out_o[x] = (o[0][x] + o[1][x]) + (o[2][x] + o[3][x]);
        sum = (l[0] + l[1]) + (l[2] + l[3]);
    }
    if (!live) return;
    const float inv = 1.f / sum;
    const int node = r / p.G;
    const int64_t out = static_cast<int64_t>(s.t0 + node) * p.Hq + head * p.G + r - node * p.G;
    uint32_t k[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) k[j] = pack_bf16x2(out_o[2 * j] * inv, out_o[2 * j + 1] * inv);
    *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.o) + out * DV + c0) = make_uint4(k[0], k[1], k[2], k[3]);
    if (p.lse && c0 == 0) p.lse[out] = (m + log2f(sum)) * kLn2;
}

template <int DK, int DV>
cudaError_t launch(const AttnParams &p, int sms, cudaStream_t s) {
    constexpr int bytes = Smem<DK, DV>::kBytes;
    if (!smem_opt_in<attn_tc_kernel<DK, DV>>(bytes)) return cudaErrorInvalidValue;
    const cudaError_t e = launch_after(attn_tc_kernel<DK, DV>, dim3(sms), kTcThreads, bytes, s, p);
    if (e != cudaSuccess) return e;
    const dim3 grid(p.N, p.Hkv * tc_tiles_of(p.max_nodes * p.G), DV / kCombCols);
    if (static_cast<int64_t>(grid.x) * grid.y * grid.z <= 2048) return launch_after(combine_tc_kernel<DV, 4>, grid, 4 * kTcRows, 0, s, p);
    return launch_after(combine_tc_kernel<DV, 1>, grid, kTcRows, 0, s, p);
}

}  // namespace

cudaError_t launch_attn_tc(const AttnParams &p, int dk, int dv, int sms, cudaStream_t s) {
    if (dk == 128) return dv == 128 ? launch<128, 128>(p, sms, s) : launch<128, 64>(p, sms, s);
    return dv == 128 ? launch<64, 128>(p, sms, s) : launch<64, 64>(p, sms, s);
}

}  // namespace attn
}  // namespace kda
