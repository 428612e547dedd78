// Attention over a shared prefix on the tcgen05 tensor cores (bf16).
//
// With R query rows per KV head a key costs 2 (dk + dv) R operations against 2 (dk + dv) bytes, so the bytes bound it up to
// about 280 rows and the tensor cores beyond.  One CTA per SM works on two streams of 128 rows x 128 keys:
//   a block of more than 128 rows: stream s has rows 128 s .. of it, both take every key tile;
//   a smaller block:               both streams have its rows, stream s takes the key tiles of parity s.
// Per step of a stream S = Q K^T (128 x 128, fp32, TMEM), its softmax warps turn S into weights P (bf16, over S in TMEM),
// O += P V (P from TMEM, V as an MN-major operand).  While one stream's softmax runs, the tensor cores work for the other.
//
// The softmax of a step is one pass: weights are taken against the reference that the row has, while the maximum is looked for
// beside them.  Only where the maximum lies more than 2^8 above the reference (or, before there is any weight, 2^60 below it)
// does the reference move there; the step's scores, which are still in TMEM, are then read again and O is rescaled.  (fp32 and
// bf16 have the range for weights up to 2^8.)  So the maximum is not waited for, and the exponentials start with the first
// scores.  P is bf16 because both operands of a product have one type and V is bf16; that rounds a weight by at most 2^-8 of
// it. The row's sum is fp32, of the weights before that rounding.
//
// Warps:  0-3 and 4-7 softmax of stream 0 and 1 (a thread per row), 8 fills the ring, 9 issues the MMAs.
// TMEM:   S0 0..127, S1 128..255, O0 256.., O1 384.. (512 columns).
// Shared memory: two Q tiles and a ring of 128-row K or V tiles, all with the 128-byte swizzle (two 64-channel halves).  A tile of
// keys is a page's part of 128 rows, or as many whole pages as fit, each from a row that is a multiple of eight (page_size 20: five
// pages at rows 0, 24, ..); TMA copies one page's rows at a time.  (A page of 136 rows is two tiles, of 128 keys and of 8: 16
// prompts of 4,080 82 us, where pages of 64, 128 or 256 take 65 to 66, of 264 71, of 200 68 and of 24 66.)  What lies between the
// pages, and in the last tile behind the prefix, is masked in S and zero in V.  The ring holds the tiles in the order in which
// they are consumed: K_0 .. K_{L-1}, V_0, K_L, V_1, K_{L+1}, .. with L = 1 for two row tiles and 2 for one.
//
// 20 to 32 bytes of spills remain at 168 registers.
//
// Of 112k clocks of a CTA of the rollout case (16 prompts, 68 us) 23k go by before its first scores: 9k until lengths are read
// and the plan is made, the rest the first walk, copies and products, code that no cache has yet as much as data.  So the
// launch may begin before the one ahead of it has ended (26 -> 21 us for one prompt together with the next), and the first
// segment is looked up once for all warps.  A step of two streams takes 3,050 clocks, of which the tensor cores work 1,800;
// issuing from two warps was slower (the streams fell into step).
//
// Every wait is bounded (2 s): a role that gives up raises the abort flag, which ends all the others' waits; the MMAs issued so
// far are drained and the TMEM is freed.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "kda_f32x2.cuh"
#include "kda_prefix_attn.cuh"
#include "sm100_ptx.cuh"

namespace kda {
namespace prefix {
namespace {

using namespace ptx;

constexpr int kSoftmaxWarps = 8, kSoftmaxThreads = 32 * kSoftmaxWarps;
constexpr int kThreads = 320;
constexpr int kRow = 128;        // rows of a tile, and keys
constexpr float kRaise = 8.f, kSink = -60.f;
constexpr int kNever = 0x7fffffff;

struct Control {
    uint64_t full[8], empty[8], q_full[2], q_empty[2], s_full[2], p_full[2], o_full[2], o_empty, x_full, drained;
    uint32_t tmem;
    int abort, bad_seen;         // a role gave up; a page was out of range
    uint32_t bad_segment[8];     // [n % 8]: n + 1, if segment n has such a page (the filling side is less than eight segments ahead)
    float2 x[2][kRow];           // a small block: both streams' references and sums
};

template <int DK, int DV>
struct Smem {
    static constexpr int kHalf = 128 * 128;                     // bytes of 128 rows x 64 channels
    static constexpr int kQ = DK / 64 * kHalf;
    static constexpr int kSlot = (DK > DV ? DK : DV) / 64 * kHalf;
    static constexpr int kSlots = kSlot == 2 * kHalf ? 5 : 8;
    static constexpr int kControl = 2 * kQ + kSlots * kSlot;
    static constexpr int kBytes = kControl + static_cast<int>(sizeof(Control));
};

struct TcParams {
    PrefixParams p;
    int page_rows;               // rows that a page takes of a tile (pages_per_tile > 0)
    int box_rows;                // rows of a copy
    bool q_boxed;                // query rows come as a tile of whole tokens, or row by row
    int head_step_k, page_step_k, head_step_v, page_step_v;  // 0 where an axis of the pool has no stride
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// A wait that ends after about 2 s (4e9 clocks, counted from the 64th look), or once another role has given up.
constexpr long long kPatience = 4000000000ll;
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, Control &c) {
    if (mbar_try_wait(bar, parity)) return true;
    long long t0 = 0;
    for (uint32_t spins = 1; !mbar_try_wait(bar, parity); ++spins) {
        if (spins & 63u) continue;
        if (*reinterpret_cast<volatile int *>(&c.abort)) return false;
        const long long now = clock64();
        if (t0 == 0) t0 = now;
        if (now - t0 > kPatience) {
            *reinterpret_cast<volatile int *>(&c.abort) = 1;
            return false;
        }
    }
    return true;
}
// By a converged warp, whose lanes stay together also where it gives up: instructions and searches of whole warps follow.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, Control &c) {
    long long t0 = 0;
    for (uint32_t spins = 1; !__all_sync(0xffffffffu, mbar_try_wait(bar, parity)); ++spins) {
        if (spins & 63u) continue;
        const long long now = clock64();
        if (t0 == 0) t0 = now;
        if (__any_sync(0xffffffffu, *reinterpret_cast<volatile int *>(&c.abort) || now - t0 > kPatience)) {
            *reinterpret_cast<volatile int *>(&c.abort) = 1;
            return false;
        }
    }
    return true;
}

// 32 columns of this thread's TMEM lane.  The registers are not to be touched before landed32.
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
__device__ __forceinline__ void landed32(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                   "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                   "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]) 
                 :: "memory");
    asm volatile("" : "+r"(r[29]), "+r"(r[30]), "+r"(r[31]) :: "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
        "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]),
        "r"(r[31])
        : "memory");
}

// ---- the tiles of a unit's keys -----------------------------------------------------------------------------------
// Keys in tile t; key_of_row gives a row's place among them (kNever: between pages).
__device__ __forceinline__ int keys_of(const TcParams &a, int len, int t) {
    if (a.p.pages_per_tile > 0) {
        const int per = a.p.pages_per_tile * a.p.c.page_size, left = len - t * per;
        return left < per ? left : per;
    }
    const int page = t / a.p.tiles_per_page, r0 = (t - page * a.p.tiles_per_page) * kRow;
    const int in_page = min(len - page * a.p.c.page_size, a.p.c.page_size) - r0;
    return in_page < kRow ? in_page : kRow;
}
__device__ __forceinline__ int key_of_row(const TcParams &a, int r) {
    if (a.p.pages_per_tile == 0) return r;
    const int j = r / a.page_rows, o = r - j * a.page_rows;
    return j < a.p.pages_per_tile && o < a.p.c.page_size ? j * a.p.c.page_size + o : kNever;
}
// Tiles that are full have their 128 rows all in place.
__device__ __forceinline__ bool has_holes(const TcParams &a) { return a.p.pages_per_tile > 0 && a.p.pages_per_tile * a.p.c.page_size != kRow; }

// ---- filling side (one warp) --------------------------------------------------------------------------------------
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, int c3, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// The first row of a block: token tok0 of the group, query head rem0 of the KV head's G.  (T Hq is below 2^31.)
struct BlockRows {
    uint32_t tok0;
    int rem0, left;  // left: rows of the block
    __device__ __forceinline__ BlockRows(const PrefixParams &p, const SegmentWalk &w) {
        const uint32_t r0 = static_cast<uint32_t>(w.block) * p.rows, rows = static_cast<uint32_t>(w.tokens) * p.G;
        tok0 = r0 / static_cast<uint32_t>(p.G);
        rem0 = static_cast<int>(r0 - tok0 * p.G);
        left = static_cast<int>(rows - r0 < p.rows ? rows - r0 : p.rows);
    }
};

// Returns the number of ring tiles issued.  The query rows come with the first keys; rows of a tile beyond them have what was
// there or rows of others (their results go nowhere).  Where G divides a tile the rows of whole tokens are a box: 32 lanes
// copying 256 rows each by itself took 10k clocks, as long as three steps, boxes of eight rows 9k.
template <int DK, int DV>
__device__ uint32_t fill(const TcParams &a, SegmentWalk w, const CUtensorMap *q_map, const CUtensorMap *k_map, const CUtensorMap *v_map, Control &c,
                         uint32_t q_smem, uint32_t ring, uint32_t (&q_uses)[2]) {
    using S = Smem<DK, DV>;
    const PrefixParams &p = a.p;
    const int lane = threadIdx.x & 31;
    uint32_t item = 0, segment = 0;
    int alone = 0;
    for (; w.live(); w.next(p), ++segment) {
        const BlockRows rows(p, w);
        const bool pair = rows.left > kRow;
        auto copy_queries = [&] {
            for (int s = 0; s < (pair ? 2 : 1); ++s) {
                const int b = pair ? s : alone & 1, n = min(rows.left - s * kRow, kRow);
                if (!wait_warp(&c.q_empty[b], (q_uses[b]++ & 1) ^ 1, c)) return false;
                if (a.q_boxed) {
                    constexpr int kHalves = DK / 64;
                    mbar_arrive_expect_tx(&c.q_full[b], lane < kHalves ? S::kHalf : 0u);
                    if (lane < kHalves)
                        tma_load_3d(q_smem + b * S::kQ + lane * S::kHalf, q_map, lane * 64, w.head * p.G,
                                    w.t0 + static_cast<int>(rows.tok0) + (s ? kRow / p.G : 0), &c.q_full[b]);
                    __syncwarp();
                    continue;
                }
                constexpr int kUnits = DK / 8, kSide = 32 / kUnits;  // 16-byte units of a row; rows side by side
                const int u = lane % kUnits;
                const __nv_bfloat16 *base = static_cast<const __nv_bfloat16 *>(p.q) + (static_cast<int64_t>(w.t0) + rows.tok0) * p.qs +
                                            static_cast<int64_t>(w.head) * p.G * DK + u * 8;
                const uint32_t dst = q_smem + b * S::kQ + (u >> 3) * S::kHalf;
                // x / G for x below G + 256 (G <= 4096)
                const uint64_t magic = (0x100000000ull + p.G - 1) / static_cast<uint32_t>(p.G);
#pragma unroll 4
                for (int r = lane / kUnits; r < n; r += kSide) {
                    const int at = rows.rem0 + s * kRow + r, tok = static_cast<int>((static_cast<uint64_t>(at) * magic) >> 32);
                    cp16(dst + r * 128 + (((u & 7) ^ (r & 7)) << 4), base + tok * p.qs + (at - tok * p.G) * DK);
                }
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&c.q_full[b])) : "memory");
            }
            if (!pair) ++alone;
            return true;
        };
        // What the page table says for this lane in tile t, and the page (-1: none).
        struct Entry {
            int page;
            bool is;
        };
        auto look_up = [&](int t) {
            int at = -1;
            if (t < w.k1) {
                if (p.pages_per_tile > 0) {
                    if (lane * p.c.page_size < keys_of(a, w.len, t) && lane < p.pages_per_tile) at = t * p.pages_per_tile + lane;
                } else if (lane == 0) {
                    at = t / p.tiles_per_page;
                }
            }
            return at < 0 ? Entry{-1, false} : Entry{p.c.table[static_cast<int64_t>(w.g) * p.c.table_stride + at], true};
        };
        auto page_of = [&](const Entry &e) {
            if (!e.is || (e.page >= 0 && e.page < p.c.num_pages)) return e.page;
            *reinterpret_cast<volatile uint32_t *>(&c.bad_segment[segment & 7]) = segment + 1;
            *reinterpret_cast<volatile int *>(&c.bad_seen) = 1;
            return -1;
        };
        auto copy = [&](const CUtensorMap *map, int halves, int head_step, int page_step, int t, int page) {
            const uint32_t slot = item % S::kSlots;
            if (!wait_warp(&c.empty[slot], ((item / S::kSlots) & 1) ^ 1, c)) return false;
            uint64_t *bar = &c.full[slot];
            const int pages = __popc(__ballot_sync(0xffffffffu, page >= 0));
            if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(pages * halves * a.box_rows) * 128u);
            __syncwarp();
            if (page >= 0) {
                const int row = p.pages_per_tile > 0 ? 0 : t % p.tiles_per_page * kRow;
                const uint32_t dst = ring + slot * S::kSlot + (p.pages_per_tile > 0 ? lane * a.page_rows * 128 : 0);
                for (int h = 0; h < halves; ++h) tma_load_4d(dst + h * S::kHalf, map, h * 64, row, w.head * head_step, page * page_step, bar);
            }
            ++item;
            return true;
        };
        const int lead = pair ? 1 : 2;
        Entry e0 = look_up(w.k0), e1 = look_up(w.k0 + 1);
        if (segment == 0 && !copy_queries()) return item;  // (while the table is read)
        int before[2] = {-1, -1};  // of the last tiles whose keys were issued
        for (int t = w.k0; t < w.k1 + lead; ++t) {
            const int page = page_of(e0);
            e0 = e1;
            e1 = look_up(t + 2);
            if (t - lead >= w.k0 && !copy(v_map, DV / 64, a.head_step_v, a.page_step_v, t - lead, lead == 1 ? before[0] : before[1])) return item;
            if (t < w.k1 && !copy(k_map, DK / 64, a.head_step_k, a.page_step_k, t, page)) return item;
            if (t == w.k0 && segment > 0 && !copy_queries()) return item;
            before[1] = before[0];
            before[0] = page;
        }
    }
    return item;
}

// ---- issuing side (one warp) --------------------------------------------------------------------------------------
// The two streams' steps follow one another through this one warp, so every instruction of it counts: it shares its scheduler
// with two softmax warps, and at one election, descriptor and vote per MMA and wait, with all it waited for long there, it took
// 3.4k clocks for a step of two streams, of which the tensor cores worked 1.8k.  So a product's MMAs are one block with one
// election, ring places and parities are counted along, and a wait looks once before anything else.
__device__ __forceinline__ uint32_t same(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }  // known to be the same in all lanes

// S = Q K^T: 128 x 128, 4 or 8 steps of 16 channels; halves of 64 channels are 16 KB apart.
template <int kSteps>
__device__ __forceinline__ void scores_mma(uint32_t d, uint64_t q, uint64_t k, uint32_t id, uint64_t *bar) {
    static_assert(kSteps == 4 || kSteps == 8, "64 or 128 channels");
    if constexpr (kSteps == 8) {
        asm volatile(
            "{\n\t.reg .pred e, no, yes;\n\t.reg .b64 a, b;\n\t"
            "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 no, 0, 0;\n\tsetp.eq.b32 yes, 0, 0;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, no;\n\t"
            "add.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, yes;\n\t"
            "add.s64 a, %1, 4;\n\tadd.s64 b, %2, 4;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, yes;\n\t"
            "add.s64 a, %1, 6;\n\tadd.s64 b, %2, 6;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, yes;\n\t"
            "add.s64 a, %1, 1024;\n\tadd.s64 b, %2, 1024;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, yes;\n\t"
            "add.s64 a, %1, 1026;\n\tadd.s64 b, %2, 1026;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, yes;\n\t"
            "add.s64 a, %1, 1028;\n\tadd.s64 b, %2, 1028;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, yes;\n\t"
            "add.s64 a, %1, 1030;\n\tadd.s64 b, %2, 1030;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, yes;\n\t"
            "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n\t}\n" ::"r"(d),
            "l"(q), "l"(k), "r"(id), "r"(smem_u32(bar))
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred e, no, yes;\n\t.reg .b64 a, b;\n\t"
            "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 no, 0, 0;\n\tsetp.eq.b32 yes, 0, 0;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, no;\n\t"
            "add.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, yes;\n\t"
            "add.s64 a, %1, 4;\n\tadd.s64 b, %2, 4;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, yes;\n\t"
            "add.s64 a, %1, 6;\n\tadd.s64 b, %2, 6;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, yes;\n\t"
            "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n\t}\n" ::"r"(d),
            "l"(q), "l"(k), "r"(id), "r"(smem_u32(bar))
            : "memory");
    }
}
// O += P V: 8 steps of 16 keys, 2 KB apart in V, 8 columns in P.
__device__ __forceinline__ void values_mma(uint32_t d, uint32_t p, uint64_t v, uint32_t id, uint32_t add_first) {
    asm volatile(
        "{\n\t.reg .pred e, first, yes;\n\t.reg .b32 a;\n\t.reg .b64 b;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 first, %4, 0;\n\tsetp.eq.b32 yes, 0, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, first;\n\t"
        "add.u32 a, %1, 8;\n\tadd.s64 b, %2, 128;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, yes;\n\t"
        "add.u32 a, %1, 16;\n\tadd.s64 b, %2, 256;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, yes;\n\t"
        "add.u32 a, %1, 24;\n\tadd.s64 b, %2, 384;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, yes;\n\t"
        "add.u32 a, %1, 32;\n\tadd.s64 b, %2, 512;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, yes;\n\t"
        "add.u32 a, %1, 40;\n\tadd.s64 b, %2, 640;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, yes;\n\t"
        "add.u32 a, %1, 48;\n\tadd.s64 b, %2, 768;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, yes;\n\t"
        "add.u32 a, %1, 56;\n\tadd.s64 b, %2, 896;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, yes;\n\t}\n" ::"r"(d),
        "r"(p), "l"(v), "r"(id), "r"(add_first)
        : "memory");
}

template <int DK, int DV>
__device__ void issue(const TcParams &a, SegmentWalk w, Control &c, char *smem, uint32_t q_smem, uint32_t ring, uint32_t tmem_any) {
    using S = Smem<DK, DV>;
    const PrefixParams &p = a.p;
    constexpr uint32_t id_s = idesc_bf16(128, kRow, false, false);  // K-major keys
    constexpr uint32_t id_o = idesc_bf16(128, DV, false, true);     // values: MN-major
    const int lane = threadIdx.x & 31;
    const uint32_t tmem = same(tmem_any);
    // descriptors of the first query tile and ring place; a place or tile on is an addition
    const uint64_t q_desc = sdesc_sw128(q_smem, 16, 1024), k_desc = sdesc_sw128(ring, 16, 1024), v_desc = sdesc_sw128(ring, S::kHalf, 1024);
    struct Place {
        uint32_t slot, parity;  // of the next ring tile
        __device__ __forceinline__ void next() {
            ++slot;
            if (slot == S::kSlots) slot = 0, parity ^= 1u;
        }
    } at{0, 0};
    uint32_t q_uses[2] = {0, 0}, p_parity[2] = {0, 0}, segment = 0;
    int alone = 0;
    auto ready = [&](uint64_t *bar, uint32_t parity) {
        if (mbar_try_wait(bar, parity)) return true;
        return wait(bar, parity, c);
    };
    auto scores = [&](int s, int b, uint32_t slot) {
        scores_mma<DK / 16>(tmem + s * 128, q_desc + static_cast<uint64_t>(b * (S::kQ >> 4)),
                            k_desc + static_cast<uint64_t>(slot * (S::kSlot >> 4)), id_s, &c.s_full[s]);
    };
    auto values = [&](int s, uint32_t slot, bool first) {
        values_mma(tmem + 256 + s * 128, tmem + s * 128, v_desc + static_cast<uint64_t>(slot * (S::kSlot >> 4)), id_o, first ? 0u : 1u);
    };
    auto release = [&](uint32_t slot) { mma_commit_warp(&c.empty[slot]); };
    for (; w.live(); w.next(p), ++segment) {
        const int nt = static_cast<int>(same(static_cast<uint32_t>(w.k1 - w.k0)));
        const bool pair = same(w.tokens * static_cast<int64_t>(p.G) - static_cast<int64_t>(w.block) * p.rows > kRow ? 1u : 0u) != 0;
        // Values have landed: in the unit's last tile the rows that are no keys become zeros.
        const int last = same(w.k1 == w.tiles ? 1u : 0u) ? nt - 1 : -1;
        auto clear_values = [&](uint32_t slot) {
            const int keys = keys_of(a, w.len, w.tiles - 1);
            if (keys < kRow || has_holes(a)) {
                char *tile = smem + (ring - q_smem) + slot * S::kSlot;
                for (int r = lane; r < kRow; r += 32)
                    if (key_of_row(a, r) >= keys)
                        for (int u = 0; u < DV / 8; ++u)
                            *reinterpret_cast<uint4 *>(tile + (u >> 3) * S::kHalf + r * 128 + (u & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async_smem();
            }
            __syncwarp();
        };
        // a role that gives up makes all give up: lanes that saw it differ for a moment only
        bool ok = true;
        auto first_weights = [&](int s) {  // the stream's first weights, and O has been read
            ok = ok && ready(&c.p_full[s], p_parity[s]) && ready(&c.o_empty, (segment & 1) ^ 1);
            p_parity[s] ^= 1u;
        };
        if (pair) {
            for (int b = 0; b < 2; ++b) ok = ok && ready(&c.q_full[b], q_uses[b]++ & 1);
            fence_proxy_async_smem();
            ok = ok && ready(&c.full[at.slot], at.parity);
            if (!__all_sync(0xffffffffu, ok)) return;
            tc_fence_after();
            scores(0, 0, at.slot);
            scores(1, 1, at.slot);
            release(at.slot);
            at.next();
            auto release_queries = [&] {
                mma_commit_warp(&c.q_empty[0]);
                mma_commit_warp(&c.q_empty[1]);
            };
            if (nt == 1) release_queries();
            for (int t = 0; t < nt; ++t) {
                const uint32_t v = at.slot;
                ok = ready(&c.full[v], at.parity);
                at.next();
                if (t == last) clear_values(v);
                const uint32_t k = at.slot;
                const bool more = t + 1 < nt;
                if (more) {
                    ok = ok && ready(&c.full[k], at.parity);
                    at.next();
                }
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (t == 0) {
                        first_weights(s);
                    } else {
                        ok = ok && ready(&c.p_full[s], p_parity[s]);
                        p_parity[s] ^= 1u;
                    }
                    if (!__all_sync(0xffffffffu, ok)) return;
                    tc_fence_after();
                    values(s, v, t == 0);
                    if (more) scores(s, s, k);
                    else mma_commit_warp(&c.o_full[s]);
                }
                release(v);
                if (more) release(k);
                if (t + 2 == nt) release_queries();  // the last scores are on their way
            }
        } else {
            const int b = alone & 1;
            ok = ready(&c.q_full[b], q_uses[b]++ & 1);
            fence_proxy_async_smem();
            for (int t = 0; t < (nt < 2 ? nt : 2); ++t) {
                ok = ok && ready(&c.full[at.slot], at.parity);
                if (!__all_sync(0xffffffffu, ok)) return;
                tc_fence_after();
                scores(t, b, at.slot);
                release(at.slot);
                at.next();
            }
            for (int t = 0; t < nt; ++t) {
                const int s = t & 1;
                const uint32_t v = at.slot;
                ok = ready(&c.full[v], at.parity);
                at.next();
                if (t == last) clear_values(v);
                const uint32_t k = at.slot;
                const bool more = t + 2 < nt;
                if (more) {
                    ok = ok && ready(&c.full[k], at.parity);
                    at.next();
                }
                if (t < 2) {
                    first_weights(s);
                } else {
                    ok = ok && ready(&c.p_full[s], p_parity[s]);
                    p_parity[s] ^= 1u;
                }
                if (!__all_sync(0xffffffffu, ok)) return;
                tc_fence_after();
                values(s, v, t < 2);
                if (more) scores(s, b, k);
                else mma_commit_warp(&c.o_full[s]);
                release(v);
                if (more) release(k);
            }
            mma_commit_warp(&c.q_empty[b]);
            ++alone;
        }
    }
}

// ---- softmax side (a thread per row of its stream) ------------------------------------------------------------------
// A step's weights from 32 scores each: packed, their sum and the largest exponent.
struct Step {
    uint64_t sum[2];
    float top;
};
__device__ __forceinline__ void weigh32(const uint32_t (&v)[32], uint64_t scale2, uint64_t base2, uint32_t *packed, Step &st) {
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
        const float2 a = both(fma2(f2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), scale2, base2));
        const float2 b = both(fma2(f2(__uint_as_float(v[2 * i + 2]), __uint_as_float(v[2 * i + 3])), scale2, base2));
        st.top = fmaxf(fmaxf(st.top, a.x), a.y);
        st.top = fmaxf(fmaxf(st.top, b.x), b.y);
        const float e0 = ex2(a.x), e1 = ex2(a.y), e2 = ex2(b.x), e3 = ex2(b.y);
        st.sum[0] = add2(st.sum[0], f2(e0, e1));
        st.sum[1] = add2(st.sum[1], f2(e2, e3));
        packed[i] = pack_bf16x2(e0, e1);
        packed[i + 1] = pack_bf16x2(e2, e3);
    }
}

template <int DK, int DV>
__device__ void softmax(const TcParams &a, SegmentWalk w, Control &c, uint32_t tmem) {
    const PrefixParams &p = a.p;
    const int s = threadIdx.x >> 7, row = threadIdx.x & 127, lane = threadIdx.x & 31;
    const uint32_t lanes = static_cast<uint32_t>(row & 96) << 16;
    const uint32_t ts = tmem + lanes + s * 128, to = tmem + lanes + 256;
    // a masked score is the one that the scale takes to -inf; a scale of zero has no such score, nor has it a row whose
    // weights differ: it becomes the smallest one that has
    const float given = p.scale * kLog2e;
    const float scale = given == 0.f ? 1e-37f : given;
    const uint32_t hidden = __float_as_uint(scale > 0.f ? -INFINITY : INFINITY);
    const uint64_t scale2 = f2(scale, scale);
    int place[4];  // keys of the columns that this lane looks after in a ragged tile
#pragma unroll
    for (int i = 0; i < 4; ++i) place[i] = key_of_row(a, 32 * i + lane);
    const bool holes = has_holes(a);
    uint32_t s_uses = 0, o_uses[2] = {0, 0}, x_uses = 0, segment = 0;
    for (; w.live(); w.next(p), ++segment) {
        const BlockRows rows(p, w);
        const bool pair = rows.left > kRow;
        const int nt = w.k1 - w.k0, step = pair ? 1 : 2, first = pair ? 0 : s;
        // where this thread's row goes, and its tail, on its way to the cache meanwhile
        const int in_block = (pair ? s * kRow : 0) + row;
        const bool there = in_block < rows.left;
        const int row_tok = (rows.rem0 + in_block) / p.G;
        const int64_t out = (static_cast<int64_t>(w.t0) + rows.tok0 + row_tok) * p.Hq + w.head * p.G + (rows.rem0 + in_block - row_tok * p.G);
        float lse_tail = 0.f;
        if (there && w.whole && p.lse_tail) {
            lse_tail = p.lse_tail[out];
            const __nv_bfloat16 *tail = static_cast<const __nv_bfloat16 *>(p.o_tail) + out * DV;
#pragma unroll
            for (int x = 0; x < DV; x += 64) asm volatile("prefetch.global.L1 [%0];" ::"l"(tail + x));
        }
        float ref = 0.f, sum = 0.f;  // weights are 2^(score - ref)
        // a single tile is weighed against its maximum: one key alone has the weight 1 then, and its value comes out as it is
        const float sink = w.tiles == 1 ? kRaise : kSink;
        for (int t = first; t < nt; t += step) {
            const int keys = keys_of(a, w.len, w.k0 + t);
            const bool ragged = holes || keys < kRow;
            uint32_t bits[4];
            if (ragged) {
#pragma unroll
                for (int i = 0; i < 4; ++i) bits[i] = __ballot_sync(0xffffffffu, place[i] < keys);
            }
            if (!wait_warp(&c.s_full[s], s_uses++ & 1, c)) return;
            tc_fence_after();
            uint32_t pk[2][32];
            Step st;
            for (bool again = false;; again = true) {
                const uint64_t base2 = f2(-ref, -ref);
                st.sum[0] = st.sum[1] = 0ull;
                st.top = -INFINITY;
                uint32_t v[2][32];
                tmem_ld32(ts, v[0]);
                landed32(v[0]);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    if (x < 3) tmem_ld32(ts + 32 * (x + 1), v[(x + 1) & 1]);
                    if (ragged) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!((bits[x] >> i) & 1u)) v[x & 1][i] = hidden;
                    }
                    weigh32(v[x & 1], scale2, base2, &pk[x >> 1][(x & 1) * 16], st);
                    if (x < 3) landed32(v[(x + 1) & 1]);
                }
                if (again) break;
                const bool move = there && (st.top > kRaise || (sum == 0.f && st.top < sink && st.top > -INFINITY));
                if (!__any_sync(0xffffffffu, move)) break;
                const float f = move && sum != 0.f ? ex2(-st.top) : 1.f;
                if (move) ref += st.top;
                sum *= f;
                if (t > first) {  // O holds sums: the scores being there, the products before them are done
#pragma unroll 1
                    for (int x = 0; x < DV; x += 32) {
                        uint32_t o[32];
                        tmem_ld32(to + s * 128 + x, o);
                        landed32(o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                        tmem_st32(to + s * 128 + x, o);
                    }
                }
            }
            tmem_st32(ts, pk[0]);  // over scores that have been read
            tmem_st32(ts + 32, pk[1]);
            const float2 sa = both(st.sum[0]), sb = both(st.sum[1]);
            sum += (sa.x + sa.y) + (sb.x + sb.y);
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&c.p_full[s]);
        }

        // the block's result: a row's columns [c0, c0 + cols) of stream s, or of both streams
        int c0 = 0;
        float f0 = 1.f, f1 = 0.f;
        if (!pair) {
            // (every thread is done with the segment before, whose values lie there)
            if (segment > 0 && !wait_warp(&c.o_empty, (segment - 1) & 1, c)) return;
            c.x[s][row] = make_float2(ref, first < nt ? sum : 0.f);
            mbar_arrive(&c.x_full);
            if (!wait_warp(&c.x_full, x_uses++ & 1, c)) return;
            const float2 x0 = c.x[0][row], x1 = c.x[1][row];
            ref = x1.y != 0.f && (x0.y == 0.f || x1.x > x0.x) ? x1.x : x0.x;
            f0 = x0.y != 0.f ? ex2(x0.x - ref) : 0.f;
            f1 = x1.y != 0.f ? ex2(x1.x - ref) : 0.f;
            // (a NaN sum is not zero and stays)
            sum = (x0.y != 0.f ? f0 * x0.y : 0.f) + (x1.y != 0.f ? f1 * x1.y : 0.f);
            c0 = s * (DV / 2);
        }
        const int cols = pair ? DV : DV / 2;
        if (pair) {
            if (!wait_warp(&c.o_full[s], o_uses[s]++ & 1, c)) return;
        } else {
            if (!wait_warp(&c.o_full[0], o_uses[0]++ & 1, c)) return;
            if (nt > 1 && !wait_warp(&c.o_full[1], o_uses[1]++ & 1, c)) return;
        }
        if (pair) ++o_uses[s ^ 1];
        tc_fence_after();
        const bool err = *reinterpret_cast<volatile uint32_t *>(&c.bad_segment[segment & 7]) == segment + 1;
        const bool live = there && !(err && w.whole);
        Join j{1.f, 0.f, 0.f};
        if (live && w.whole) j = join_tail(ref, sum, p.lse_tail != nullptr, lse_tail);
        const int64_t slot = static_cast<int64_t>(w.slot) * p.pitch + in_block;
        f0 *= j.prefix;
        f1 *= j.prefix;
        const bool use0 = pair ? sum != 0.f : f0 != 0.f, use1 = f1 != 0.f;
#pragma unroll 1
        for (int x = c0; x < c0 + cols; x += 32) {
            uint32_t v[32];
            tmem_ld32(to + (pair ? s * 128 : 0) + x, v);
            landed32(v);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = use0 ? __float_as_uint(__uint_as_float(v[i]) * f0) : 0u;
            if (!pair && nt > 1) {
                uint32_t y[32];
                tmem_ld32(to + 128 + x, y);
                landed32(y);
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = use1 ? __float_as_uint(fmaf(__uint_as_float(y[i]), f1, __uint_as_float(v[i]))) : v[i];
            }
            if (!live) continue;
            if (!w.whole) {
                uint4 *dst = reinterpret_cast<uint4 *>(p.part_o + slot * DV + x);
#pragma unroll
                for (int i = 0; i < 8; ++i) dst[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                continue;
            }
            const uint4 *tail = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.o_tail) + out * DV + x);
            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.o) + out * DV + x);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float y[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) y[k] = __uint_as_float(v[8 * i + k]);
                if (j.tail != 0.f) {
                    float z[8];
                    unpack16(tail[i], z);
#pragma unroll
                    for (int k = 0; k < 8; ++k) y[k] = fmaf(j.tail, z[k], y[k]);
                }
                dst[i] = pack16(y);
            }
        }
        tc_fence_before();
        mbar_arrive(&c.o_empty);
        if (live && !w.whole && c0 == 0) p.part_ml[slot] = make_float2(ref, err ? -1.f : sum);
        if (w.whole && p.lse && c0 == 0) {
            // in a small block two threads read lse_tail, which may be lse
            if (!pair && !wait_warp(&c.o_empty, segment & 1, c)) return;
            if (live) p.lse[out] = j.lse;
        }
    }
}

template <int DK, int DV>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_tc_kernel(const __grid_constant__ TcParams a, const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map) {
    using S = Smem<DK, DV>;
    extern __shared__ __align__(1024) char raw[];
    Control &c = *reinterpret_cast<Control *>(raw + S::kControl);
    const PrefixParams &p = a.p;
    const int warp = threadIdx.x >> 5;
    const uint32_t q_smem = smem_u32(raw), ring = q_smem + 2 * S::kQ;
    if (warp == kSoftmaxWarps) {
        if (a.q_boxed) tma_prefetch_desc(&q_map);
        tma_prefetch_desc(&k_map);
        tma_prefetch_desc(&v_map);
    }
    grid_wait();
    grid_go();
    if (!p.planned) make_plan(p, *reinterpret_cast<PlanScratch *>(raw));
    SegmentWalk w;  // here, and not by each role for itself: that is code that none of them finds in a cache
    w.start(p);
    if (!w.live()) {
        if (threadIdx.x == 0) p.errors[blockIdx.x] = 0;
        return;
    }
    if (threadIdx.x < 8) c.bad_segment[threadIdx.x] = 0;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kSlots; ++i) {
            mbar_init(&c.full[i], 1);
            mbar_init(&c.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&c.q_full[i], 32);
            mbar_init(&c.q_empty[i], 1);
            mbar_init(&c.s_full[i], 1);
            mbar_init(&c.p_full[i], 128);
            mbar_init(&c.o_full[i], 1);
        }
        mbar_init(&c.o_empty, kSoftmaxThreads);
        mbar_init(&c.x_full, kSoftmaxThreads);
        mbar_init(&c.drained, 1);
        c.abort = c.bad_seen = 0;
        fence_mbar_init();
    }
    if (has_holes(a)) {  // rows between pages stay as they are: zeros
        for (int i = threadIdx.x; i < S::kSlots * S::kSlot / 16; i += kThreads)
            reinterpret_cast<uint4 *>(raw + 2 * S::kQ)[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();  // these zeros, and the plan's scratch, lie where copies will write
    if (warp == kSoftmaxWarps + 1) {
        tmem_alloc(&c.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = c.tmem;
    if (warp < kSoftmaxWarps) {
        softmax<DK, DV>(a, w, c, tmem);
    } else if (warp == kSoftmaxWarps) {
        uint32_t q_uses[2] = {0, 0};
        const uint32_t items = fill<DK, DV>(a, w, &q_map, &k_map, &v_map, c, q_smem, ring, q_uses);
        asm volatile("cp.async.wait_all;" ::: "memory");
        // the copies issued last end before the shared memory goes (after a wait that gave up, too)
        const long long t0 = clock64();
        for (uint32_t i = items > S::kSlots ? items - S::kSlots : 0; i < items; ++i)
            while (!mbar_try_wait(&c.full[i % S::kSlots], (i / S::kSlots) & 1) && clock64() - t0 < kPatience) {}
        for (int b = 0; b < 2; ++b)
            while (q_uses[b] > 0 && !mbar_try_wait(&c.q_full[b], (q_uses[b] - 1) & 1) && clock64() - t0 < kPatience) {}
        __syncwarp();
    } else {
        issue<DK, DV>(a, w, c, raw, q_smem, ring, tmem);
        __syncwarp();
        mma_commit_warp(&c.drained);  // everything issued so far ends before the TMEM goes
        const long long t0 = clock64();
        while (!mbar_try_wait(&c.drained, 0) && clock64() - t0 < kPatience) {}
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kSoftmaxWarps + 1) tmem_dealloc(tmem, 512);
    if (threadIdx.x == 0) p.errors[blockIdx.x] = (c.bad_seen ? DEV_ERR_PAGE : 0u) | (c.abort ? DEV_ERR_TIMEOUT : 0u);
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        cudaDriverEntryPointQueryResult q;
        void *ptr = nullptr;
        const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr) : nullptr;
    }();
    return fn;
}

// A pool [pages, rows, heads, d]; an axis without a stride counts as one entry.
bool encode_pool(CUtensorMap *map, const void *base, const Pages &c, int heads, int d, int64_t rs, int64_t hs, int64_t ps, int box_rows,
                 int *head_step, int *page_step) {
    auto enc = encoder();
    if (!enc) return false;
    *head_step = hs > 0 ? 1 : 0;
    *page_step = ps > 0 ? 1 : 0;
    const int64_t pages = c.num_pages < 1 ? 1 : c.num_pages > 0x7fffffffLL ? 0x7fffffffLL : c.num_pages;  // (a page's number is an int32)
    cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(c.page_size), static_cast<cuuint64_t>(hs > 0 ? heads : 1),
                          static_cast<cuuint64_t>(ps > 0 ? pages : 1)};
    cuuint64_t strides[3] = {static_cast<cuuint64_t>(rs > 0 ? rs : d) * 2, static_cast<cuuint64_t>(hs > 0 ? hs : d) * 2,
                             static_cast<cuuint64_t>(ps > 0 ? ps : d) * 2};
    cuuint32_t box[4] = {64, static_cast<cuuint32_t>(box_rows), 1, 1};
    cuuint32_t es[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Queries [T, Hq, d]: boxes of the G heads of a tile's tokens.
bool encode_queries(CUtensorMap *map, const PrefixParams &p, int d) {
    auto enc = encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(p.Hq), static_cast<cuuint64_t>(p.T)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(p.qs) * 2};
    cuuint32_t box[3] = {64, static_cast<cuuint32_t>(p.G), static_cast<cuuint32_t>(kRow / p.G)};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p.q), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DK, int DV>
cudaError_t launch(const PrefixParams &p, cudaStream_t s) {
    TcParams a{};
    a.p = p;
    a.page_rows = (p.c.page_size + 7) / 8 * 8;
    a.box_rows = p.c.page_size < kRow ? p.c.page_size : kRow;
    CUtensorMap q_map{}, k_map, v_map;
    a.q_boxed = kRow % p.G == 0 && encode_queries(&q_map, p, DK);  // otherwise a tile begins or ends within a token
    // (a pool without pages has no address; nothing is copied then)
    const void *k = p.c.k ? static_cast<const void *>(p.c.k) : p.q, *v = p.c.v ? static_cast<const void *>(p.c.v) : p.q;
    if (!encode_pool(&k_map, k, p.c, p.Hkv, DK, p.c.kr, p.c.kh, p.c.kp, a.box_rows, &a.head_step_k, &a.page_step_k) ||
        !encode_pool(&v_map, v, p.c, p.Hkv, DV, p.c.vr, p.c.vh, p.c.vp, a.box_rows, &a.head_step_v, &a.page_step_v))
        return cudaErrorInvalidValue;
    constexpr int bytes = Smem<DK, DV>::kBytes;
    static_assert(bytes <= 232448, "more shared memory than a CTA has");
    if (!smem_opt_in<prefix_tc_kernel<DK, DV>>(bytes)) return cudaErrorInvalidValue;
    return launch_after(prefix_tc_kernel<DK, DV>, dim3(static_cast<unsigned>(p.ctas)), kThreads, bytes, s, a, q_map, k_map, v_map);
}

}  // namespace

void tc_cut(PrefixParams *p) {
    const int rows = (p->c.page_size + 7) / 8 * 8;
    p->tile_keys = kRow;
    p->pages_per_tile = p->c.page_size < kRow ? kRow / rows : 0;
    p->tiles_per_page = p->c.page_size < kRow ? 0 : (p->c.page_size + kRow - 1) / kRow;
}

cudaError_t launch_prefix_tc(const PrefixParams &p, int dk, int dv, cudaStream_t s) {
    if (dk == 128) return dv == 128 ? launch<128, 128>(p, s) : launch<128, 64>(p, s);
    return dv == 128 ? launch<64, 128>(p, s) : launch<64, 64>(p, s);
}

}  // namespace prefix
}  // namespace kda
