// Attention of drafted trees over a paged cache.
//
// Node i of a sequence attends to the sequence's context rows in the cache, to its ancestors among the
// drafted nodes and to itself: o = sum_j softmax_j(scale q.k_j) v_j.  The G = Hq / Hkv query heads of a KV head and
// the sequence's nodes form the R = m G rows of one matrix product per KV head, so that a
// key or value is read once for all of them.
//
// One pass over the keys with a running maximum and sum per row (base-2 exponentials of
// scale log2(e) q.k).  A sequence's context is cut into parts of `chunk` keys (split_of below); a unit
// of work is (sequence, KV head, row tile, part), the last part taking the drafted nodes' own keys as one more
// tile with the ancestor masks.  The units are numbered sequence by sequence; a persistent grid takes a
// contiguous run of them per CTA and streams their key tiles through one ring of stages filled by 16-byte asynchronous
// copies, across unit borders.  Parts leave their unnormalised sums, maximum and weight sum in the workspace and
// combine_kernel joins them in part order.  Everything a unit does depends on its own sequence alone,
// so a sequence's bits do not depend on the batch.
//
// Bounded by the bytes of the cache: 128 sequences of 1 to 4 nodes over 1 to 4,096 keys (8 KV heads, bf16) take 209 us, 5.2 TB/s; 16 rows
// over 131,072 keys 187 us, 5.7 TB/s.  The four warps of a CTA take a quarter of a tile's 64 keys each (half, on two row
// groups) and are joined through shared memory at the end of a part; three CTAs of two stages per SM cover one another's part ends
// (two CTAs of three stages: 224 us).  From 33 rows on (bf16) the tcgen05 kernel takes over: mma.sync falls behind the
// loads there (40 rows over 131,072 keys: 358 us, there 232).  fp32: 41 us for seven sequences of 1 to 13 nodes over 1 to 4,099 keys,
// neither at the bytes (4.4 us) nor at the tensor rate (the pipe is busy 9.5% of the time): a part has a few tiles, two warps
// share a scheduler, and what they wait for is their own chain of copies, splits, products and the join.
//
// bf16 weights meet the values as bf16 (half a step, 2^-9 of a weight): a tensor-core product takes both operands in one type, and a
// second product with the remainders would double the work on the values.  Sums and maxima are fp32, of the weights before
// that rounding.
//
// plan_kernel, one launch before: checks the lengths, lists the sequences with their first unit and their place among the partial
// results, turns the parents into ancestor masks (one 64-bit word per node, by pointer doubling), and copies the drafted values
// without infinities and NaN, which combine_kernel adds to the rows that see them (2.5 of the 209 us).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "kda_tree_attn.cuh"

namespace kda {
namespace {

using namespace attn;

constexpr int kAttnThreads = 128;

// `before`: the largest of cu[0 .. n - 1].  A sequence that begins below it shares nodes with an earlier one: the masks and the
// room for partial results hold each packed node once.
__device__ __forceinline__ uint32_t seq_check(const AttnParams &p, int n, int before, int *t0, int *m, int *ctx) {
    const int64_t a = p.cu[n], b = p.cu[n + 1], c = p.c.ctx_len[n];
    *t0 = static_cast<int>(a);
    *m = static_cast<int>(b - a);
    *ctx = static_cast<int>(c);
    if (a < 0 || a > b || b > p.T || b - a > p.max_nodes || (n == 0 && a != 0) || a < before) return DEV_ERR_SEQLENS;
    if (c < 0 || c > static_cast<int64_t>(p.c.max_pages) * p.c.page_size) return DEV_ERR_PAGE;
    return 0;
}

constexpr int kPlanThreads = 256;

// CTA 0: the list of sequences and units, and the status word.  The next seq_ctas, a warp per sequence: masks.  The others, a warp
// per packed node: the finite copy of its values.
template <typename T>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const AttnParams p, int seq_ctas, int dv) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_go();
    if (blockIdx.x == 0) {
        // both lists at once: units of the register kernels, row tiles of the tcgen05 kernel; and the rows of partial results
        __shared__ int warp_tot[3][kPlanThreads / 32];
        __shared__ int warp_top[kPlanThreads / 32];
        __shared__ int base_units[3], base_top;
        __shared__ uint32_t errors;
        if (threadIdx.x == 0) {
            base_units[0] = base_units[1] = base_units[2] = 0;
            base_top = INT32_MIN;
            errors = 0;
        }
        __syncthreads();
        for (int base = 0; base < p.N; base += kPlanThreads) {
            const int n = base + threadIdx.x;
            // the running maximum of cu ahead of this sequence
            int top = n < p.N ? p.cu[n] : INT32_MIN;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, top, o);
                if (lane >= o) top = max(top, y);
            }
            if (lane == 31) warp_top[warp] = top;
            int before = __shfl_up_sync(0xffffffffu, top, 1);
            __syncthreads();
            before = lane == 0 ? base_top : max(before, base_top);
            for (int w = 0; w < warp; ++w) before = max(before, warp_top[w]);
            SeqInfo s{};
            int units[3] = {0, 0, 0};
            if (n < p.N) {
                const uint32_t err = seq_check(p, n, before, &s.t0, &s.nodes, &s.ctx);
                if (err) atomicOr(&errors, err);
                const int rows = s.nodes * p.G;
                if (!err && rows > 0) {
                    if (p.tc && rows > kTcLeast) {
                        s.tiles = tc_tiles_of(rows);
                        tc_split_of(s.ctx, p.Hkv, s.tiles, &s.nsplit, &s.chunk);
                        units[1] = s.nsplit * s.tiles * p.Hkv;
                    } else {
                        s.tiles = tiles_of(rows);
                        split_of(s.ctx, rows, p.Hkv, s.tiles, p.wide, &s.nsplit, &s.chunk);
                        units[0] = s.nsplit * s.tiles * (p.Hkv / heads_of(rows, p.Hkv, p.wide));
                    }
                    units[2] = static_cast<int>(part_rows(p.tc, s.nodes, p.Hq, p.Hkv, s.nsplit));
                }
            }
            int upto[3] = {units[0], units[1], units[2]};
#pragma unroll
            for (int o = 1; o < 32; o <<= 1)
#pragma unroll
                for (int x = 0; x < 3; ++x) {
                    const int y = __shfl_up_sync(0xffffffffu, upto[x], o);
                    if (lane >= o) upto[x] += y;
                }
            if (lane == 31) {
#pragma unroll
                for (int x = 0; x < 3; ++x) warp_tot[x][warp] = upto[x];
            }
            __syncthreads();
            int off[3] = {base_units[0], base_units[1], base_units[2]};
            for (int w = 0; w < warp; ++w)
#pragma unroll
                for (int x = 0; x < 3; ++x) off[x] += warp_tot[x][w];
            if (n < p.N) {
                s.part0 = off[2] + upto[2] - units[2];
                s.unit0 = off[0] + upto[0] - units[0];
                p.info[n] = s;
                if (p.tc) {
                    s.unit0 = off[1] + upto[1] - units[1];
                    p.info_tc[n] = s;
                }
            }
            __syncthreads();
            if (threadIdx.x == kPlanThreads - 1) {
#pragma unroll
                for (int x = 0; x < 3; ++x) base_units[x] = off[x] + upto[x];
                base_top = max(before, top);
            }
            __syncthreads();
        }
        if (threadIdx.x == 0) {
            SeqInfo s{};
            s.unit0 = base_units[0];
            p.info[p.N] = s;
            if (p.tc) {
                s.unit0 = base_units[1];
                p.info_tc[p.N] = s;
            }
            *p.status = errors;
        }
        return;
    }
    if (blockIdx.x > seq_ctas) {
        const int64_t t = static_cast<int64_t>(blockIdx.x - 1 - seq_ctas) * (kPlanThreads / 32) + warp;
        if (t >= p.T) return;
        if (t >= p.cu[p.N]) {  // not to be read, unless cu falls and an earlier sequence has the node
            int top = 0;
            for (int i = lane; i < p.N; i += 32) top = max(top, p.cu[i]);
            if (t >= __reduce_max_sync(0xffffffffu, top)) return;
        }
        const int units = p.Hkv * dv / Elem<T>::kVec;
        const uint4 *from = reinterpret_cast<const uint4 *>(static_cast<const T *>(p.given_v) + t * p.given_vs);
        uint4 *to = reinterpret_cast<uint4 *>(const_cast<void *>(p.v)) + t * units;
        bool odd = false;
#pragma unroll 4
        for (int u = lane; u < units; u += 32) to[u] = finite_only<T>(from[u], odd);
        odd = __any_sync(0xffffffffu, odd);
        if (lane == 0) p.odd[t] = odd;
        return;
    }
    const int n0 = (blockIdx.x - 1) * (kPlanThreads / 32), n = n0 + warp;
    int before = lane < warp && n0 + lane < p.N ? p.cu[n0 + lane] : INT32_MIN;
    if (n0 > 0) {  // (the same for the whole CTA)
        __shared__ int warp_top[kPlanThreads / 32];
        int top = INT32_MIN;
        for (int i = threadIdx.x; i < n0; i += kPlanThreads) top = max(top, p.cu[i]);
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0) warp_top[warp] = top;
        __syncthreads();
        if (lane < kPlanThreads / 32) before = max(before, warp_top[lane]);
    }
    before = __reduce_max_sync(0xffffffffu, before);
    if (n >= p.N) return;
    int t0, m, ctx;
    const bool ok = seq_check(p, n, before, &t0, &m, &ctx) == 0;
    if (!ok) m = 0;
    uint64_t mask[2];
    int up[2];
    bool wrong = false;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const int i = lane + 32 * w;
        up[w] = i < m && i > 0 ? (p.parent ? p.parent[t0 + i] : i - 1) : -1;
        if (i > 0 && i < m && (up[w] < 0 || up[w] >= i)) {
            wrong = true;
            up[w] = -1;
        }
        mask[w] = i < 64 ? 1ull << i : 0ull;
    }
    // after round r a mask holds 2^r generations and `up` the next one
#pragma unroll
    for (int r = 0; r < 6; ++r) {
        uint64_t grown[2];
        int next[2];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const int a = up[w] < 0 ? 0 : up[w];
            const uint64_t m0 = __shfl_sync(0xffffffffu, mask[0], a & 31), m1 = __shfl_sync(0xffffffffu, mask[1], a & 31);
            const int u0 = __shfl_sync(0xffffffffu, up[0], a & 31), u1 = __shfl_sync(0xffffffffu, up[1], a & 31);
            grown[w] = up[w] < 0 ? mask[w] : mask[w] | (a < 32 ? m0 : m1);
            next[w] = up[w] < 0 ? -1 : (a < 32 ? u0 : u1);
        }
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            mask[w] = grown[w];
            up[w] = next[w];
        }
    }
    wrong = __any_sync(0xffffffffu, wrong);
    if (lane == 0) p.bad[n] = wrong ? DEV_ERR_TREE : 0u;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const int i = lane + 32 * w;
        if (i < m) {
            p.sees[t0 + i] = mask[w];
            p.seq_of[t0 + i] = n;
        }
    }
}

// ---------------------------------------------------------------------------------------------------------------
// The walk over a CTA's units and key tiles (one instance fills the ring, one consumes it)
// ---------------------------------------------------------------------------------------------------------------
struct Walk {
    int unit, end;                      // units left: [unit, end)
    int n, head, tile, split;           // of the unit
    int ctx, nodes, t0, nsplit, chunk, tiles, next0;  // of the sequence; next0: the first unit after it
    int heads;                          // KV heads of a unit (1 or 4); `head` counts groups of them
    int key, key_end;                   // context keys left in the unit
    int node, node_end;                 // drafted keys left in the unit

    __device__ __forceinline__ void begin_unit() {
        key = split * chunk;
        key_end = ctx - key < chunk ? ctx : key + chunk;  // (a context may end right below 2^31: nothing is added to a key past it)
        node = 0;
        node_end = split == nsplit - 1 ? nodes : 0;
    }
    __device__ __forceinline__ bool unit_done() const { return key >= key_end && node >= node_end; }
    __device__ __forceinline__ void enter_seq(const AttnParams &p) {
        // sequences without units (empty or bad) have the unit0 of the next one
        int next = __ldg(&p.info[n + 1].unit0);
        while (unit >= next && n + 1 < p.N) {
            ++n;
            next = __ldg(&p.info[n + 1].unit0);
        }
        const int4 a = __ldg(reinterpret_cast<const int4 *>(p.info + n));
        const int4 b = __ldg(reinterpret_cast<const int4 *>(p.info + n) + 1);
        ctx = a.x; nodes = a.y; t0 = a.z; nsplit = b.x; chunk = b.y; tiles = b.z;
        next0 = next;
        heads = heads_of(nodes * p.G, p.Hkv, p.wide);
        const int u = unit - a.w, ht = u / nsplit;
        split = u - ht * nsplit;
        head = ht / tiles;
        tile = ht - head * tiles;
        begin_unit();
    }
    // Every lane of a converged warp.
    __device__ __forceinline__ void start(const AttnParams &p, int first, int last) {
        unit = first;
        end = last;
        if (unit >= end) return;
        n = warp_find([&](int i) { return __ldg(&p.info[i].unit0); }, p.N, unit);
        enter_seq(p);
    }
    __device__ __forceinline__ void next_unit(const AttnParams &p) {
        if (++unit >= end) return;
        if (unit >= next0) {
            ++n;
            enter_seq(p);
            return;
        }
        if (++split == nsplit) {
            split = 0;
            if (++tile == tiles) {
                tile = 0;
                ++head;
            }
        }
        begin_unit();
    }
};

// A key row of a tile: byte offsets of its K and V rows from the tile's bases (multiples of 16), each with bit 0 set where there is
// no such row (zeros; the copy of no bytes still names an aligned address, the base's).
struct __align__(16) TileRow {
    int64_t k, v;
};
constexpr TileRow kNoRow{1, 1};
__device__ __forceinline__ bool row_there(int64_t off) { return (off & 1) == 0; }
__device__ __forceinline__ int64_t row_offset(int64_t off) { return off & ~static_cast<int64_t>(1); }

// The ring of key / value tiles.  A tile is kKeys rows of K, then kKeys rows of V; the 16-byte
// units of a row are permuted by its low three row bits, so that both a column of eight rows and a row are read
// without bank conflicts.
template <typename T, int DK, int DV>
struct Ring {
    static constexpr int kKeys = sizeof(T) == 2 ? 64 : 32;
    static constexpr int kThreads = 128;
    static constexpr int kStages = sizeof(T) == 2 ? 2 : 3;
    static constexpr int kPerSm = sizeof(T) == 2 ? 3 : 2;  // CTAs (bf16 with three stages and two CTAs: 224 us for 204, before drafted values were copied)
    static constexpr int kUnitsK = DK * static_cast<int>(sizeof(T)) / 16, kUnitsV = DV * static_cast<int>(sizeof(T)) / 16;
    static constexpr int kBytesK = kKeys * kUnitsK * 16, kBytesV = kKeys * kUnitsV * 16;
    static constexpr int kStage = kBytesK + kBytesV;

    char *smem;                  // kStages * kStage bytes
    TileRow (*rows)[kKeys];      // [2]: rows of the next tile to be issued, by tile parity
    int *bad_seen;               // a page of this CTA's units was out of range
    Walk w;                      // the tile after the one whose rows were looked up last
    int tile;                    // tiles consumed so far
    const char *kbase, *vbase;   // bases of the looked-up tile's rows (null: no tile)

    // Rows of the walk's tile; moves the walk past it.  Every thread takes part, threads < kKeys have a row.
    __device__ __forceinline__ TileRow look(const AttnParams &p) {
        constexpr int64_t es = sizeof(T);
        TileRow r = kNoRow;
        kbase = nullptr;
        if (w.unit >= w.end) return r;
        // a unit of four heads has a quarter of the tile for each
        const int per = w.heads == 4 ? kKeys / 4 : kKeys, j = threadIdx.x % per, h = threadIdx.x / per;
        const bool mine = threadIdx.x < kKeys;
        if (w.key < w.key_end) {
            kbase = p.c.k + w.head * w.heads * p.c.kh * es;
            vbase = p.c.v + w.head * w.heads * p.c.vh * es;
            if (mine && j < w.key_end - w.key) {
                const int at = w.key + j, pg = at / p.c.page_size, slot = at - pg * p.c.page_size;
                const int page = __ldg(p.c.table + static_cast<int64_t>(w.n) * p.c.table_stride + pg);
                if (page >= 0 && page < p.c.num_pages) {
                    r = TileRow{(page * p.c.kp + slot * p.c.kr + h * p.c.kh) * es, (page * p.c.vp + slot * p.c.vr + h * p.c.vh) * es};
                } else {
                    atomicOr(p.bad + w.n, static_cast<uint32_t>(DEV_ERR_PAGE));
                    atomicOr(p.status, static_cast<uint32_t>(DEV_ERR_PAGE));
                    *bad_seen = 1;
                }
            }
            w.key = w.key_end - w.key < per ? w.key_end : w.key + per;
        } else {
            kbase = static_cast<const char *>(p.k) + static_cast<int64_t>(w.head) * w.heads * DK * es;
            vbase = static_cast<const char *>(p.v) + static_cast<int64_t>(w.head) * w.heads * DV * es;
            if (mine && w.node + j < w.node_end) {
                const int64_t t = w.t0 + w.node + j;
                r = TileRow{(t * p.ks + h * DK) * es, (t * p.vs + h * DV) * es};
            }
            w.node += per;
        }
        if (w.unit_done()) w.next_unit(p);
        return r;
    }
    __device__ __forceinline__ void put(TileRow r, int parity) {
        if (threadIdx.x < kKeys) rows[parity][threadIdx.x] = r;
    }
    // Byte of unit u of row r0 + step (rows a multiple of 8 apart share their permutation).
    template <int kUnits>
    static __device__ __forceinline__ uint32_t place(int r0, int step, int u) {
        const int r = (kThreads / kUnits) % 8 == 0 ? r0 : r0 + step;
        return (r0 + step) * (kUnits * 16) + ((u ^ (r & 7)) << 4);
    }
    // Starts the copies of the looked-up tile of the given number: a thread takes one 16-byte unit of every
    // kThreads / units-th row.
    __device__ __forceinline__ void issue(const AttnParams &p, int number) {
        if (kbase) {
            const TileRow *tr = rows[number & 1];
            const uint32_t dst = ptx::smem_u32(smem) + static_cast<uint32_t>(number % kStages) * kStage;
            if constexpr (kUnitsK == kUnitsV) {
                constexpr int kSide = kThreads / kUnitsK;
                const int u = threadIdx.x % kUnitsK, r0 = threadIdx.x / kUnitsK;
                const char *ks = kbase + u * 16, *vs = vbase + u * 16;
#pragma unroll
                for (int i = 0; i < kKeys / kSide; ++i) {
                    const TileRow x = tr[r0 + i * kSide];
                    const bool there = row_there(x.k);
                    const uint32_t to = dst + place<kUnitsK>(r0, i * kSide, u);
                    cp16(to, ks + row_offset(x.k), there);
                    cp16(to + kBytesK, vs + row_offset(x.v), there);
                }
            } else {
                copy<kUnitsK>(dst, &tr->k, kbase);
                copy<kUnitsV>(dst + kBytesK, &tr->v, vbase);
            }
        }
        cp_commit();
    }
    template <int kUnits>
    __device__ __forceinline__ void copy(uint32_t dst, const int64_t *off, const char *base) {
        constexpr int kSide = kThreads / kUnits;
        const int u = threadIdx.x % kUnits, r0 = threadIdx.x / kUnits;
#pragma unroll
        for (int i = 0; i < kKeys / kSide; ++i) {
            const int64_t x = off[2 * (r0 + i * kSide)];
            cp16(dst + place<kUnits>(r0, i * kSide, u), base + u * 16 + row_offset(x), row_there(x));
        }
    }
    __device__ __forceinline__ void start(const AttnParams &p, const Walk &from) {
        tile = 0;
        w = from;
#pragma unroll
        for (int i = 0; i < kStages; ++i) {
            put(look(p), i & 1);
            __syncthreads();
            if (i < kStages - 1) issue(p, i);
        }
    }
    // Waits for the next tile, refills the stage freed before it, and looks one tile further; returns the
    // looked-up row, to be stored by end_tile after the tile's work (its latency is covered by it).
    __device__ __forceinline__ TileRow begin_tile(const AttnParams &p) {
        cp_wait<kStages - 2>();
        __syncthreads();
        issue(p, tile + kStages - 1);
        return look(p);
    }
    __device__ __forceinline__ void end_tile(TileRow r) {
        put(r, (tile + kStages) & 1);
        ++tile;
    }
    __device__ __forceinline__ const char *stage() const { return smem + (tile % kStages) * kStage; }
    // The stage of the last consumed tile: free from a barrier after end_tile up to the next begin_tile.
    __device__ __forceinline__ char *scratch() const { return smem + ((tile + kStages - 1) % kStages) * kStage; }
};

// Whether a unit of the walk's sequence may write: `flag` is what the plan left (a bad parent); a bad
// page can only have been met by this CTA itself if it matters here (a unit that writes o has seen all pages).
__device__ __forceinline__ bool may_write(const AttnParams &p, int n, uint32_t flag, int *bad_seen) {
    if (*reinterpret_cast<volatile int *>(bad_seen)) flag |= __ldcg(p.bad + n);
    return flag == 0;
}

// ---------------------------------------------------------------------------------------------------------------
// bf16: 16-row fragments of mma.sync, RW of the four warps on different rows and the rest on different keys
// ---------------------------------------------------------------------------------------------------------------
__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The warps along the keys joined in order: maxima and sums in all of them, and of the fragments of o (row quad in
// elements 0 and 1, quad + 8 in 2 and 3) each warp has the part kg of KW.
template <int WARPS, int RW, int DV>
__device__ __forceinline__ void join_warps(char *scratch, float2 (*ml)[16], float (&o)[DV / 8][4], float (&mx)[2], float (&sum)[2]) {
    constexpr int KW = WARPS / RW, NP = DV / 8 / KW;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rg = warp % RW, kg = warp / RW, quad = lane >> 2;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
        sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
    }
    if constexpr (KW > 1) {
        // [part][other warp][rg][fragment element][lane]
        float *buf = reinterpret_cast<float *>(scratch) + lane;
        auto place = [&](int part, int from) { return ((part * (KW - 1) + (from < part ? from : from - 1)) * RW + rg) * (NP * 4 * 32); };
        __syncthreads();  // the last tile's readers are done with the stage
        if ((lane & 3) == 0) {
            ml[warp][quad] = make_float2(mx[0], sum[0]);
            ml[warp][quad + 8] = make_float2(mx[1], sum[1]);
        }
#pragma unroll
        for (int part = 0; part < KW; ++part)
            if (part != kg) {
                float *to = buf + place(part, kg);
#pragma unroll
                for (int j = 0; j < NP; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) to[(j * 4 + e) * 32] = o[part * NP + j][e];
            }
        __syncthreads();
        float f[KW][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float2 x[KW];
            float m = -INFINITY;
#pragma unroll
            for (int g = 0; g < KW; ++g) {
                x[g] = ml[g * RW + rg][quad + 8 * i];
                m = fmaxf(m, x[g].x);
            }
            const float base = m == -INFINITY ? 0.f : m;
            float l = 0.f;
#pragma unroll
            for (int g = 0; g < KW; ++g) {
                f[g][i] = ex2(x[g].x - base);
                l += f[g][i] * x[g].y;
            }
            mx[i] = m;
            sum[i] = l;
        }
#pragma unroll
        for (int part = 0; part < KW; ++part)
            if (part == kg) {
#pragma unroll
                for (int j = 0; j < NP; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float x = 0.f;
#pragma unroll
                        for (int g = 0; g < KW; ++g)
                            x += f[g][e >> 1] * (g == part ? o[part * NP + j][e] : buf[place(part, g) + (j * 4 + e) * 32]);
                        o[part * NP + j][e] = x;
                    }
            }
    }
}

template <int DK, int DV, int RW>
__device__ __forceinline__ void unit_bf16(const AttnParams &p, Ring<__nv_bfloat16, DK, DV> &ring, Walk &cw, float2 (*ml)[16],
                                          uint32_t (&qf)[DK / 16][4], bool same_rows) {
    using R = Ring<__nv_bfloat16, DK, DV>;
    constexpr int KW = 4 / RW, NT = 8 / KW;  // warps along the keys; 8-key columns of a warp
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rg = warp % RW, kg = warp / RW, key0 = kg * (64 / KW);
    const int quad = lane >> 2, two = (lane & 3) * 2;
    const int n = cw.n, t0 = cw.t0, split = cw.split, nsplit = cw.nsplit, rows = cw.nodes * p.G;
    const uint32_t flag = __ldcg(p.bad + n);
    const float c = p.scale * kLog2e;

    // this thread's two rows: node and query head
    int node[2], hq[2];
    bool live[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = cw.tile * kTileRows + rg * 16 + quad + 8 * i;
        live[i] = r < rows;
        node[i] = live[i] ? r / p.G : 0;
        hq[i] = cw.head * p.G + (live[i] ? r - node[i] * p.G : 0);
    }
    if (!same_rows)  // (the part before this one had the same)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(p.q) + (t0 + node[i]) * p.qs + static_cast<int64_t>(hq[i]) * DK + two;
#pragma unroll
        for (int k = 0; k < DK / 16; ++k) {
            qf[k][i] = live[i] ? *reinterpret_cast<const uint32_t *>(src + k * 16) : 0u;
            qf[k][2 + i] = live[i] ? *reinterpret_cast<const uint32_t *>(src + k * 16 + 8) : 0u;
        }
    }
    float o[DV / 8][4];
#pragma unroll
    for (int j = 0; j < DV / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    float mx[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};

    while (!cw.unit_done()) {
        const bool drafted = cw.key >= cw.key_end;
        const int first = drafted ? cw.node : 0;
        const int count = drafted ? cw.node_end - cw.node : cw.key_end - cw.key;  // keys from here on
        if (drafted) cw.node += R::kKeys; else cw.key = count < R::kKeys ? cw.key_end : cw.key + R::kKeys;
        const TileRow ahead = ring.begin_tile(p);
        const uint32_t ks = ptx::smem_u32(ring.stage()), vs = ks + R::kBytesK;
        // scores of 16 rows x NT * 8 keys
        float s[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
        for (int k = 0; k < DK / 16; ++k)
#pragma unroll
            for (int j = 0; j < NT; j += 2) {
                const int row = key0 + (j + (lane >> 4)) * 8 + (lane & 7), u = 2 * k + ((lane >> 3) & 1);
                uint32_t b[4];
                ldm4(b, ks + row * (R::kUnitsK * 16) + ((u ^ (row & 7)) << 4));
                mma16816(s[j], qf[k], b[0], b[1]);
                mma16816(s[j + 1], qf[k], b[2], b[3]);
            }
        uint64_t sees[2] = {~0ull, ~0ull};
        if (drafted) {
#pragma unroll
            for (int i = 0; i < 2; ++i) sees[i] = __ldg(p.sees + t0 + node[i]) >> first;
        }
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int key = key0 + j * 8 + two + (e & 1);
                float t = s[j][e] * c;
                if (key >= count || !((sees[e >> 1] >> key) & 1)) t = -INFINITY;
                s[j][e] = t;
                top[e >> 1] = fmaxf(top[e >> 1], t);
            }
        float old[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
            top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
            const float now = fmaxf(mx[i], top[i]);
            const float base = now == -INFINITY ? 0.f : now;
            old[i] = ex2(mx[i] - base);
            mx[i] = now;
            top[i] = base;
            sum[i] *= old[i];
        }
        uint32_t pf[NT][2];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            float e[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                e[x] = ex2(s[j][x] - top[x >> 1]);
                sum[x >> 1] += e[x];
            }
            pf[j][0] = ptx::pack_bf16x2(e[0], e[1]);
            pf[j][1] = ptx::pack_bf16x2(e[2], e[3]);
        }
        if (__any_sync(0xffffffffu, old[0] != 1.f || old[1] != 1.f)) {
#pragma unroll
            for (int j = 0; j < DV / 8; ++j) {
                o[j][0] *= old[0];
                o[j][1] *= old[0];
                o[j][2] *= old[1];
                o[j][3] *= old[1];
            }
        }
#pragma unroll
        for (int k = 0; k < NT / 2; ++k) {
            const uint32_t a[4] = {pf[2 * k][0], pf[2 * k][1], pf[2 * k + 1][0], pf[2 * k + 1][1]};
#pragma unroll
            for (int j = 0; j < DV / 8; j += 2) {
                const int row = key0 + k * 16 + (lane & 15), u = j + (lane >> 4);
                uint32_t b[4];
                ldm4t(b, vs + row * (R::kUnitsV * 16) + ((u ^ (row & 7)) << 4));
                mma16816(o[j], a, b[0], b[1]);
                mma16816(o[j + 1], a, b[2], b[3]);
            }
        }
        ring.end_tile(ahead);
    }
    join_warps<4, RW, DV>(ring.scratch(), ml, o, mx, sum);
    const bool ok = may_write(p, n, flag, ring.bad_seen);
    if (flag && threadIdx.x == 0) atomicOr(p.status, flag);
    constexpr int NP = DV / 8 / KW;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (!live[i] || !ok) continue;
        const int64_t row = static_cast<int64_t>(t0 + node[i]) * p.Hq + hq[i];
        const bool whole = nsplit == 1, first_lane = kg == 0 && (lane & 3) == 0;
        if (whole) {
            const float inv = 1.f / sum[i];
            uint32_t *to = reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(p.o) + row * DV + two);
#pragma unroll
            for (int part = 0; part < KW; ++part)
                if (part == kg) {
#pragma unroll
                    for (int j = part * NP; j < (part + 1) * NP; ++j) to[j * 4] = ptx::pack_bf16x2(o[j][2 * i] * inv, o[j][2 * i + 1] * inv);
                }
            if (p.lse && first_lane) p.lse[row] = (mx[i] + log2f(sum[i])) * kLn2;
        } else {
            const int64_t at = __ldg(&p.info[n].part0) + (row - static_cast<int64_t>(t0) * p.Hq) * nsplit + split;
            float2 *to = reinterpret_cast<float2 *>(p.part_o + at * DV + two);
#pragma unroll
            for (int part = 0; part < KW; ++part)
                if (part == kg) {
#pragma unroll
                    for (int j = part * NP; j < (part + 1) * NP; ++j) to[j * 4] = make_float2(o[j][2 * i], o[j][2 * i + 1]);
                }
            if (first_lane) p.part_ml[at] = make_float2(mx[i], sum[i]);
        }
    }
}

// ---------------------------------------------------------------------------------------------------------------
// fp32: the same walk with m16n8k8 products in three tf32 terms
// ---------------------------------------------------------------------------------------------------------------
// x = hi + lo + at most 2^-23 |x|, both with the 11 significant bits of tf32; a product is hi hi + hi lo + lo hi, which
// leaves about the rounding of an fp32 sum of this length, at a third of the tensor rate (and at that rate
// this path is bound: fused multiply-adds took several times as long).  hi is rounded to nearest, so that lo has either
// sign and the lo lo left out does not add up (with a truncated hi the result was three times as far off); the largest
// finite values round down.  An infinity or NaN is all in hi, and 0 in `fin`, the hi of the two cross terms, so that they
// add nothing to what it makes of the first one.
struct Split {
    uint32_t hi, fin, lo;
};
constexpr uint32_t kTf32 = 0xffffe000u;
__device__ __forceinline__ Split split_any(float x) {
    const uint32_t bits = __float_as_uint(x), size = bits & 0x7fffffffu;
    const uint32_t near = (min(size + 0x1000u, 0x7f7fffffu) & kTf32) | (bits & 0x80000000u);
    const bool ok = size < 0x7f800000u;
    return {ok ? near : bits & kTf32, ok ? near : 0u, ok ? __float_as_uint(x - __uint_as_float(near)) & kTf32 : 0u};
}
// The same for values whose square is finite (as that of others is not, a sum of squares tells).
__device__ __forceinline__ Split split(float x) {
    const uint32_t hi = (__float_as_uint(x) + 0x1000u) & kTf32;
    return {hi, hi, __float_as_uint(x - __uint_as_float(hi)) & kTf32};
}
template <bool kAny>
__device__ __forceinline__ Split split_as(float x) {
    if constexpr (kAny) return split_any(x);
    else return split(x);
}
__device__ __forceinline__ void mma1688(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The order in which an instruction's k index runs over channels or keys is free as long as both operands agree: a lane takes
// eight consecutive channels of every 32 (two 16-byte reads without bank conflicts), and the weights' accumulator fragment
// is the next product's operand as it is.
template <int DK, int DV, int RW, bool kHeads>
__device__ __forceinline__ void unit_f32(const AttnParams &p, Ring<float, DK, DV> &ring, Walk &cw, float2 (*ml)[16],
                                         float (&qf)[DK / 32][2][8], bool same_rows) {
    using R = Ring<float, DK, DV>;
    constexpr int KT = R::kThreads / 32 / RW, NT = R::kKeys / 8 / KT;
    constexpr int KW = kHeads ? 1 : KT;
    constexpr int kStep = kHeads ? R::kKeys / 4 : R::kKeys;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rg = warp % RW, kg = kHeads ? 0 : warp / RW, row0 = warp / RW * (R::kKeys / KT), key0 = kHeads ? 0 : row0;
    const int head = kHeads ? cw.head * 4 + warp : cw.head;
    const int quad = lane >> 2, j4 = lane & 3;
    const int n = cw.n, t0 = cw.t0, split_no = cw.split, nsplit = cw.nsplit, rows = cw.nodes * p.G;
    const uint32_t flag = __ldcg(p.bad + n);
    const float c = p.scale * kLog2e;
    int node[2], hq[2];
    bool live[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = cw.tile * kTileRows + rg * 16 + quad + 8 * i;
        live[i] = r < rows;
        node[i] = live[i] ? r / p.G : 0;
        hq[i] = head * p.G + (live[i] ? r - node[i] * p.G : 0);
    }
    if (!same_rows)  // channels 32 g + 8 j4 + 0..7 of the two rows
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float *src = static_cast<const float *>(p.q) + (t0 + node[i]) * p.qs + static_cast<int64_t>(hq[i]) * DK + 8 * j4;
#pragma unroll
        for (int g = 0; g < DK / 32; ++g)
#pragma unroll
            for (int x = 0; x < 8; x += 4)
                *reinterpret_cast<float4 *>(&qf[g][i][x]) = live[i] ? *reinterpret_cast<const float4 *>(src + 32 * g + x) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float q_size = 0.f;  // sum of squares: finite unless a value is not, or far too large
#pragma unroll
    for (int g = 0; g < DK / 32; ++g)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int x = 0; x < 8; ++x) q_size = fmaf(qf[g][i][x], qf[g][i][x], q_size);
    q_size = q_size < INFINITY ? 0.f : INFINITY;
    float o[DV / 8][4];  // fragment 4 g + q: columns 32 g + 8 j4 + q and + 4 of the two rows
#pragma unroll
    for (int j = 0; j < DV / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    float mx[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};

    while (!cw.unit_done()) {
        const bool drafted = cw.key >= cw.key_end;
        const int first = drafted ? cw.node : 0;
        const int count = drafted ? cw.node_end - cw.node : cw.key_end - cw.key;
        if (drafted) cw.node += kStep; else cw.key = count < kStep ? cw.key_end : cw.key + kStep;
        const TileRow ahead = ring.begin_tile(p);
        const char *ks = ring.stage(), *vs = ks + R::kBytesK;
        float s[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
        for (int g = 0; g < DK / 32; ++g)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float kf[NT][4];
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const int row = row0 + j * 8 + quad, u = 8 * g + 2 * j4 + h;
                    *reinterpret_cast<float4 *>(kf[j]) = *reinterpret_cast<const float4 *>(ks + row * (R::kUnitsK * 16) + ((u ^ (row & 7)) << 4));
                }
                float size = q_size;
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int y = 0; y < 4; ++y) size = fmaf(kf[j][y], kf[j][y], size);
                // The tensor cores cut sums off instead of rounding them: sixteen channels are summed there, the small terms first,
                // and what comes out is added with rounding (one sum through was three times as far off).
                auto products = [&](auto any) {
                    constexpr bool kAny = decltype(any)::value;
                    // (split again for every tile: kept between them, the parts would not fit the registers)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int y = 0; y < 4; ++y) asm volatile("" : "+f"(qf[g][i][4 * h + y]));
                    Split a[2][4];
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int e = 0; e < 4; ++e) a[y][e] = split_as<kAny>(qf[g][e & 1][4 * h + 2 * y + (e >> 1)]);
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        float t[4] = {0.f, 0.f, 0.f, 0.f};
                        Split b[2][2];
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            b[y][0] = split_as<kAny>(kf[j][2 * y]);
                            b[y][1] = split_as<kAny>(kf[j][2 * y + 1]);
                            const uint32_t af[4] = {a[y][0].fin, a[y][1].fin, a[y][2].fin, a[y][3].fin};
                            const uint32_t al[4] = {a[y][0].lo, a[y][1].lo, a[y][2].lo, a[y][3].lo};
                            mma1688(t, af, b[y][0].lo, b[y][1].lo);
                            mma1688(t, al, b[y][0].fin, b[y][1].fin);
                        }
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const uint32_t ah[4] = {a[y][0].hi, a[y][1].hi, a[y][2].hi, a[y][3].hi};
                            mma1688(t, ah, b[y][0].hi, b[y][1].hi);
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[j][e] += t[e];
                    }
                };
                if (__any_sync(0xffffffffu, !(size < INFINITY))) products(std::true_type{});
                else products(std::false_type{});
            }
        uint64_t sees[2] = {~0ull, ~0ull};
        if (drafted) {
#pragma unroll
            for (int i = 0; i < 2; ++i) sees[i] = __ldg(p.sees + t0 + node[i]) >> first;
        }
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int key = key0 + j * 8 + 2 * j4 + (e & 1);
                float t = s[j][e] * c;
                if (key >= count || !((sees[e >> 1] >> key) & 1)) t = -INFINITY;
                s[j][e] = t;
                top[e >> 1] = fmaxf(top[e >> 1], t);
            }
        float old[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
            top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
            const float now = fmaxf(mx[i], top[i]);
            const float base = now == -INFINITY ? 0.f : now;
            old[i] = exp2f(mx[i] - base);
            mx[i] = now;
            top[i] = base;
            sum[i] *= old[i];
        }
        if (__any_sync(0xffffffffu, old[0] != 1.f || old[1] != 1.f)) {
#pragma unroll
            for (int j = 0; j < DV / 8; ++j) {
                o[j][0] *= old[0];
                o[j][1] *= old[0];
                o[j][2] *= old[1];
                o[j][3] *= old[1];
            }
        }
#pragma unroll
        for (int k = 0; k < NT; ++k) {
            // weights of keys 8 k + 2 j4 (k index j4) and + 1 (j4 + 4)
            float e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                e[i] = exp2f(s[k][i] - top[i >> 1]);
                sum[i >> 1] += e[i];
            }
            // (weights are at most 1, or NaN, which their sum passes on to the whole row)
            const Split a0 = split(e[0]), a1 = split(e[2]), a2 = split(e[1]), a3 = split(e[3]);
            const uint32_t ah[4] = {a0.hi, a1.hi, a2.hi, a3.hi}, al[4] = {a0.lo, a1.lo, a2.lo, a3.lo};
            const int row = row0 + 8 * k + 2 * j4;
#pragma unroll
            for (int g = 0; g < DV / 32; ++g) {
                float v0[4], v1[4];  // columns 32 g + 4 quad + 0..3 of the two keys
                const int u = 8 * g + quad;
                *reinterpret_cast<float4 *>(v0) = *reinterpret_cast<const float4 *>(vs + row * (R::kUnitsV * 16) + ((u ^ (row & 7)) << 4));
                *reinterpret_cast<float4 *>(v1) = *reinterpret_cast<const float4 *>(vs + (row + 1) * (R::kUnitsV * 16) + ((u ^ ((row + 1) & 7)) << 4));
                float size = 0.f;
#pragma unroll
                for (int q = 0; q < 4; ++q) size = fmaf(v0[q], v0[q], fmaf(v1[q], v1[q], size));
                auto products = [&](auto any) {
                    constexpr bool kAny = decltype(any)::value;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const Split b0 = split_as<kAny>(v0[q]), b1 = split_as<kAny>(v1[q]);
                        float t[4] = {0.f, 0.f, 0.f, 0.f};
                        mma1688(t, ah, b0.lo, b1.lo);
                        mma1688(t, al, b0.fin, b1.fin);
                        mma1688(t, ah, b0.hi, b1.hi);
#pragma unroll
                        for (int e2 = 0; e2 < 4; ++e2) o[4 * g + q][e2] += t[e2];
                    }
                };
                if (__any_sync(0xffffffffu, !(size < INFINITY))) products(std::true_type{});
                else products(std::false_type{});
            }
        }
        ring.end_tile(ahead);
    }
    join_warps<R::kThreads / 32, kHeads ? R::kThreads / 32 : RW, DV>(ring.scratch(), ml, o, mx, sum);
    const bool ok = may_write(p, n, flag, ring.bad_seen);
    if (flag && threadIdx.x == 0) atomicOr(p.status, flag);
    constexpr int NP = DV / 8 / KW;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (!live[i] || !ok) continue;
        const int64_t row = static_cast<int64_t>(t0 + node[i]) * p.Hq + hq[i];
        const bool whole = nsplit == 1;
        const int64_t at = whole ? 0 : __ldg(&p.info[n].part0) + (row - static_cast<int64_t>(t0) * p.Hq) * nsplit + split_no;
        const float f = whole ? 1.f / sum[i] : 1.f;
        float *to = (whole ? static_cast<float *>(p.o) + row * DV : p.part_o + at * DV) + 8 * j4;
#pragma unroll
        for (int part = 0; part < KW; ++part)
            if (part == kg) {
#pragma unroll
                for (int j = part * NP; j < (part + 1) * NP; j += NP > 1 ? 2 : 1)  // fragments 4 g + q, q + 1
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float *at_j = to + 32 * (j / 4) + 4 * h + j % 4;
                        if constexpr (NP > 1) *reinterpret_cast<float2 *>(at_j) = make_float2(o[j][2 * i + h] * f, o[j + 1][2 * i + h] * f);
                        else *at_j = o[j][2 * i + h] * f;
                    }
            }
        if (kg == 0 && j4 == 0) {
            if (!whole) p.part_ml[at] = make_float2(mx[i], sum[i]);
            else if (p.lse) p.lse[row] = (mx[i] + log2f(sum[i])) * kLn2;
        }
    }
}

template <typename T, int DK, int DV>
__global__ void __launch_bounds__(Ring<T, DK, DV>::kThreads, Ring<T, DK, DV>::kPerSm) attn_kernel(const AttnParams p) {
    using R = Ring<T, DK, DV>;
    extern __shared__ __align__(128) char smem[];
    __shared__ TileRow rows[2][R::kKeys];
    __shared__ float2 ml[R::kThreads / 32][16];
    __shared__ int bad_seen;
    grid_wait();
    grid_go();
    const int64_t units = __ldg(&p.info[p.N].unit0);
    const int first = static_cast<int>(units * blockIdx.x / gridDim.x);
    const int last = static_cast<int>(units * (blockIdx.x + 1) / gridDim.x);
    if (first >= last) return;
    if (threadIdx.x == 0) bad_seen = 0;
    __syncthreads();
    R ring;
    ring.smem = smem;
    ring.rows = rows;
    ring.bad_seen = &bad_seen;
    Walk cw;
    cw.start(p, first, last);
    ring.start(p, cw);
    std::conditional_t<sizeof(T) == 2, uint32_t[DK / 16][4], float[DK / 32][2][8]> qf;
    bool same = false;
    while (cw.unit < cw.end) {
        const int left = cw.nodes * p.G - cw.tile * kTileRows;
        if constexpr (sizeof(T) == 2) {
            if (left <= 16) unit_bf16<DK, DV, 1>(p, ring, cw, ml, qf, same);
            else unit_bf16<DK, DV, 2>(p, ring, cw, ml, qf, same);  // (more rows: the tcgen05 kernel)
        } else {
            if (cw.heads == 4) unit_f32<DK, DV, 1, true>(p, ring, cw, ml, qf, same);
            else if (left <= 16) unit_f32<DK, DV, 1, false>(p, ring, cw, ml, qf, same);
            else if (left <= 32) unit_f32<DK, DV, 2, false>(p, ring, cw, ml, qf, same);
            else unit_f32<DK, DV, 4, false>(p, ring, cw, ml, qf, same);
        }
        same = cw.split + 1 < cw.nsplit;
        cw.next_unit(p);
    }
}

// ---------------------------------------------------------------------------------------------------------------
// The last kernel: the parts of a row (node, query head) joined, and what its nodes' values that are not finite add to it.  Joined: four sums of every fourth part, added in order.  kWarps = 1: a warp has all
// four; 4: a warp each, where there are few rows (one warp per row took 28 us for 256 rows of 114 parts).  A lane has DV / 32 columns.
// ---------------------------------------------------------------------------------------------------------------
template <typename T, int DV, int kWarps>
__global__ void __launch_bounds__(kAttnThreads) combine_kernel(const AttnParams p) {
    constexpr int VL = DV / 32, kSums = 4 / kWarps;  // sums of a warp
    __shared__ float share[kWarps == 4 ? 4 : 1][VL + 1][32];
    grid_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = kWarps == 4 ? static_cast<int64_t>(blockIdx.x) : static_cast<int64_t>(blockIdx.x) * (kAttnThreads / 32) + warp;
    if (row >= p.T * p.Hq) return;
    const int64_t t = row / p.Hq;
    // (a packed node beyond the last sequence has no entry: whatever is read there does not contain it)
    const int n = p.seq_of[t];
    if (n < 0 || n >= p.N) return;
    const SeqInfo s = p.info[n];
    if (s.nsplit < 1 || t < s.t0 || t >= s.t0 + s.nodes || p.bad[n]) return;
    uint64_t odd = 0;  // nodes that the row sees and whose values are not all finite
    if (p.odd) {
        const uint64_t sees = p.sees[t];
        const bool low = ((sees >> lane) & 1) && p.odd[s.t0 + lane], high = ((sees >> (lane + 32)) & 1) && p.odd[s.t0 + lane + 32];
        odd = (static_cast<uint64_t>(__ballot_sync(0xffffffffu, high)) << 32) | __ballot_sync(0xffffffffu, low);
    }
    T *to = static_cast<T *>(p.o) + row * DV + lane * VL;
    auto add_odd = [&](float (&x)[VL]) {
        const int64_t column = (row - t * p.Hq) / p.G * DV + lane * VL;
        for (; odd; odd &= odd - 1) {
            const T *src = static_cast<const T *>(p.given_v) + (s.t0 + __ffsll(static_cast<long long>(odd)) - 1) * p.given_vs + column;
#pragma unroll
            for (int i = 0; i < VL; ++i) {
                const float v = Elem<T>::to_f(src[i]);
                if (!(fabsf(v) < INFINITY)) x[i] += v;
            }
        }
    };
    const int parts = s.nsplit;
    if (parts == 1 || (p.tc && s.nodes * p.G > kTcLeast)) {  // complete but for those
        if (odd && (kWarps == 1 || warp == 0)) {
            float x[VL];
#pragma unroll
            for (int i = 0; i < VL; ++i) x[i] = Elem<T>::to_f(to[i]);
            add_odd(x);
#pragma unroll
            for (int i = 0; i < VL; ++i) to[i] = Elem<T>::from_f(x[i]);
        }
        return;
    }
    const int64_t part0 = s.part0 + (row - static_cast<int64_t>(s.t0) * p.Hq) * parts;
    const float2 *ml = p.part_ml + part0;
    float m = -INFINITY;
    for (int i = lane; i < parts; i += 32) m = fmaxf(m, ml[i].x);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
    const float base = m == -INFINITY ? 0.f : m;
    float l[kSums] = {}, o[kSums][VL] = {};
    const float *src = p.part_o + part0 * DV + lane * VL;
    const int first = kWarps == 4 ? warp : 0;
#pragma unroll 4
    for (int i0 = first; i0 < parts; i0 += 4)
#pragma unroll
        for (int c = 0; c < kSums; ++c) {
            const int i = i0 + c;
            if (i < parts) {
                const float2 part = ml[i];
                const float f = exp2f(part.x - base);
                l[c] = fmaf(f, part.y, l[c]);
#pragma unroll
                for (int x = 0; x < VL; x += 2) {
                    const float2 v = *reinterpret_cast<const float2 *>(src + static_cast<int64_t>(i) * DV + x);
                    o[c][x] = fmaf(f, v.x, o[c][x]);
                    o[c][x + 1] = fmaf(f, v.y, o[c][x + 1]);
                }
            }
        }
    float sum, out[VL];
    if constexpr (kWarps == 4) {
        auto &all = share;
#pragma unroll
        for (int x = 0; x < VL; ++x) all[warp][x][lane] = o[0][x];
        all[warp][VL][lane] = l[0];
        __syncthreads();
        if (warp > 0) return;
#pragma unroll
        for (int x = 0; x < VL; ++x) out[x] = (all[0][x][lane] + all[1][x][lane]) + (all[2][x][lane] + all[3][x][lane]);
        sum = (all[0][VL][lane] + all[1][VL][lane]) + (all[2][VL][lane] + all[3][VL][lane]);
    } else {
#pragma unroll
        for (int x = 0; x < VL; ++x) out[x] = (o[0][x] + o[1][x]) + (o[2][x] + o[3][x]);
        sum = (l[0] + l[1]) + (l[2] + l[3]);
    }
    const float inv = 1.f / sum;
#pragma unroll
    for (int x = 0; x < VL; ++x) out[x] *= inv;
    if (odd) add_odd(out);
#pragma unroll
    for (int x = 0; x < VL; ++x) to[x] = Elem<T>::from_f(out[x]);
    if (p.lse && lane == 0) p.lse[row] = (m + log2f(sum)) * kLn2;
}

template <typename T, int DV>
cudaError_t launch_combine(const AttnParams &p, cudaStream_t s) {
    const int64_t rows = p.T * p.Hq;
    if (rows <= 4096) return launch_after(combine_kernel<T, DV, 4>, dim3(static_cast<unsigned>(rows)), kAttnThreads, 0, s, p);
    constexpr int kPer = kAttnThreads / 32;
    return launch_after(combine_kernel<T, DV, 1>, dim3(static_cast<unsigned>((rows + kPer - 1) / kPer)), kAttnThreads, 0, s, p);
}

// ---------------------------------------------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------------------------------------------
size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

struct AttnLayout {
    size_t info, info_tc, bad, seq_of, sees, odd, copy_v, part_ml, part_o, total;
    int max_nodes;               // of a tree that T nodes can hold
    bool tc, parts;              // some tree is for the tcgen05 kernel; some sequence can have more than one part
    int64_t units;               // at most so many in either list (tcgen05: row tiles times parts)
    int64_t part_rows;           // at most so many rows of partial results
};
// The most that any batch of N trees of T nodes in all can ask for, each over a context of up to max_ctx rows.
AttnLayout layout_of(kda_dtype dtype, int N, int64_t T, int Hq, int Hkv, int dv, int max_nodes, int64_t max_ctx) {
    AttnLayout l{};
    const bool wide = dtype == KDA_F32;
    const int G = Hq / Hkv;
    if (max_nodes > T) max_nodes = static_cast<int>(T < 1 ? 1 : T);
    l.max_nodes = max_nodes;
    l.tc = !wide && max_nodes * G > kTcLeast;
    // By a tree's size: its rows of partial results (a cut has no more parts over a shorter context).
    int64_t rows_of[KDA_MAX_TREE_NODES + 1] = {}, most_units = 0;
    int least = 1, best = 1;     // the largest tree of the register kernels; the one of most rows per node
    for (int m = 1; m <= max_nodes; ++m) {
        const int rows = m * G;
        int splits;
        int64_t units;
        if (!wide && rows > kTcLeast) {
            splits = tc_splits_of(max_ctx, Hkv, tc_groups_of(tc_tiles_of(rows)));
            units = static_cast<int64_t>(splits) * tc_tiles_of(rows) * Hkv;
        } else {
            const int heads = heads_of(rows, Hkv, wide);
            splits = splits_of(max_ctx, least_chunk(rows, wide, heads), Hkv / heads, tiles_of(rows));
            units = static_cast<int64_t>(splits) * tiles_of(rows) * (Hkv / heads);
            least = m;
        }
        l.parts |= splits > 1;
        rows_of[m] = part_rows(l.tc, m, Hq, Hkv, splits);
        if (units > most_units) most_units = units;
        if (rows_of[m] * best > rows_of[best] * m) best = m;
    }
    l.units = most_units * N;
    // For any price of a node, no batch has more rows than the price of all nodes and, for each tree, what the best size has over it.
    l.part_rows = INT64_MAX;
    const int next = least < max_nodes ? least + 1 : least;
    const int64_t prices[] = {0, (rows_of[best] + best - 1) / best, (rows_of[least] + least - 1) / least, (rows_of[next] + next - 1) / next,
                              (rows_of[max_nodes] + max_nodes - 1) / max_nodes};
    for (const int64_t price : prices) {
        int64_t over = 0;
        for (int m = 1; m <= max_nodes; ++m)
            if (rows_of[m] - price * m > over) over = rows_of[m] - price * m;
        const int64_t rows = price * T + over * N;
        if (rows < l.part_rows) l.part_rows = rows;
    }
    size_t off = KDA_WS_HEADER_BYTES;
    auto take = [&](size_t bytes) { const size_t at = off; off = align256(off + bytes); return at; };
    l.info = take((static_cast<size_t>(N) + 1) * sizeof(SeqInfo));
    l.info_tc = take(l.tc ? (static_cast<size_t>(N) + 1) * sizeof(SeqInfo) : 0);
    l.bad = take(static_cast<size_t>(N) * 4);
    l.seq_of = take(static_cast<size_t>(T) * 4);
    l.sees = take(static_cast<size_t>(T) * 8);
    l.odd = take(static_cast<size_t>(T) * 4);
    l.copy_v = take(max_nodes > 1 ? static_cast<size_t>(T) * Hkv * dv * sizeof(float) : 0);
    l.part_ml = take(static_cast<size_t>(l.part_rows) * sizeof(float2));
    l.part_o = take(static_cast<size_t>(l.part_rows) * dv * sizeof(float));
    l.total = off;
    return l;
}

template <int DK, int DV>
kda_status launch_attn(const AttnParams &p, kda_dtype dtype, const AttnLayout &l, cudaStream_t s) {
    const int sms = sm_count();
    if (sms <= 0) return KDA_ERR_CUDA;
    const int64_t seq_ctas = (static_cast<int64_t>(p.N) + kPlanThreads / 32 - 1) / (kPlanThreads / 32);
    const int64_t node_ctas = p.odd ? (p.T + kPlanThreads / 32 - 1) / (kPlanThreads / 32) : 0;
    const unsigned plan_ctas = static_cast<unsigned>(1 + seq_ctas + node_ctas);
    if (dtype == KDA_BF16) plan_kernel<__nv_bfloat16><<<plan_ctas, kPlanThreads, 0, s>>>(p, static_cast<int>(seq_ctas), DV);
    else plan_kernel<float><<<plan_ctas, kPlanThreads, 0, s>>>(p, static_cast<int>(seq_ctas), DV);
    const int64_t most = static_cast<int64_t>(sms) * (dtype == KDA_BF16 ? Ring<__nv_bfloat16, DK, DV>::kPerSm : Ring<float, DK, DV>::kPerSm);
    const dim3 grid(static_cast<unsigned>(l.units < most ? l.units : most));
    if (dtype == KDA_BF16) {
        using R = Ring<__nv_bfloat16, DK, DV>;
        constexpr int smem = R::kStages * R::kStage;
        if (!smem_opt_in<attn_kernel<__nv_bfloat16, DK, DV>>(smem)) return KDA_ERR_CUDA;
        if (launch_after(attn_kernel<__nv_bfloat16, DK, DV>, grid, R::kThreads, smem, s, p) != cudaSuccess) return KDA_ERR_CUDA;
        if (p.tc && launch_attn_tc(p, DK, DV, sms, s) != cudaSuccess) return KDA_ERR_CUDA;
    } else {
        using R = Ring<float, DK, DV>;
        constexpr int smem = R::kStages * R::kStage;
        if (!smem_opt_in<attn_kernel<float, DK, DV>>(smem)) return KDA_ERR_CUDA;
        if (launch_after(attn_kernel<float, DK, DV>, grid, R::kThreads, smem, s, p) != cudaSuccess) return KDA_ERR_CUDA;
    }
    if ((l.parts || p.odd) && (dtype == KDA_BF16 ? launch_combine<__nv_bfloat16, DV>(p, s) : launch_combine<float, DV>(p, s)) != cudaSuccess)
        return KDA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace
}  // namespace kda

extern "C" {

size_t kda_tree_attn_workspace_size_for(kda_dtype dtype, int N, int64_t T, int Hq, int Hkv, int dv, int max_nodes, int64_t max_ctx) {
    if (!kda::spec::dtype_ok(dtype) || N < 0 || T < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || !kda::spec::dim_ok(dv) || max_nodes < 1 ||
        max_nodes > KDA_MAX_TREE_NODES || max_ctx < 0 || max_ctx > 0x7fffffffLL)
        return 0;
    return kda::layout_of(dtype, N, T, Hq, Hkv, dv, max_nodes, max_ctx).total;
}

size_t kda_tree_attn_workspace_size(int N, int64_t T, int Hq, int Hkv, int dv, int max_nodes, int64_t max_ctx) {
    const size_t a = kda_tree_attn_workspace_size_for(KDA_BF16, N, T, Hq, Hkv, dv, max_nodes, max_ctx);
    const size_t b = kda_tree_attn_workspace_size_for(KDA_F32, N, T, Hq, Hkv, dv, max_nodes, max_ctx);
    return a > b ? a : b;
}

kda_status kda_tree_attn(const void *q, const void *k, const void *v, kda_dtype dtype, const kda_paged_kv *cache,
                         const int32_t *cu_nodes, const int32_t *parent, int N, int64_t T, int Hq, int Hkv, int dk,
                         int dv, int64_t q_stride, int64_t k_stride, int64_t v_stride, int max_nodes, float scale,
                         void *o, float *lse, void *workspace, size_t ws_bytes, void *stream) {
    using namespace kda::spec;
    if (!dtype_ok(dtype) || !dim_ok(dk) || !dim_ok(dv)) return KDA_ERR_UNSUPPORTED;
    if (N < 0 || N > (1 << 20) || T < 0 || T > 0x7fffffffLL || Hq <= 0 || Hkv <= 0 || Hq > 4096 || Hq % Hkv || T * Hq > 0x7fffffffLL)
        return KDA_ERR_INVALID_ARGUMENT;
    if (max_nodes < 1 || max_nodes > KDA_MAX_TREE_NODES || T > static_cast<int64_t>(N) * max_nodes) return KDA_ERR_INVALID_ARGUMENT;
    Pages c;
    kda_status st = check_pages(cache, dtype, N, &c);
    if (st != KDA_OK) return st;
    const int64_t max_ctx = static_cast<int64_t>(c.page_size) * c.max_pages;
    const kda::AttnLayout l = kda::layout_of(dtype, N, T, Hq, Hkv, dv, max_nodes, max_ctx);
    if (!workspace || !aligned_to(workspace, 16) || ws_bytes < l.total) return KDA_ERR_WORKSPACE;
    const int64_t vec = 16 / static_cast<int64_t>(elem_size(dtype));
    if (!q_stride) q_stride = static_cast<int64_t>(Hq) * dk;
    if (!k_stride) k_stride = static_cast<int64_t>(Hkv) * dk;
    if (!v_stride) v_stride = static_cast<int64_t>(Hkv) * dv;
    if (q_stride < static_cast<int64_t>(Hq) * dk || k_stride < static_cast<int64_t>(Hkv) * dk ||
        v_stride < static_cast<int64_t>(Hkv) * dv || q_stride % vec || k_stride % vec || v_stride % vec)
        return KDA_ERR_INVALID_ARGUMENT;
    if (N > 0 && (!cu_nodes || !aligned_to(cu_nodes, 4) || !aligned_to(parent, 4))) return KDA_ERR_INVALID_ARGUMENT;
    if (T > 0 && (!q || !k || !v || !o)) return KDA_ERR_INVALID_ARGUMENT;
    if (!aligned_to(q, 16) || !aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(o, 16) || !aligned_to(lse, 4))
        return KDA_ERR_INVALID_ARGUMENT;
    if (l.units > 0x7fffffffLL || l.part_rows > 0x7fffffffLL) return KDA_ERR_INVALID_ARGUMENT;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (N == 0 || T == 0) return cudaMemsetAsync(workspace, 0, sizeof(uint32_t), s) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
    char *ws = static_cast<char *>(workspace);
    kda::attn::AttnParams p{};
    p.q = q; p.k = k; p.v = v; p.o = o; p.lse = lse; p.c = c; p.cu = cu_nodes; p.parent = parent;
    p.T = T; p.qs = q_stride; p.ks = k_stride; p.vs = v_stride;
    p.N = N; p.Hq = Hq; p.Hkv = Hkv; p.G = Hq / Hkv; p.max_nodes = l.max_nodes; p.scale = scale;
    p.status = reinterpret_cast<uint32_t *>(ws);
    p.info = reinterpret_cast<kda::attn::SeqInfo *>(ws + l.info);
    p.info_tc = reinterpret_cast<kda::attn::SeqInfo *>(ws + l.info_tc);
    p.wide = dtype == KDA_F32;
    p.tc = l.tc;
    p.bad = reinterpret_cast<uint32_t *>(ws + l.bad);
    p.seq_of = reinterpret_cast<int32_t *>(ws + l.seq_of);
    p.sees = reinterpret_cast<uint64_t *>(ws + l.sees);
    if (l.max_nodes > 1) {
        p.given_v = v;
        p.given_vs = v_stride;
        p.v = ws + l.copy_v;
        p.vs = static_cast<int64_t>(Hkv) * dv;
        p.odd = reinterpret_cast<int32_t *>(ws + l.odd);
    }
    p.part_ml = reinterpret_cast<float2 *>(ws + l.part_ml);
    p.part_o = reinterpret_cast<float *>(ws + l.part_o);
    if (dk == 128) return dv == 128 ? kda::launch_attn<128, 128>(p, dtype, l, s) : kda::launch_attn<128, 64>(p, dtype, l, s);
    return dv == 128 ? kda::launch_attn<64, 128>(p, dtype, l, s) : kda::launch_attn<64, 64>(p, dtype, l, s);
}

}  // extern "C"
