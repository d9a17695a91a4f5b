// bd_attn_tile.cu -- attention of many query rows on the same keys: prefill, and
// the shared prefixes of a decode step.
//
// A unit is up to 256 query rows on one key/value head: the rows are (token,
// query head of the group) pairs, so that a group's heads read their keys once.
// 4 head_dim flops a row and key against 4 head_dim bytes a key: with 256 rows
// the tensor cores bound it.  One block a SM: two warps load keys and values by TMA
// through two rings, two issue the tcgen05 products (one of them loads the
// queries, too), two groups of four warps own 128 rows each, one thread a row.  Per block of 128 keys and group: S = Q K^T
// (both operands in shared memory); the row's thread takes its 128 scores to
// registers, keeps the running maximum and sum, and writes P as bf16 to tensor memory,
// from where O += P V reads it.  Tensor memory: one S (128 columns) that both groups
// take turns in -- it is free again as soon as it is in registers, so the next scores
// never wait for a softmax or for the product before -- P (64) and O (head_dim) of
// each group.  While one group works on its softmax the products of the other run.
// The output is only rescaled when a row's maximum has grown by more than 2^8
// since the last time (with every growth 750 us where this took 737 on 8192 tokens); P is then at most
// 2^8 and rounds no worse.  Its rounding to bf16 is the one that the products ask for;
// scores, maxima, sums and outputs stay f32.
// Measured (64 query heads on 8 of 128): a prompt of 8192 tokens 705-730 us call after
// call = 1.51-1.56 PFLOP/s, 79-82% of the measured bf16 burst rate and 88-91% of the sustained
// one (1360 W, the power cap holds the clock at 1.8 GHz), and 670 us in a short burst after a
// pause; 8 prompts of 333 to 2048 tokens behind up to 700, seeing
// 4 + 1024 keys, 267 us (their visible pairs alone 133).  The tensor pipe is active 73% of
// an SM's busy cycles; what is left are the hand-overs of S -- product to softmax and back,
// ~600 cycles each of ~1500 that a group's turn takes.  Blocks of 80 keys, for which both
// groups' S have room, took 896 us where 128 took 768: a softmax step costs ~600 cycles
// whatever its width.  With two or three warps a scheduler, an instruction on the way from
// one wait to the next costs 5 to 10 cycles: hence no divisions between units, no votes in
// the waits.  (The kernel is compiled with 152 bytes of spill stores and 172 of loads a
// thread: a softmax thread keeps a row's 128 scores beside the walk over the units.)
//
// With enough units each block takes whole ones and writes the result.  Else the
// blocks of keys of all units form one line that is cut into equal parts for the
// thread blocks, which leave unnormalised parts in the workspace; the decode
// kernel joins them with the requests' own keys, the join kernel those of a prefill.
#include <math.h>

#include <algorithm>

#include "bd_attn_math.cuh"
#include "bd_sm100.cuh"
#include "bd_tc_common.cuh"

namespace bd {
namespace attn {
namespace {

using namespace sm100;

constexpr int kKeys = 128;                 // of a block
constexpr int kThreads = 384;
constexpr uint32_t kLimit = 1u << 20;      // tries of a wait, of 1 us at most each
// Blocks that joining the parts costs about as much as.  Split / whole: 64 new tokens on
// 16,000 keys 46 / 182 us, on 2,000 29 / 34; but 700 tokens of a new prompt 54 / 23.
constexpr int kSplitPrice = 8;
constexpr float kGrow = 8.f;               // powers of two that a maximum may grow before a rescale

// Which of a tensor map's outer dimensions is which.
struct MapOrder {
    int32_t head, token, slot;
};

template <int D>
struct Tile {
    static constexpr int kHalves = D / 64;                 // 128-byte wide parts of a row
    static constexpr int kQ = 128 * D * 2;                 // bytes of 128 rows
    static constexpr int kK = D == 128 ? 3 : 4, kV = D == 128 ? 2 : 4;   // stages
    static constexpr int kSmem = 1024 + (2 + kK + kV) * kQ;
};

// Of a source: `head` blocks from its first key on, and `tail` blocks from key
// `from` on (a copy may start at any key, so a window costs no block for its
// alignment).
struct Span {
    int32_t head, from, tail;
};

// Keys [0, min(sinks, hi)) and [lo, hi) of a source.
__device__ __forceinline__ Span span_of(int lo, int hi, int sinks) {
    Span s;
    hi = max(hi, 0);
    lo = min(max(lo, 0), hi);
    s.head = (min(max(sinks, 0), hi) + kKeys - 1) / kKeys;
    s.from = max(lo, s.head * kKeys);
    s.tail = (max(hi - s.from, 0) + kKeys - 1) / kKeys;
    return s;
}

__device__ __forceinline__ int tokens_of_tile(int G) { return kPartRows / G; }

// The row tile's keys: a prefix (source 0) and the request's own (source 1).
__device__ __forceinline__ void set_keys(const Args& a, RowTile& t, int plen, int lo_min, int own_hi) {
    const Span p = span_of(lo_min, plen, a.sinks), o = span_of(lo_min - plen, own_hi, a.sinks - plen);
    t.off = plen;
    t.own_hi = own_hi;
    t.lo_min = lo_min;
    t.head[0] = p.head;
    t.from[0] = p.from;
    t.tail[0] = p.tail;
    t.head[1] = o.head;
    t.from[1] = o.from;
    t.tail[1] = o.tail;
    // a unit without keys still has its rows to write
    t.blocks = max(1, p.head + p.tail + o.head + o.tail);
}

// The largest v with table[v] <= x (table ascending, table[0] <= x).
template <typename T, typename X>
__device__ __forceinline__ int last_at_most(const T* table, int n, X x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (table[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

constexpr int kPlanThreads = 256;
constexpr int kLengths = 1024;
constexpr int kCached = 512;              // requests that the plan keeps in shared memory

// Sum of the threads before this one; the block's total.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* part, int64_t* total) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int64_t incl = v;
    for (int x = 1; x < 32; x <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, incl, x);
        if (lane >= x) incl += o;
    }
    if (lane == 31) part[warp] = incl;
    __syncthreads();
    int64_t before = 0, all = 0;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        before += w < warp ? part[w] : 0;
        all += part[w];
    }
    __syncthreads();
    *total = all;
    return before + incl - v;
}

// Lays out the row tiles of a call (one block).  Prefill: every request's rows in
// tiles of whole tokens.  Prefixes: the requests sorted by prefix (stably), every
// prefix's requests in tiles.  `split`: whether a prefill may be split; it is where
// a block's equal part of the line, with the parts' price, is less than the longest
// unit.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const Args a, const TilePlan plan, int blocks, int split) {
    extern __shared__ int32_t counts[];     // [P + 1] of each prefix, then its first place
    __shared__ int64_t part[kPlanThreads / 32];
    __shared__ Request cached[kCached];
    __shared__ int32_t first_tile[kCached];
    __shared__ int64_t lines[kPlanThreads];
    __shared__ int lengths[kLengths];       // tiles of each number of blocks
    __shared__ int longest, broken;
    grid_go_on();
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int per_tile = tokens_of_tile(a.G);
    int tiles = 0, sorted = 0;
    if (tid == 0) {
        longest = 0;
        broken = a.B;
    }
    __syncthreads();
    for (int b = tid; b < a.B; b += kPlanThreads) {
        if (b < kCached) cached[b] = read_request(a, b);
        // the first request whose rows do not follow from the ones before: it and those
        // behind it have no keys, and the rows from its own on become zeros (so the
        // tiles of a call never cover more than its rows)
        if (a.cu_q && (a.cu_q[b] < 0 || a.cu_q[b + 1] < a.cu_q[b] || a.cu_q[b + 1] > a.T)) atomicMin(&broken, b);
    }
    for (int i = tid; i < kLengths; i += kPlanThreads) lengths[i] = 0;
    if (!a.cu_q)
        for (int p = tid; p <= a.P; p += kPlanThreads) counts[p] = 0;
    __syncthreads();
    auto without_keys = [&](Request r, int b) {
        r.row0 = b == broken ? min(max(a.cu_q[b], 0), a.T) : a.T;
        r.rows = a.T - r.row0;
        r.len = r.plen = 0;
        return r;
    };
    if (broken < a.B) {
        for (int b = broken + tid; b < min(a.B, kCached); b += kPlanThreads) cached[b] = without_keys(cached[b], b);
        __syncthreads();
    }
    auto request = [&](int b) {
        if (b < kCached) return cached[b];
        const Request r = read_request(a, b);
        return b < broken ? r : without_keys(r, b);
    };
    if (a.cu_q) {
        for (int base = 0; base < a.B; base += kPlanThreads) {
            const int b = base + tid;
            const int n = b < a.B ? (request(b).rows + per_tile - 1) / per_tile : 0;
            int64_t all;
            const int first = tiles + (int)block_scan(n, part, &all);
            if (b < a.B) {
                if (b < kCached) first_tile[b] = first;
                plan.req_tile[b] = first;
            }
            tiles += (int)all;
        }
    } else {
        for (int b = tid; b < a.B; b += kPlanThreads) {
            if (request(b).plen > 0) atomicAdd(counts + a.prefix_ids[b], 1);
            else plan.req_tile[b] = -1;
        }
        __syncthreads();
        int first = 0;
        for (int base = 0; base < a.P; base += kPlanThreads) {
            const int p = base + tid;
            const int n = p < a.P ? counts[p] : 0;
            int64_t all, all_tiles;
            const int at = first + (int)block_scan(n, part, &all);
            const int t0 = tiles + (int)block_scan((n + per_tile - 1) / per_tile, part, &all_tiles);
            if (p < a.P) counts[p] = at;
            // what every tile of the group shares
            for (int i = 0; i * per_tile < n; ++i) {
                RowTile t{};
                t.slot[0] = a.prefix_slots[p];
                t.row0 = at + i * per_tile;
                t.tokens = min(per_tile, n - i * per_tile);
                t.off = a.prefix_lens[p];
                plan.tiles[t0 + i] = t;
            }
            first += (int)all;
            tiles += (int)all_tiles;
        }
        sorted = first;
        __syncthreads();
        if (warp == 0) {
            // stable placement, 32 requests at a time
            for (int base = 0; base < a.B; base += 32) {
                const int b = base + lane;
                int id = -1, pos = 0;
                if (b < a.B) {
                    const Request r = request(b);
                    id = r.plen > 0 ? a.prefix_ids[b] : -1;
                    pos = r.plen + r.len - 1;
                }
                const unsigned same = __match_any_sync(0xffffffffu, id);
                const int rank = __popc(same & ((1u << lane) - 1));
                const int at = id >= 0 ? counts[id] : 0;
                __syncwarp();
                if (id >= 0) {
                    plan.order[at + rank] = make_int2(b, pos);
                    if (rank == 0) counts[id] = at + __popc(same);
                }
                __syncwarp();
            }
        }
        __syncthreads();
        // a warp a tile: where its requests are, and the earliest key that they see
        for (int i = warp; i < tiles; i += kPlanThreads / 32) {
            const int row0 = plan.tiles[i].row0, n = plan.tiles[i].tokens;
            int lo = 0x7fffffff;
            for (int j = lane; j < n; j += 32) {
                const int2 r = plan.order[row0 + j];
                lo = min(lo, window_lo(a, r.y));
                plan.req_tile[r.x] = i;
                plan.req_row[r.x] = j * a.G;
            }
            lo = __reduce_min_sync(0xffffffffu, lo);
            if (lane == 0) plan.tiles[i].lo_min = lo;
        }
    }
    __syncthreads();
    // the tiles, and their places on the line of blocks
    auto tile_of = [&](int i) {
        RowTile t{};
        if (!a.cu_q) {
            t = plan.tiles[i];
            set_keys(a, t, t.off, t.lo_min, 0);
            return t;
        }
        const int b = a.B <= kCached ? last_at_most(first_tile, a.B, i) : last_at_most(plan.req_tile, a.B, i);
        const Request r = request(b);
        const int i0 = (i - (b < kCached ? first_tile[b] : plan.req_tile[b])) * per_tile;
        t.slot[0] = r.pslot;
        t.slot[1] = r.slot;
        t.row0 = r.row0 + i0;
        t.tokens = min(per_tile, r.rows - i0);
        t.t0 = r.plen + r.len - r.rows + i0;
        const int end = min(r.plen + r.len, t.t0 + t.tokens);
        set_keys(a, t, r.plen, window_lo(a, t.t0), max(0, end - r.plen));
        return t;
    };
    int64_t line = 0, rows = 0;
    for (int base = 0; base < tiles; base += kPlanThreads) {
        const int i = base + tid;
        RowTile t{};
        if (i < tiles) t = tile_of(i);
        int64_t all, all_rows;
        t.line = line + block_scan(t.blocks, part, &all);
        t.rows_before = rows + block_scan(t.tokens * a.G, part, &all_rows);
        line += all;
        rows += all_rows;
        if (i < tiles) {
            plan.tiles[i] = t;
            atomicMax(&longest, t.blocks);
            atomicAdd(lengths + min(t.blocks, kLengths - 1), 1);
        }
        if (base == 0) lines[tid] = t.line;
    }
    __syncthreads();
    const int64_t per = max((int64_t)1, (line * a.Hk + blocks - 1) / blocks);
    if (split && (!a.cu_q || longest > per + kSplitPrice)) {
        for (int c = tid; c < blocks && c * per < line * a.Hk; c += kPlanThreads) {
            // (the tiles' places: on chip where they are few)
            const int64_t x = c * per / a.Hk;
            int i = last_at_most(lines, min(tiles, kPlanThreads), x);
            if (tiles > kPlanThreads && plan.tiles[kPlanThreads].line <= x) {
                int lo = kPlanThreads, hi = tiles;
                while (hi - lo > 1) {
                    const int mid = (lo + hi) / 2;
                    if (plan.tiles[mid].line <= x) lo = mid;
                    else hi = mid;
                }
                i = lo;
            }
            const int n = plan.tiles[i].blocks;
            const int64_t in = c * per - plan.tiles[i].line * a.Hk;
            plan.starts[c] = make_int4(i, (int)(in / n), (int)(in % n), 0);
        }
    } else {
        split = 0;
    }
    if (!split && (int64_t)tiles * a.Hk > blocks) {
        // whole units are dealt from the last on: the tiles by their length (which of
        // two equal ones comes first changes no result)
        int mine = 0;
        for (int i = 0; i < kLengths / kPlanThreads; ++i) mine += lengths[tid * (kLengths / kPlanThreads) + i];
        int64_t all;
        int at = (int)block_scan(mine, part, &all);
        for (int i = 0; i < kLengths / kPlanThreads; ++i) {
            const int n = lengths[tid * (kLengths / kPlanThreads) + i];
            lengths[tid * (kLengths / kPlanThreads) + i] = at;
            at += n;
        }
        __syncthreads();
        for (int i = tid; i < tiles; i += kPlanThreads) {
            const RowTile t = tile_of(i);
            plan.tiles[atomicAdd(lengths + min(t.blocks, kLengths - 1), 1)] = t;
        }
    }
    if (tid == 0) *plan.head = PlanHead{tiles, line * a.Hk, per, split, sorted};
    // (the kernel before it has waited for all that this reads, and lets it begin beside itself)
    if (a.few) grid_wait();
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2,
                                            int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* r) {
    uint32_t* u = reinterpret_cast<uint32_t*>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
          "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
          "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
          "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
        : "r"(taddr));
}

// The way of a wait that one try did not end.
__device__ __forceinline__ void wait_on(uint64_t* bar, uint32_t parity, unsigned* status, unsigned where, volatile unsigned* dead) {
    for (uint32_t i = 0; i < kLimit; ++i)
        if (mbar_try_wait_ns(bar, parity, 1000) || *dead) return;
    *dead = 1;
    report(status, BD_ERR_TIMEOUT);
    atomicCAS(status + 2, 0u, where);
}
// The end of what is in flight, however the waits before went.
__device__ __forceinline__ void settle(uint64_t* bar, uint32_t parity) {
    for (uint32_t i = 0; i < kLimit; ++i)
        if (mbar_try_wait_ns(bar, parity, 1000)) return;
}

// Whether a phase is complete, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// The n lowest bits of a word (none below 0, all from 32).
__device__ __forceinline__ uint32_t first_bits(int n) {
    return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1;
}

// Two floats in a register pair, and the operations on both at once.
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float first_of(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float second_of(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
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
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Shared-memory descriptor of a 16-key slice of V: rows of 64 head_dim values
// (128 bytes, 128-byte swizzle), the reduction running over rows: groups of 8 rows
// are 1024 bytes apart, the second 64 values of a row 128 rows further.
__device__ __forceinline__ uint64_t desc_v(uint32_t addr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((addr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>((kKeys * 128) >> 4) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}
constexpr uint32_t kTransposeB = 1u << 16;   // instruction descriptor: B's rows run along the reduction

// One part of a unit that a block works on.
struct Segment {
    int tile, hk, first, last;               // blocks [first, last) of the unit
};

// The segments of this block, in order: its part of the line, or whole units from
// the last one on, dealt to the blocks to and fro (always the same way round, the
// first block would get the longest unit of every round: 11% of the SMs' time idle on
// a prompt of 8192 tokens).
struct Walk {
    int64_t left;                             // places of the part that are left
    int tile, hk, first;                      // the unit to come (tile < 0: none)
    int back_tiles, back_heads;               // how far the next whole unit lies before it,
    int then_tiles, then_heads;               // and the one after that before the next
    bool whole;
    __device__ __forceinline__ bool next(const Args& a, const TilePlan& plan, Segment& s) {
        if (whole ? tile < 0 : left <= 0) return false;
        const int n = plan.tiles[tile].blocks;
        s.tile = tile;
        s.hk = hk;
        s.first = first;
        s.last = n;
        if (whole) {
            tile -= back_tiles;
            hk -= back_heads;
            if (hk < 0) {
                hk += a.Hk;
                --tile;
            }
            const int tiles = back_tiles, heads = back_heads;
            back_tiles = then_tiles;
            back_heads = then_heads;
            then_tiles = tiles;
            then_heads = heads;
            return true;
        }
        if (n - first > left) s.last = first + (int)left;
        left -= s.last - first;
        first = 0;
        if (++hk == a.Hk) {
            hk = 0;
            ++tile;
        }
        return true;
    }
};

// Block i of a row tile: its source, first key and the source's end.
struct Block {
    int src, slot, key, end, off, run;       // run: blocks from this one on that follow one another
};
__device__ __forceinline__ Block block_of(const RowTile& t, int i) {
    Block b;
    b.src = i >= t.head[0] + t.tail[0];
    if (b.src) i -= t.head[0] + t.tail[0];
    const int head = b.src ? t.head[1] : t.head[0], from = b.src ? t.from[1] : t.from[0];
    b.key = i < head ? i * kKeys : from + (i - head) * kKeys;
    b.slot = b.src ? t.slot[1] : t.slot[0];
    b.run = i < head ? head - i : head + (b.src ? t.tail[1] : t.tail[0]) - i;
    if (b.run < 1) b.run = 1;
    b.off = b.src ? t.off : 0;
    b.end = b.src ? t.own_hi : t.off;
    return b;
}

// A thread's row of a unit: its row of q (-1: none), its head and the positions
// [lo, hi) that it sees; a row that is none sees all.
struct RowOf {
    int row, head, lo, hi;
    int lo_unit, rows;                         // the least lo of the unit's rows, their number
    int skipped;                               // blocks of units before it without a part of its group
};
__device__ __forceinline__ RowOf row_of(const Args& a, const TilePlan& plan, const RowTile& t, int hk, int r) {
    RowOf o{-1, hk * a.G, 0, 0x7fffffff, t.lo_min, t.tokens * a.G, 0};
    const int token = r / a.G;
    if (token >= t.tokens) return o;
    o.head += r - token * a.G;
    o.row = t.row0 + token;
    int pos = t.t0 + token;
    if (!a.cu_q) {
        const int2 r = plan.order[o.row];
        o.row = r.x;
        pos = r.y;
    }
    o.hi = pos + 1;
    o.lo = window_lo(a, pos);
    return o;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    tile_kernel(const Args a, const TilePlan plan, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap, const MapOrder order) {
    using T = Tile<D>;
    constexpr int NK = T::kK, NV = T::kV;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t k_full[NK], k_empty[NK], v_full[NV], v_empty[NV], q_full, q_empty, s_full[2], s_free, p_full[2],
        pv_done[2], drained[2];
    __shared__ uint32_t tmem_at;
    __shared__ unsigned dead;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    unsigned* status = a.status;
    // Waits.  One that runs out ends all others at once, and the status word tells: no
    // copy is started any more (a barrier that still expects one may not be armed
    // again), the other roles go through their steps without waiting, on whatever is
    // there, and the copies and products under way are waited for at the end.
    auto wait = [&](uint64_t* bar, uint32_t parity, unsigned where) {
        if (!mbar_try_wait(bar, parity & 1)) wait_on(bar, parity & 1, status, where, &dead);
    };
    auto is_dead = [&]() { return *static_cast<volatile unsigned*>(&dead) != 0; };
    auto warp_waits = [&](uint64_t* bar, uint32_t parity, unsigned where) {
        wait(bar, parity, where);
        __syncwarp();
    };
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    const uint32_t q_at = base, k_at = base + 2 * T::kQ, v_at = k_at + NK * T::kQ;

    if (warp == 8) tmem_alloc(&tmem_at, 512);
    if (tid == 0) {
        for (int i = 0; i < NK; ++i) {
            mbar_init(k_full + i, 1);
            mbar_init(k_empty + i, 1);
        }
        for (int i = 0; i < NV; ++i) {
            mbar_init(v_full + i, 1);
            mbar_init(v_empty + i, 1);
        }
        dead = 0;
        mbar_init(&s_free, 4);
        mbar_init(&q_full, 1);
        mbar_init(&q_empty, 1);
        mbar_init(drained, 1);
        mbar_init(drained + 1, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full + i, 1);
            mbar_init(p_full + i, 4);
            mbar_init(pv_done + i, 1);
        }
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_wait();                              // the plan
    grid_go_on();
    const PlanHead head = *plan.head;
    const bool split = head.split;
    Walk walk{};
    if (split) {
        const int64_t at = min(head.line, head.per * blockIdx.x);
        walk.left = min(head.line - at, head.per);
        if (walk.left > 0) {
            const int4 start = plan.starts[blockIdx.x];
            walk.tile = start.x;
            walk.hk = start.y;
            walk.first = start.z;
        }
    } else {
        // the last tile of a prompt has the most keys: begin there
        const int64_t u = head.tiles * a.Hk - 1 - blockIdx.x;
        walk.tile = u < 0 ? -1 : (int)(u / a.Hk);
        walk.hk = u < 0 ? 0 : (int)(u % a.Hk);
        const int to = 2 * (int)(gridDim.x - blockIdx.x) - 1, fro = 2 * (int)blockIdx.x + 1;
        walk.back_tiles = to / a.Hk;
        walk.back_heads = to % a.Hk;
        walk.then_tiles = fro / a.Hk;
        walk.then_heads = fro % a.Hk;
        walk.whole = true;
    }
    const uint32_t tmem = tmem_at;

    // registers: 3 x 168 for each lane of the three warp groups at launch; the loading
    // and issuing group gives 32 of its own to each of the others, whose threads keep
    // a row's 128 scores
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        if ((warp == 8 || warp == 11) && lane == 0) {
            // keys (warp 8) and values (warp 11)
            const bool keys = warp == 8;
            const CUtensorMap* map = keys ? &kmap : &vmap;
            uint64_t *full = keys ? k_full : v_full, *empty = keys ? k_empty : v_empty;
            const int stages = keys ? NK : NV;
            const uint32_t to = keys ? k_at : v_at;
            prefetch_tensormap(map);
            int st = 0, put = 0;
            uint32_t phase = 1;                    // of the fill before the one to come
            Segment s;
            while (!is_dead() && walk.next(a, plan, s)) {
                const RowTile t = plan.tiles[s.tile];
                for (int i = s.first; i < s.last; ++i, ++put) {
                    const Block b = block_of(t, i);
                    auto at = [&](int dim) { return dim == order.token ? b.key : dim == order.head ? s.hk : b.slot; };
                    if (put >= stages) wait(empty + st, phase, 1);
                    if (is_dead()) break;
                    mbar_expect_tx(full + st, T::kQ);
                    for (int h = 0; h < T::kHalves; ++h)
                        tma_load_4d(to + st * T::kQ + h * kKeys * 128, map, full + st, h * 64, at(0), at(1), at(2));
                    if (++st == stages) {
                        st = 0;
                        phase ^= 1;
                    }
                }
            }
            // nothing may still be on its way into shared memory when the block ends
            for (int i = max(0, put - stages); i < put; ++i) settle(full + i % stages, i / stages & 1);
        }
        // Two warps issue the products, one the scores' and one the outputs'.  A product's
        // issue takes as long as the product (64 cycles for 128 x 128 x 16), and the waits
        // and the bookkeeping between two batches half as long as a batch: so they overlap
        // the other warp's products.
        constexpr uint32_t idesc_s = idesc_bf16(128, kKeys), idesc_o = idesc_bf16(128, D) | kTransposeB;
        if (warp == 9) {
            const uint64_t q_desc = desc_sw128(q_at), k_desc = desc_sw128(k_at);
            uint32_t st = 0, phase = 0, n = 0, n1 = 0, units = 0;
            Segment s;
            if (lane == 0) prefetch_tensormap(&qmap);
            while (walk.next(a, plan, s)) {
                const int groups = plan.tiles[s.tile].tokens * a.G > 128 ? 2 : 1;
                const int row0 = plan.tiles[s.tile].row0;
                // the unit's queries, in the order of its rows (the tile's whole room: what
                // lies behind its tokens belongs to rows that are none)
                if (units > 0) warp_waits(&q_empty, units - 1, 2);
                if (is_dead()) break;
                if (elect_one()) {
                    mbar_expect_tx(&q_full, T::kHalves * tokens_of_tile(a.G) * a.G * 128);
                    for (int h = 0; h < T::kHalves; ++h) tma_load_3d(q_at + h * kPartRows * 128, &qmap, &q_full, h * 64, s.hk * a.G, row0);
                }
                __syncwarp();
                wait(&q_full, units++, 3);
                for (int i = s.first; i < s.last; ++i) {
                    const uint64_t kd = k_desc + (st * T::kQ >> 4);
                    wait(k_full + st, phase, 4);
                    for (int g = 0; g < groups; ++g) {
                        const uint64_t qd = q_desc + (g * 128 * 128 >> 4);
                        const bool last = g == groups - 1;
                        // (so that the issuer of the outputs, which looks for the second group's
                        // next scores, finds them one phase ahead at most)
                        if (g == 1 && n1++ > 1 && i > s.first + 1) wait(pv_done + 1, n1 - 3, 12);
                        // the scores before, of whichever group, are in registers
                        if (n > 0) wait(&s_free, n - 1, 5);
                        __syncwarp();
                        ++n;
                        tc_fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < D / 16; ++k)
                                mma_ss(tmem, qd + (((k / 4) * (kPartRows * 128) + (k % 4) * 32) >> 4), kd + (((k / 4) * (kKeys * 128) + (k % 4) * 32) >> 4),
                                       idesc_s, k > 0);
                            mma_commit(s_full + g);
                            if (last) mma_commit(k_empty + st);
                            if (last && i + 1 == s.last) mma_commit(&q_empty);
                        }
                        __syncwarp();
                    }
                    if (++st == NK) {
                        st = 0;
                        phase ^= 1;
                    }
                }
            }
            // the products in flight end before the tensor memory is given back
            if (elect_one()) mma_commit(drained);
            __syncwarp();
            settle(drained, 0);
            if (units > 0) settle(&q_full, units - 1 & 1);
        }
        if (warp == 10) {
            const uint64_t v_desc = desc_v(v_at);
            uint32_t st = 0, phase = 0, done0 = 0, done1 = 0;
            Segment s;
            while (walk.next(a, plan, s)) {
                const int groups = plan.tiles[s.tile].tokens * a.G > 128 ? 2 : 1;
                for (int i = s.first; i < s.last; ++i) {
                    wait(v_full + st, phase, 6);
                    for (int g = 0; g < groups; ++g) {
                        warp_waits(p_full + g, g ? done1++ : done0++, 7);
                        // the second group's output after its next scores: these are the ones that
                        // a hand-over waits for (8192 tokens 755 -> 716 us; the first group's would
                        // be looked for too late at a unit's end)
                        if (g == 1 && i + 1 < s.last) warp_waits(s_full + 1, done1, 13);
                        tc_fence_after();
                        if (elect_one()) {
                            const uint64_t vd = v_desc + (st * T::kQ >> 4);
                            const uint32_t o = tmem + 256 + g * D, p = tmem + 128 + g * 64;
#pragma unroll
                            for (int k = 0; k < kKeys / 16; ++k)
                                mma_ts(o, p + k * 8, vd + (k * 2048 >> 4), idesc_o, i > s.first || k > 0);
                            mma_commit(pv_done + g);
                            if (g == groups - 1) mma_commit(v_empty + st);
                        }
                        __syncwarp();
                    }
                    if (++st == NV) {
                        st = 0;
                        phase ^= 1;
                    }
                }
            }
            if (elect_one()) mma_commit(drained + 1);
            __syncwarp();
            settle(drained + 1, 0);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        // a group of 128 rows, one thread a row
        const int g = warp / 4, r = g * 128 + tid % 128;
        const uint32_t lanes = static_cast<uint32_t>((warp % 4) * 32) << 16;
        const uint32_t s_at = tmem + lanes, p_at = s_at + 128 + g * 64, o_at = s_at + 256 + g * D;
        const float scale = fmaxf(fabsf(a.scale_log2), 1.2e-38f);   // never 0: a hidden score's -inf stays -inf
        int step = 0, put = 0;
        bool more = true;
        Segment s, coming;
        RowOf now{}, next{};
        // this thread's row of the next unit that its group has a part in
        auto begin_next = [&]() {
            while ((more = walk.next(a, plan, coming))) {
                const RowTile& t = plan.tiles[coming.tile];
                const int tokens = t.tokens;
                if (g == 0 || tokens * a.G > 128) {
                    const int skipped = next.skipped;
                    next = row_of(a, plan, t, coming.hk, r);
                    next.skipped = skipped;
                    break;
                }
                next.skipped += coming.last - coming.first;
            }
        };
        begin_next();
        while (more) {
            s = coming;
            now = next;
            next.skipped = 0;
            put += now.skipped;
            // the warp's rows all see [lo_all, hi_all)
            const int hi_all = __reduce_min_sync(0xffffffffu, now.hi), lo_all = __reduce_max_sync(0xffffffffu, now.lo);
            float m = -INFINITY, l = 0.f;
            int p0 = 0, src_end = 0, run = 0;      // the block's first position, its source's end, blocks until another source or a gap
            for (int i = s.first; i < s.last; ++i, ++step, ++put) {
                if (run == 0) {
                    const RowTile t = plan.tiles[s.tile];
                    const Block b = block_of(t, i);
                    p0 = b.off + b.key;
                    src_end = b.off + b.end;
                    run = b.run;
                }
                warp_waits(s_full + g, step, 8);
                tc_fence_after();
                float v[kKeys];
#pragma unroll
                for (int c = 0; c < kKeys; c += 32) tmem_ld32(s_at + c, v + c);
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_free);
                // asked now, needed later: P and O are free when the block before is done
                const bool free = step == 0 || mbar_test(pv_done + g, (step - 1) & 1);
                if (a.scale_log2 < 0.f) {
                    // scores are scaled by its size
#pragma unroll
                    for (int c = 0; c < kKeys; ++c) {
                        asm volatile("" : "+f"(v[c]));
                        v[c] = -v[c];
                    }
                }
                if (!(p0 + kKeys <= min(src_end, hi_all) && (p0 >= lo_all || p0 + kKeys <= a.sinks))) {
                    const int n = min(now.hi, src_end) - p0, from = now.lo - p0, sinks = a.sinks - p0;
#pragma unroll
                    for (int c = 0; c < kKeys; c += 32) {
                        uint32_t seen = first_bits(n - c) & (first_bits(sinks - c) | ~first_bits(from - c));
                        // (opaque, or the compiler evaluates the masks of all blocks)
                        asm volatile("" : "+r"(seen));
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[c + e] = seen >> e & 1 ? v[c + e] : -INFINITY;
                    }
                }
                float top[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    top[e] = fmaxf(v[e], v[4 + e]);
#pragma unroll
                    for (int c = 8; c < kKeys; c += 8) top[e] = max3(top[e], v[c + e], v[c + 4 + e]);
                }
                const float mx = max3(top[0], top[1], fmaxf(top[2], top[3]));
                const float mn = fmaxf(m, mx == -INFINITY ? -INFINITY : mx * scale);
                const bool grows = mn > m + kGrow || (m == -INFINITY && mn > m);
                const bool edge = g == 0 && !(p0 + kKeys <= src_end && (p0 >= now.lo_unit || p0 + kKeys <= a.sinks));
                const bool rescales = i > s.first && grows;
                if (i == s.first) m = mn;
                if (__any_sync(0xffffffffu, rescales || edge || !free)) {
                    if (step > 0) warp_waits(pv_done + g, step - 1, 9);
                    if (edge) {
                        // values that no row of the unit sees may be anything: they are
                        // multiplied by zero, so they have to be finite.  (The first group
                        // has a part in every unit and its product comes first.)
                        const int pos = p0 + tid, st = put % NV;
                        warp_waits(v_full + st, put / NV, 10);
                        if (!(pos < src_end && (pos < a.sinks || pos >= now.lo_unit)))
#pragma unroll
                            for (int c = 0; c < D / 8; ++c)
                                asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(v_at + st * T::kQ + (c / 8) * (kKeys * 128) + tid * 128 + (c % 8) * 16), "r"(0u)
                                             : "memory");
                        fence_proxy_async_smem();
                    }
                    if (__any_sync(0xffffffffu, rescales)) {
                        tc_fence_after();
                        float f = 1.f;
                        if (rescales) {
                            f = exp2_approx(m - mn);
                            m = mn;
                            l *= f;
                        }
#pragma unroll
                        for (int c = 0; c < D; c += 16) {
                            uint32_t o[16];
                            tmem_ld16(o_at + c, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st16(o_at + c, o);
                        }
                    }
                }
                tc_fence_after();
                const float use = m == -INFINITY ? 0.f : m;
                const uint64_t scale2 = pair(scale, scale), use2 = pair(-use, -use);
                uint64_t sum[2] = {0, 0};
#pragma unroll
                for (int c = 0; c < kKeys; c += 32) {
                    uint32_t p[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const uint64_t x = fma2(pair(v[c + e], v[c + e + 1]), scale2, use2);
                        const float y0 = exp2_approx(first_of(x)), y1 = exp2_approx(second_of(x));
                        sum[e / 2 % 2] = add2(sum[e / 2 % 2], pair(y0, y1));
                        p[e / 2] = pack_bf16(y0, y1);
                    }
                    tmem_st16(p_at + c / 2, p);
                }
                sum[0] = add2(sum[0], sum[1]);
                l += first_of(sum[0]) + second_of(sum[0]);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + g);
                p0 += kKeys;
                --run;
            }
            begin_next();
            warp_waits(pv_done + g, step - 1, 11);
            tc_fence_after();
            const bool real = now.row >= 0;
            const float inv = inverse(l);
            if (split) {
                const int64_t part_row = plan.tiles[s.tile].rows_before * a.Hk + (int64_t)s.hk * now.rows + (int64_t)blockIdx.x * kPartRows;
                if (real) plan.ml[part_row + r] = make_float2(m, l);
                // four values of all rows, then the next four: a warp writes 512 bytes in a row
                float4* to = reinterpret_cast<float4*>(plan.o + part_row * D) + r;
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    float o[32];
                    tmem_ld32(o_at + c, o);
                    tmem_ld_wait();
                    if (real)
#pragma unroll
                        for (int e = 0; e < 8; ++e) to[(int64_t)(c / 4 + e) * now.rows] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                }
            } else {
                // four lanes exchange 16-byte pieces, so that they write 64 bytes of a row
                // together: one lane a row would touch a line with every 16 bytes
                int64_t at[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = __shfl_sync(0xffffffffu, now.row, lane / 4 * 4 + i), head_at = __shfl_sync(0xffffffffu, now.head, lane / 4 * 4 + i);
                    at[i] = row < 0 ? -1 : ((int64_t)row * a.Hq + head_at) * D + lane % 4 * 8;
                }
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    float o[32];
                    tmem_ld32(o_at + c, o);
                    tmem_ld_wait();
                    uint32_t x[4][4];
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[e / 4][e % 4] = pack_bf16(o[2 * e] * inv, o[2 * e + 1] * inv);
#pragma unroll
                    for (int bit = 1; bit < 4; bit *= 2)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (!(i & bit))
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const bool up = lane & bit;
                                    const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? x[i][e] : x[i + bit][e], bit);
                                    x[i][e] = up ? got : x[i][e];
                                    x[i + bit][e] = up ? x[i + bit][e] : got;
                                }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (at[i] >= 0) *reinterpret_cast<uint4*>(a.out + at[i] + c) = make_uint4(x[i][0], x[i][1], x[i][2], x[i][3]);
                }
            }
            tc_fence_before();
        }
    }
    __syncthreads();
    if (warp == 8) tmem_dealloc(tmem, 512);
}

// Adds the parts of row r of a unit of `rows` rows, four values; four parts at a
// time, so that their loads are under way together.
template <int D>
__device__ __forceinline__ void add_parts(const TilePlan& plan, const Parts& p, int rows, int r, int col, float& m, float& l, float4& o) {
    for (int s0 = 0; s0 < p.n; s0 += 4) {
        float2 ml[4];
        float4 v[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int64_t at = p.row0 + (int64_t)min(s0 + s, p.n - 1) * kPartRows;
            ml[s] = plan.ml[at + r];
            v[s] = reinterpret_cast<const float4*>(plan.o + at * D)[(int64_t)(col / 4) * rows + r];
        }
        float top = m;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            if (s0 + s >= p.n) ml[s] = make_float2(-INFINITY, 0.f);
            top = fmaxf(top, ml[s].x);
        }
        const float use = top == -INFINITY ? 0.f : top;
        float f = exp2_approx(m - use);
        l *= f;
        o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            if (s0 + s >= p.n) break;
            f = exp2_approx(ml[s].x - use);
            l += f * ml[s].y;
            o.x += f * v[s].x;
            o.y += f * v[s].y;
            o.z += f * v[s].z;
            o.w += f * v[s].w;
        }
        m = top;
    }
}

__device__ __forceinline__ uint2 result(float4 o, float l) {
    const float inv = inverse(l);
    return make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
}

// Joins the parts of a split prefill: one thread four values of a row.
template <int D>
__global__ void __launch_bounds__(256) join_kernel(const Args a, const TilePlan plan) {
    grid_wait();
    const PlanHead head = *plan.head;
    if (!head.split) return;
    const int u = blockIdx.x;
    if (u >= head.tiles * a.Hk) return;
    const RowTile& t = plan.tiles[u / a.Hk];
    const int hk = u % a.Hk, rows = t.tokens * a.G;
    const Parts parts = parts_of(t, head, a.Hk, hk, a.G);
    for (int i = blockIdx.y * 256 + threadIdx.x; i < rows * (D / 4); i += 256 * gridDim.y) {
        const int r = i % rows, col = i / rows * 4;
        float m = -INFINITY, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        add_parts<D>(plan, parts, rows, r, col, m, l, o);
        const int64_t to = ((int64_t)(t.row0 + r / a.G) * a.Hq + hk * a.G + r % a.G) * D + col;
        *reinterpret_cast<uint2*>(a.out + to) = result(o, l);
    }
}

// Joins a decode step's parts: what a row's own keys gave (the decode kernel) and
// what its prefix gave.
template <int D>
__global__ void __launch_bounds__(256) join_prefix_kernel(const Args a, const TilePlan plan, const DecodeBuffers buf) {
    grid_wait();
    // 8 rows of one column after the other, then the next column
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, eight = i / (8 * (D / 4));
    const int64_t row = eight * 8 + i % 8;
    if (row >= (int64_t)a.B * a.Hq) return;
    const int col = (int)(i / 8 % (D / 4)) * 4, b = (int)(row / a.Hq), h = (int)(row % a.Hq);
    const float2 ml = buf.own_ml[row];
    float m = ml.x, l = ml.y;
    float4 o = *reinterpret_cast<const float4*>(buf.own + row * D + col);
    const int tile = plan.req_tile[b];
    if (tile >= 0) {
        const RowTile& t = plan.tiles[tile];
        add_parts<D>(plan, parts_of(t, *plan.head, a.Hk, h / a.G, a.G), t.tokens * a.G, plan.req_row[b] + h % a.G, col, m, l, o);
    }
    *reinterpret_cast<uint2*>(a.out + row * D + col) = result(o, l);
    if (a.weights && col == 0) buf.lse[row] = log_sum(m, l);
}

// The cache as a 4-D tensor whose dimensions follow their strides, whichever
// layout it has; a dimension of one entry comes last.
bool cache_map(CUtensorMap* map, MapOrder* order, const void* base, const Args& a, int D) {
    struct Dim {
        int64_t stride, size;
        int32_t* place;
        uint32_t box;
    } d[3] = {{a.sh, a.Hk, &order->head, 1}, {a.st, a.capacity, &order->token, kKeys}, {a.ss, a.n_slots, &order->slot, 1}};
    std::sort(d, d + 3, [](const Dim& x, const Dim& y) {
        return (x.size == 1) != (y.size == 1) ? y.size == 1 : x.size > 1 && x.stride < y.stride;
    });
    uint64_t dims[4] = {(uint64_t)D}, strides[3];
    uint32_t box[4] = {64};
    int64_t next = D;
    for (int i = 0; i < 3; ++i) {
        const int64_t stride = d[i].size == 1 ? next : d[i].stride;
        next = stride * d[i].size;
        strides[i] = (uint64_t)stride * 2;
        dims[i + 1] = (uint64_t)d[i].size;
        box[i + 1] = d[i].box;
        *d[i].place = i;
    }
    return make_tmap_bf16_sw128_nd(map, base, 4, dims, strides, box);
}

// Rows of q: a box is the heads of a group of a tile's tokens.
bool query_map(CUtensorMap* map, const void* q, int64_t q_stride, const Args& a, int D) {
    const uint64_t dims[3] = {(uint64_t)D, (uint64_t)a.Hq, (uint64_t)a.T};
    const uint64_t strides[2] = {(uint64_t)D * 2, (uint64_t)q_stride * 2};
    const uint32_t box[3] = {64, (uint32_t)a.G, (uint32_t)(kPartRows / a.G)};
    return make_tmap_bf16_sw128_nd(map, q, 3, dims, strides, box);
}

template <int D>
bd_status launch_kernel(const Args& a, const TilePlan& plan, cudaStream_t stream) {
    const void* kernel = reinterpret_cast<const void*>(tile_kernel<D>);
    if (!set_smem_attr(kernel, Tile<D>::kSmem, D == 128 ? 8 : 9)) return BD_ERR_CUDA;
    CUtensorMap qmap, kmap, vmap;
    MapOrder order{};
    // (a decode step's queries were put in the order of the prefixes)
    if (!query_map(&qmap, a.cu_q ? a.q : plan.sorted_q, a.cu_q ? a.q_stride : (int64_t)a.Hq * D, a, D)) return BD_ERR_CUDA;
    if (!cache_map(&kmap, &order, a.k, a, D) || !cache_map(&vmap, &order, a.v, a, D)) return BD_ERR_CUDA;
    return launch_close(tile_kernel<D>, tile_blocks(), kThreads, Tile<D>::kSmem, stream, a, plan, qmap, kmap, vmap, order);
}

}  // namespace

// Row tiles that a call can have at most.
int64_t most_tiles(int64_t tokens, int64_t batch, int G) { return tokens / (kPartRows / G) + batch; }

int tile_blocks() { return decode_blocks(); }
int64_t split_below() { return 2 * (int64_t)tile_blocks(); }

// Row tiles that this call can have at most.  (Of requests that have more than `few` rows there are fewer; one more may
// end the rows that are served.)
int64_t most_tiles(const Args& a) {
    const int64_t most = a.few ? a.T / (a.few + 1) + 1 : a.B;
    return most_tiles(a.T, most < a.B ? most : a.B, a.G);
}

// Whether a call's parts may be left in the workspace, which holds those of few rows: a
// prefill of few units, if a unit can be longer than the parts' price at all.
bool may_split(const Args& a) {
    if (!a.cu_q) return true;
    const int source = ((a.longest ? a.longest : a.capacity) + kKeys - 1) / kKeys + 1;
    return most_tiles(a) * a.Hk < split_below() && source * (a.prefix_ids ? 2 : 1) > kSplitPrice + 1;
}

bd_status launch_plan(const Args& a, const TilePlan& plan, cudaStream_t stream) {
    const int counts = a.cu_q ? 0 : (a.P + 1) * (int)sizeof(int);
    if (!set_smem_attr(reinterpret_cast<const void*>(plan_kernel), (kMaxPrefixes + 1) * (int)sizeof(int), 10)) return BD_ERR_CUDA;
    if (a.few) return launch_close(plan_kernel, 1, kPlanThreads, counts, stream, a, plan, tile_blocks(), (int)may_split(a));
    plan_kernel<<<1, kPlanThreads, counts, stream>>>(a, plan, tile_blocks(), may_split(a));
    return launch_status();
}

bd_status launch_prefill(const Args& a, int head_dim, const TilePlan& plan, cudaStream_t stream) {
    const bd_status st = launch_plan(a, plan, stream);
    return st == BD_OK ? launch_tiles(a, head_dim, plan, stream) : st;
}

bd_status launch_tiles(const Args& a, int head_dim, const TilePlan& plan, cudaStream_t stream) {
    const bd_status st = head_dim == 128 ? launch_kernel<128>(a, plan, stream) : launch_kernel<64>(a, plan, stream);
    if (st != BD_OK || !may_split(a)) return st;
    // (few units are joined by many blocks each)
    const int64_t units = most_tiles(a) * a.Hk, each = 8 * (int64_t)tile_blocks() / units;
    const dim3 grid((unsigned)units, (unsigned)(each < 4 ? 4 : each > 32 ? 32 : each));
    return head_dim == 128 ? launch_close(join_kernel<128>, grid, 256, 0, stream, a, plan)
                           : launch_close(join_kernel<64>, grid, 256, 0, stream, a, plan);
}

bd_status launch_prefixes(const Args& a, int head_dim, const TilePlan& plan, const DecodeBuffers& buf,
                          cudaStream_t stream) {
    const bd_status st = head_dim == 128 ? launch_kernel<128>(a, plan, stream) : launch_kernel<64>(a, plan, stream);
    if (st != BD_OK) return st;
    const unsigned blocks = (unsigned)((((int64_t)a.B * a.Hq + 7) / 8 * 8 * (head_dim / 4) + 255) / 256);
    return head_dim == 128 ? launch_close(join_prefix_kernel<128>, blocks, 256, 0, stream, a, plan, buf)
                           : launch_close(join_prefix_kernel<64>, blocks, 256, 0, stream, a, plan, buf);
}

}  // namespace attn
}  // namespace bd
