// bd_attn_line.cuh -- how the decode kernels share out a call: the tiles of visible
// keys of all (request, key/value head) units form one line that is cut into equal
// parts for the blocks and again for their warps, and units that several warps or
// blocks share are joined in their order, so that the result does not depend on
// timing.
//
// `Keys` says which keys of a request a tile holds, and what a unit costs:
//   static Keys of(const Args&, const Request&),
//   int tiles() >= 1,
//   kAllKept    whether its calls have no more than kKept requests
//   kUnitCost   places of a unit besides its tiles
//   kLeast      places of a block
//   kShort      tiles up to which a unit may have a block of its own
//   kJoin       parts of a unit whose loads are under way together when they are joined
#pragma once

#include "bd_attn_math.cuh"

namespace bd {
namespace attn {

constexpr int kKept = 1024;               // requests that a block keeps on chip
constexpr int kRuns = 128;                // runs of requests that a block looks its place up in

// The line: every unit takes kUnitCost places (what a unit costs besides its tiles:
// its query, its result) and one for each tile.  If all units are short and no more
// than the blocks, each has a block of its own instead: `each` places.
template <typename Keys>
struct Line {
    int64_t lo, hi;                        // this warp's places
    int64_t per;                           // places of a block
    int32_t each;                          // 0: units follow one another
    __device__ __forceinline__ int length(int tiles) const { return each ? each : Keys::kUnitCost + tiles; }
    __device__ __forceinline__ int lead() const { return each ? 0 : Keys::kUnitCost; }
};

// A unit on the line and its tiles [tile, end) that lie in the warp's part.
template <typename Keys>
struct Cursor {
    int b, u, tiles, tile, end;
    int64_t start;                         // the unit's first place
    Request r;
    Keys k;
};

// What a block keeps of the first requests: read once, at its beginning.  Later the
// same loads would queue behind the keys' (2 to 4 thousand cycles each).
struct Kept {
    int32_t slot, len, plen;
};

struct Record {                            // an open unit of a warp
    int valid, b, u, tiles, open_start, open_end;
    int64_t start;
};

// A block's shared memory for all this.
template <int W>
struct LineBlock {
    int64_t sums[kRuns + 1];
    int longest[kRuns / 32];
    Kept kept[kKept];
    Record records[2 * W];
    int chain[2 * W];
    int last_block;
};

template <typename Keys>
__device__ __forceinline__ void load_request(const Args& a, const Kept* kept, Cursor<Keys>& c) {
    if (Keys::kAllKept || c.b < kKept) {
        c.r.slot = kept[c.b].slot;
        c.r.len = kept[c.b].len;
        c.r.plen = kept[c.b].plen;
    } else if constexpr (!Keys::kAllKept) {
        c.r = read_request<true>(a, c.b);
    }
    c.k = Keys::of(a, c.r);
    c.tiles = c.k.tiles();
}

// Goes on to the first unit from c on with tiles in the part; false if there is none.
template <typename Keys>
__device__ __forceinline__ bool seek(const Args& a, const Kept* kept, const Line<Keys>& line, Cursor<Keys>& c, int units) {
    while (c.start < line.hi) {
        const int64_t first = c.start + line.lead();
        c.tile = (int)min(max(line.lo - first, (int64_t)0), (int64_t)c.tiles);
        c.end = (int)min(max(line.hi - first, (int64_t)0), (int64_t)c.tiles);
        if (c.tile < c.end) return true;
        c.start += line.length(c.tiles);
        if (++c.u == units) {
            c.u = 0;
            if (++c.b >= a.B) return false;
            load_request(a, kept, c);
        }
    }
    return false;
}
template <typename Keys>
__device__ __forceinline__ bool next_unit(const Args& a, const Kept* kept, const Line<Keys>& line, Cursor<Keys>& c, int units) {
    c.start += line.length(c.tiles);
    if (++c.u == units) {
        c.u = 0;
        if (++c.b >= a.B) return false;
        load_request(a, kept, c);
    }
    return seek(a, kept, line, c, units);
}

// Lays out the line of the requests that read(b) gives and hands this warp its part of it; all threads of a block of W warps.
template <typename Keys, int W, typename F>
__device__ __forceinline__ Line<Keys> lay_line(const Args& a, LineBlock<W>& s, int units, F read) {
    static_assert(W * 32 >= kRuns && 2 * W <= 32, "a thread for each run, a lane for each record");
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    // places of the requests before each of kRuns runs of requests
    const int run = (a.B + kRuns - 1) / kRuns;
    {
        int64_t mine = 0;
        int most = 0;
        for (int b = tid * run; tid < kRuns && b < min(a.B, (tid + 1) * run); ++b) {
            const Request r = read(b);
            if (b < kKept) s.kept[b] = Kept{r.slot, r.len, r.plen};
            const int n = Keys::of(a, r).tiles();
            mine += Keys::kUnitCost + n;
            most = max(most, n);
        }
        int64_t incl = mine;
        for (int x = 1; x < 32; x <<= 1) {
            const int64_t o = __shfl_up_sync(0xffffffffu, incl, x);
            if (lane >= x) incl += o;
        }
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 31 && tid < kRuns) {
            s.sums[warp] = incl;
            s.longest[warp] = most;
        }
        if (tid < 2 * W) s.records[tid].valid = 0;
        __syncthreads();
        int64_t before = 0;
        for (int w = 0; w < warp && tid < kRuns; ++w) before += s.sums[w];
        __syncthreads();
        if (tid < kRuns) s.sums[tid + 1] = before + incl;
        if (tid == 0) s.sums[0] = 0;
        __syncthreads();
    }
    Line<Keys> line;
    line.each = 0;
    if ((int64_t)a.B * units <= gridDim.x) {
        int most = 0;
        for (int w = 0; w < kRuns / 32; ++w) most = max(most, s.longest[w]);
        if (most <= Keys::kShort) line.each = most;
    }
    const int64_t total = line.each ? (int64_t)a.B * units * line.each : s.sums[kRuns] * units;
    line.per = (total + gridDim.x - 1) / gridDim.x;
    if (line.each) line.per = line.each;
    else line.per = line.per < Keys::kLeast ? Keys::kLeast : line.per;
    const int64_t block_lo = min(total, line.per * blockIdx.x), block_hi = min(total, block_lo + line.per);
    line.lo = block_lo + (block_hi - block_lo) * warp / W;
    line.hi = block_lo + (block_hi - block_lo) * (warp + 1) / W;
    return line;
}

// The first unit of the warp's part; false if the part is empty.
template <typename Keys, int W>
__device__ __forceinline__ bool first_unit(const Args& a, const LineBlock<W>& sh, const Line<Keys>& line, Cursor<Keys>& c, int units) {
    if (line.lo >= line.hi) return false;
    if (line.each) {
        const int unit = (int)(line.lo / line.each);
        c.b = unit / units;
        c.u = unit % units;
        c.start = (int64_t)unit * line.each;
        load_request(a, sh.kept, c);
    } else {
        const int run = (a.B + kRuns - 1) / kRuns;
        int s = 0;                         // the run that holds place lo
        for (int step = kRuns / 2; step; step /= 2)
            if (sh.sums[s + step] * units <= line.lo) s += step;
        c.start = sh.sums[s] * units;
        c.b = s * run;
        load_request(a, sh.kept, c);
        while (line.lo - c.start >= (int64_t)line.length(c.tiles) * units && c.b + 1 < a.B) {
            c.start += (int64_t)line.length(c.tiles) * units;
            ++c.b;
            load_request(a, sh.kept, c);
        }
        c.u = min((int)((line.lo - c.start) / line.length(c.tiles)), units - 1);
        c.start += (int64_t)c.u * line.length(c.tiles);
    }
    return seek(a, sh.kept, line, c, units);
}

// Notes an open unit of this warp: its place in `records` by whether it began before.
template <typename Keys, int W>
__device__ __forceinline__ void note_open(LineBlock<W>& sh, const Line<Keys>& line, const Cursor<Keys>& c, bool open_start, bool open_end) {
    Record& rec = sh.records[2 * (threadIdx.x / 32) + (open_start ? 0 : 1)];
    rec.valid = 1;
    rec.b = c.b;
    rec.u = c.u;
    rec.tiles = c.tiles;
    rec.open_start = open_start;
    rec.open_end = open_end;
    rec.start = c.start + line.lead();
}

// Joins parts 0 .. count - 1 of one unit for one (row, four values): part(s)
// gives a part's base, O [R][D] then (m, l) [R].  N at a time, so that their
// loads are under way together.
template <int D, int R, int N, typename F>
__device__ __forceinline__ void join(int row, int col, int count, F part, float& m, float& l, float4& o) {
    for (int s0 = 0; s0 < count; s0 += N) {
        float2 ml[N];
        float4 v[N];
#pragma unroll
        for (int s = 0; s < N; ++s) {
            const float* p = part(min(s0 + s, count - 1));
            ml[s] = *reinterpret_cast<const float2*>(p + R * D + 2 * row);
            v[s] = *reinterpret_cast<const float4*>(p + row * D + col);
        }
        float top = m;
#pragma unroll
        for (int s = 0; s < N; ++s) {
            if (s0 + s >= count) ml[s] = make_float2(-INFINITY, 0.f);
            top = fmaxf(top, ml[s].x);
        }
        const float use = top == -INFINITY ? 0.f : top;
        float f = exp2_approx(m - use);
        l *= f;
        o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
#pragma unroll
        for (int s = 0; s < N; ++s) {
            if (s0 + s >= count) break;
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

// A row's joined sums become its result, or wait for the prefix's: row r of the
// group, four values.
template <int D>
__device__ __forceinline__ void finish(const Args& a, const DecodeBuffers& buf, int b, int hk, int r, int col, float m,
                                       float l, float4 o) {
    const int64_t at = (int64_t)b * a.Hq + hk * a.G + r;
    if (buf.with_prefix) {
        *reinterpret_cast<float4*>(buf.own + at * D + col) = o;
        if (col == 0) buf.own_ml[at] = make_float2(m, l);
        return;
    }
    const float inv = inverse(l);
    *reinterpret_cast<uint2*>(a.out + at * D + col) =
        make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
    if (a.weights && col == 0) buf.lse[at] = log_sum(m, l);
}

// Joins the open units of this block's warps, and those that it brings the last part
// of; all threads, after a barrier behind the last note_open.  local(k) is where the
// part of record k lies in shared memory.  Units are heads of a request in `chunks` of R rows.
template <int D, int R, typename Keys, int W, typename F>
__device__ __forceinline__ void join_open(const Args& a, const DecodeBuffers& buf, LineBlock<W>& sh, const Line<Keys>& line, int chunks, F local) {
    constexpr int kThreads = W * 32;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    // one after the other: `chain` lists the records in their order, a unit's follow one another
    unsigned valid = __ballot_sync(0xffffffffu, lane < 2 * W && sh.records[lane % (2 * W)].valid);
    if (warp == 0 && (valid >> lane & 1)) sh.chain[__popc(valid & ((1u << lane) - 1))] = lane;
    const int listed = __popc(valid);
    __syncthreads();
    for (int first = 0, next; first < listed; first = next) {
        next = first + 1;
        while (sh.records[sh.chain[next - 1]].open_end && next < listed) ++next;
        const Record& rec = sh.records[sh.chain[first]];
        const bool before = rec.open_start, after = sh.records[sh.chain[next - 1]].open_end;
        const int hk = rec.u / chunks, g0 = (rec.u - hk * chunks) * R;
        for (int i = tid; i < R * D / 4; i += kThreads) {
            const int r = i / (D / 4), col = (i % (D / 4)) * 4;
            float m = -INFINITY, l = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            join<D, R, Keys::kJoin>(r, col, next - first, [&](int j) { return local(sh.chain[first + j]); }, m, l, o);
            if (before || after) {
                float* part = buf.parts + (int64_t)(2 * blockIdx.x + (before ? 0 : 1)) * (R * D + 2 * R);
                *reinterpret_cast<float4*>(part + r * D + col) = o;
                if (col == 0) *reinterpret_cast<float2*>(part + R * D + 2 * r) = make_float2(m, l);
            } else if (g0 + r < a.G) {
                finish<D>(a, buf, rec.b, hk, g0 + r, col, m, l, o);
            }
        }
        if (before || after) {
            // the block that brings a unit's last part joins them all
            const int c0 = (int)(rec.start / line.per), c1 = (int)((rec.start + rec.tiles - 1) / line.per);
            __syncthreads();
            if (tid == 0) {
                // the ticket releases this block's part (written before the barrier) and acquires the others'
                unsigned* ticket = buf.tickets + c0 / 4;
                const int at = 8 * (c0 % 4);
                unsigned before_it;
                asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(before_it) : "l"(__cvta_generic_to_global(ticket)), "r"(1u << at) : "memory");
                sh.last_block = (int)(before_it >> at & 255u) == c1 - c0;
                if (sh.last_block) atomicAnd(ticket, ~(255u << at));
            }
            __syncthreads();
            if (sh.last_block) {
                for (int i = tid; i < R * D / 4; i += kThreads) {
                    const int r = i / (D / 4), col = (i % (D / 4)) * 4;
                    float m = -INFINITY, l = 0.f;
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                    join<D, R, Keys::kJoin>(r, col, c1 - c0 + 1,
                               [&](int s) { return buf.parts + (int64_t)(2 * (c0 + s) + (s ? 0 : 1)) * (R * D + 2 * R); }, m, l, o);
                    if (g0 + r < a.G) finish<D>(a, buf, rec.b, hk, g0 + r, col, m, l, o);
                }
            }
            __syncthreads();
        }
    }
}

}  // namespace attn
}  // namespace bd
