// bd_attn4_decode.cu -- attention of one query row a request on its own keys in the
// 4-bit cache.
//
// o = sum_j p_j v_j with p the softmax of q.k_j, k and v what the cache stands for:
// 4 head_dim flops a head and key for 17/16 head_dim bytes, so the cache's bytes bound
// it, and next to them the instructions that make f16 of 4 bits.  The line of units,
// the blocks' and warps' parts of it and their joining are those of the bf16 cache's
// decode kernel; tiles are three cache blocks, 48 keys, and begin where a block
// begins.  A warp streams its tiles, bytes as they lie, through a ring of its own (cp.async) and
// multiplies the transposed way, S^T = K Q^T and O^T = V^T P^T, with mma.m16n8k16 in f16:
// keys and dims are the 16 rows and a group's heads the 8 columns, so a group of 8 wastes nothing.  Which
// dims meet in a product's step is free, so the cache's words are laid out for the
// lanes: 16 bytes a lane are its part of a key, and a word is two steps' operand after
// nine operations (bd_cache4.cuh).  Numbers times scales are exact in f16, and so is a
// query, which a power of two of its own brings to f16's range (but values below 2^-30 of
// its largest one); the probabilities are rounded to 11 significant bits, less than the result to bf16.
// P^T comes out of S^T's layout by one 8 x 8 transposition in registers.
// What bounds it: those nine operations a word, logical ones and f16 fmas, each issued in two
// cycles and hardly beside one another.  4 requests of 90,001 to 131,072 keys (481 MB) 85 us
// = 5.7 TB/s, 84% of a copy's rate (the bf16 cache's kernel 266 us); 128 requests of 1 to
// 16,384 keys seeing 4 + 4096 of them 93 us; one of 300 keys 6.8 us.
// When the first of these took 87 us, the same loads without the arithmetic took 77 us and
// the arithmetic without the loads 82.  Other forms of it, on the same case: 8 warps with tiles of 64 keys 89,
// 16 with 32 (more do not fit) 89; one path with masks for all tiles, where those whose keys
// are all seen have their own, 91; bulk copies with barriers in place of cp.async 93; sums of
// q s, q = n + 8, that lose 8 s p and 8 s q at their end, so that the fma reads two registers and not three,
// 86, for a bound on the error that grows with q's 15 in place of n's 7: not taken.
// Requests of few rows of a prompt call come here too, each row with the keys up to its own (bd_attn4.cu).
#include <math.h>

#include <type_traits>

#include "bd_attn_line.cuh"
#include "bd_attn4.cuh"
#include "bd_cache4.cuh"
#include "bd_tc_common.cuh"

namespace bd {
namespace attn {
namespace {

using cache4::Cache;
using cache4::kBlock;
using cache4::Layout;
using cache4::Scales;

// The running maximum is kept this many powers of two below the scores' (so the largest probability is 2^6 at
// least, and others keep f16's bits down to 2^-20 of it), and moves only once a probability exceeds 2^14.
constexpr float kLift = 6.f;
// What it begins with: below any score's but -inf, so that one that is -inf weighs nothing even where no other has been
// seen (with -inf in this place it would be a NaN).
constexpr float kLowest = -3.402823466e38f;

// Looks at every request of a prompt call, those without rows too, and reports what is wrong with them; the number of
// requests before the first whose offsets do not ascend.  All threads of a block.
__device__ __forceinline__ int served_requests(const Args& a, int& served) {
    if (threadIdx.x == 0) served = a.R;
    __syncthreads();
    for (int b = threadIdx.x; b < a.R; b += blockDim.x) {
        const int lo = a.cu_q[b], hi = a.cu_q[b + 1];
        if (lo < 0 || hi < lo || hi > a.T) atomicMin(&served, b);
        read_request(a, b);
    }
    __syncthreads();
    return served;
}

// A row of a prompt call as a request of its own, with the keys up to its own; a row of no request, or of one that the
// tiles take, has length -1.  The requests from `served` on are not served: rows from there on have no keys.
__device__ __forceinline__ Request row_request(const Args& a, int served, int row) {
    Request r{};
    r.len = -1;
    int n = 0;                                          // requests that begin at the row or before it
    for (int end = served; n < end;) {
        const int mid = (n + end) / 2;
        if (a.cu_q[mid] <= row) n = mid + 1;
        else end = mid;
    }
    if (n > 0 && row < a.cu_q[n]) {
        const int b = n - 1, hi = a.cu_q[n], slot = a.slots ? a.slots[b] : b, len = a.lens[b];
        const int rows = hi - a.cu_q[b];
        if (a.few && rows > a.few) return r;            // the tiles'
        const bool ok = slot >= 0 && slot < a.n_slots && len >= rows && len <= a.longest;
        r.slot = ok ? slot : 0;
        r.len = ok ? len - (hi - 1 - row) : 0;
    } else if (served < a.R && row >= a.cu_q[served]) {
        r.len = 0;                                      // zeros
    }
    return r;
}

// Where the visible keys of a request lie: tiles from the first key on (`head` of them)
// and, behind a gap, those from tile `from` on.
// Measured on both sides: kUnitCost 1 / 2 / 4 on 128 windowed requests 96.8 / 94.1 / 96.3 us; kLeast 8 / 16 / 32 on one
// request of 4000 keys 12.7 / 15.5 / 16.8; kShort 12 / 30 / 64 on 4 requests of 600 to 1200 keys 13.7 / 11.4 / 11.4, on 8
// of 500 to 3000 15.3 / 15.2 / 17.9; kJoin 2 / 4 / 8 on 2 requests of 4000 to 8000 keys with 32
// query heads on 2 17.3 / 22.3 / 23.1 (more instructions, fetched for this alone), 1 and 2 alike.
// ROWS: the requests are the rows of a prompt call.
template <int BLOCKS, bool ROWS>
struct Keys4 {
    static constexpr int kTile = BLOCKS * kBlock;                           // keys of a tile
    static constexpr int kUnitCost = 2, kLeast = 8, kShort = 30, kJoin = 2;
    int len, lo, sinks, head, from, n;
    static constexpr bool kAllKept = ROWS;
    static __device__ __forceinline__ Keys4 of(const Args& a, const Request& r) {
        Keys4 k;
        k.len = r.len;
        k.lo = min(max(window_lo(a, r.plen + r.len - 1) - r.plen, 0), r.len);
        k.sinks = min(max(a.sinks - r.plen, 0), r.len);
        k.head = (k.sinks + kTile - 1) / kTile;
        k.from = k.lo / kTile;
        if (k.from <= k.head) k.head = k.from = 0;
        k.n = k.head + (r.len + kTile - 1) / kTile - k.from;
        return k;
    }
    __device__ __forceinline__ int tiles() const { return max(1, n); }
    // first key of a tile
    __device__ __forceinline__ int base(int tile) const { return (tile < head ? tile : tile - head + from) * kTile; }
    __device__ __forceinline__ bool sees(int key) const { return key < len && (key >= lo || key < sinks); }
    __device__ __forceinline__ bool whole(int base) const { return base + kTile <= len && (base >= lo || base + kTile <= sinks); }
};

template <int D, int R>
struct Shape4 {
    static constexpr int kWarps = R == 8 ? 12 : 8;
    static constexpr int kBlocks = 3;                          // cache blocks of a tile
    static constexpr int kStage = kBlocks * Layout<D>::kBytes;
    static constexpr int kStages = 2 * (128 / D);
    static constexpr int kRing = kStage * kStages;                          // of one warp
    static constexpr int kPart = R * D * 4 + R * 8;                         // an open unit: O, then (m, l)
    static constexpr int kSmem = kWarps * (kRing + kPart);
    static_assert(kRing >= kPart, "a warp's last open unit reuses its ring");
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// An 8 x 8 matrix of 16-bit values across the warp, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// The larger ones of two pairs (a NaN is never larger).
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Whether one of a pair exceeds 2^14.
__device__ __forceinline__ bool over(uint32_t a) {
    uint32_t r;
    asm("set.gt.u32.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(0x74007400u));
    return r != 0;
}

// W words at a time from shared memory.
template <int W>
__device__ __forceinline__ void load_words(uint32_t (&w)[W], const uint8_t* at) {
    if constexpr (W == 4) {
        const uint4 x = *reinterpret_cast<const uint4*>(at);
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    } else {
        const uint2 x = *reinterpret_cast<const uint2*>(at);
        w[0] = x.x, w[1] = x.y;
    }
}

// A tile's bytes as they lie, from its unit's first block; of a request's last one only blocks that
// hold keys.  (lane * 16 is in both addresses.)
template <int D, typename Keys>
__device__ __forceinline__ void load_tile4(const uint8_t* unit, const Keys& k, int tile, uint32_t to) {
    constexpr int kChunks = Keys::kTile / kBlock * Layout<D>::kBytes / 16;
    const int lane = threadIdx.x % 32, base = k.base(tile);
    const uint8_t* from = unit + (int64_t)base * (Layout<D>::kBytes / kBlock);
    auto copy = [&](int i) { asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(to + i * 512), "l"(from + i * 512) : "memory"); };
    if (base + Keys::kTile - kBlock < k.len) {
#pragma unroll
        for (int i = 0; i < kChunks / 32; ++i) copy(i);
        if (kChunks % 32 && lane < kChunks % 32) copy(kChunks / 32);
    } else {
        const int n = (k.len - base + kBlock - 1) / kBlock * (Layout<D>::kBytes / 16);
#pragma unroll 1
        for (int i = 0; lane + i * 32 < n; ++i) copy(i);
    }
}

template <int D, int R, bool ROWS>
__global__ void __launch_bounds__(Shape4<D, R>::kWarps * 32, 1)
    decode4_kernel(const Args a, const Cache cache, const DecodeBuffers buf) {
    using S = Shape4<D, R>;
    using Lay = Layout<D>;
    constexpr int NT = R / 8;              // columns of eight heads
    constexpr int kBlocks = S::kBlocks;
    using Keys = Keys4<kBlocks, ROWS>;
    constexpr int W = D / 32;              // words of a lane's part of a key, or of two values
    constexpr int MT = D / 16;             // sixteens of dims
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ LineBlock<S::kWarps> sh;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int chunks = (a.G + R - 1) / R;  // a group of more than 16 heads is read once a 16
    const int units = a.Hk * chunks;

    grid_wait();
    if (ROWS && a.few) grid_go_on();       // the tiles' plan is laid out and their keys are read beside this
    int served = a.B;
    if constexpr (ROWS) {
        __shared__ int least;
        served = served_requests(a, least);
    }
    const Line<Keys> line = lay_line<Keys>(a, sh, units, [&](int b) {
        if constexpr (ROWS) return row_request(a, served, b);
        else return read_request<true>(a, b);
    });
    uint8_t* const ring = smem + warp * S::kRing;
    float* const tail_part = reinterpret_cast<float*>(ring);
    float* const head_part = reinterpret_cast<float*>(smem + S::kWarps * S::kRing + warp * S::kPart);
    const cache4::Ones ones;

    Cursor<Keys> c;
    if (first_unit(a, sh, line, c, units)) {
        Cursor<Keys> ahead = c;
        bool more = true;
        int put = 0;
        const uint32_t ring_at = smem_addr(ring) + lane * 16;
        const uint8_t* unit;
        auto enter = [&]() { unit = cache.data + ahead.r.slot * cache.ss + ahead.u / chunks * cache.sh + lane * 16; };
        enter();
        auto prefetch = [&]() {
            if (more) {
                load_tile4<D>(unit, ahead.k, ahead.tile, ring_at + put * S::kStage);
                if (++ahead.tile == ahead.end) {
                    more = next_unit(a, sh.kept, line, ahead, units);
                    enter();
                }
            }
            cp_async_commit();
            if (++put == S::kStages) put = 0;
        };
#pragma unroll 1
        for (int i = 0; i < S::kStages - 1; ++i) prefetch();

        int got = 0;
        const int g = lane / 4, t = lane % 4;
        uint32_t qf[NT][2 * W][2];         // of head 8 n + g: the lane's dims of each step
        float factor[NT][2];               // scores in powers of two: of heads 8 n + 2 t, + 1
        float o[NT][MT][4], l[NT][4], m[NT][2];
        // One tile; of one that is not WHOLE some keys are not seen.
        auto tile = [&](auto whole, const uint8_t* stage, int base) {
            constexpr bool WHOLE = decltype(whole)::value;
            float s[kBlocks][NT][4];
#pragma unroll
            for (int x = 0; x < kBlocks; ++x) {
                const uint8_t* at = stage + x * Lay::kBytes;
                uint32_t ka[W], kb[W];                 // keys g and g + 8
                load_words(ka, at + g * (D / 2) + t * (4 * W));
                load_words(kb, at + (g + 8) * (D / 2) + t * (4 * W));
                const uint8_t* code = at + Lay::kScaleK + g * (D / 32) + t * (D / 32) / 4;
                const Scales sa = cache4::scale_of(code[0]), sb = cache4::scale_of(code[8 * (D / 32)]);
#pragma unroll
                for (int n = 0; n < NT; ++n) s[x][n][0] = s[x][n][1] = s[x][n][2] = s[x][n][3] = 0.f;
#pragma unroll
                for (int i = 0; i < 2 * W; ++i) {
                    const uint32_t wa = i % 2 ? cache4::swap_bytes(ka[i / 2]) : ka[i / 2], wb = i % 2 ? cache4::swap_bytes(kb[i / 2]) : kb[i / 2];
                    const uint32_t a0 = cache4::field0(wa, sa, ones), a1 = cache4::field0(wb, sb, ones);
                    const uint32_t a2 = cache4::field1(wa, sa, ones), a3 = cache4::field1(wb, sb, ones);
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma_f16(s[x][n], a0, a1, a2, a3, qf[n][i][0], qf[n][i][1]);
                }
            }
            bool seen[kBlocks][2], two[kBlocks][4];    // keys g, g + 8; keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9
#pragma unroll
            for (int x = 0; x < kBlocks; ++x) {
#pragma unroll
                for (int i = 0; i < 2; ++i) seen[x][i] = WHOLE || c.k.sees(base + x * kBlock + g + 8 * i);
#pragma unroll
                for (int i = 0; i < 4; ++i) two[x][i] = WHOLE || c.k.sees(base + x * kBlock + 2 * t + i % 2 + i / 2 * 8);
            }
            uint32_t p[kBlocks][NT][2];
            auto weigh = [&]() {
                uint32_t top = 0;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int x = 0; x < kBlocks; ++x)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float p0 = exp2_approx(fmaf(s[x][n][2 * i], factor[n][0], -m[n][0]));
                            const float p1 = exp2_approx(fmaf(s[x][n][2 * i + 1], factor[n][1], -m[n][1]));
                            p[x][n][i] = seen[x][i] ? pack_f16(p0, p1) : 0u;
                            top = max2(top, p[x][n][i]);
                        }
                return __any_sync(0xffffffffu, over(top));
            };
            if (weigh()) {
                // the maximum moves (from the lowest, at first)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float f[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float top = -INFINITY;
#pragma unroll
                        for (int x = 0; x < kBlocks; ++x)
#pragma unroll
                            for (int y = 0; y < 2; ++y)
                                if (seen[x][y]) top = fmaxf(top, s[x][n][2 * y + i] * factor[n][i]);
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16)) - kLift;
                        f[i] = top > m[n][i] ? exp2_approx(m[n][i] - top) : 1.f;
                        m[n][i] = fmaxf(m[n][i], top);
                    }
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        o[n][i][0] *= f[0];
                        o[n][i][1] *= f[1];
                        o[n][i][2] *= f[0];
                        o[n][i][3] *= f[1];
                    }
                    l[n][0] *= f[0];
                    l[n][1] *= f[1];
                    l[n][2] *= f[0];
                    l[n][3] *= f[1];
                }
                weigh();
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int x = 0; x < kBlocks; ++x)
#pragma unroll
                    for (int i = 0; i < 2; ++i) p[x][n][i] = transpose8(p[x][n][i]);
#pragma unroll
            for (int x = 0; x < kBlocks; ++x) {
                const uint8_t* at = stage + x * Lay::kBytes;
                uint32_t va[W], vb[W];                 // of keys 2 t, 2 t + 1 and of 2 t + 8, 2 t + 9
                load_words(va, at + Lay::kV + t * D + g * (4 * W));
                load_words(vb, at + Lay::kV + (t + 4) * D + g * (4 * W));
                const uint16_t* code = reinterpret_cast<const uint16_t*>(at + Lay::kScaleV + g * (D / 32) / 8 * kBlock + 2 * t);
                uint32_t pa = cache4::scale_pair(code[0]), pb = cache4::scale_pair(code[4]);
                if constexpr (!WHOLE) {
                    // values that are not seen become zeros, whatever they are
                    pa &= (two[x][0] ? 0xFFFFu : 0u) | (two[x][1] ? 0xFFFF0000u : 0u);
                    pb &= (two[x][2] ? 0xFFFFu : 0u) | (two[x][3] ? 0xFFFF0000u : 0u);
                }
                const Scales sa = cache4::scales(pa), sb = cache4::scales(pb);
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const uint32_t wa = i % 2 ? cache4::swap_bytes(va[i / 2]) : va[i / 2], wb = i % 2 ? cache4::swap_bytes(vb[i / 2]) : vb[i / 2];
                    const uint32_t a0 = cache4::field0(wa, sa, ones), a1 = cache4::field1(wa, sa, ones);
                    const uint32_t a2 = cache4::field0(wb, sb, ones), a3 = cache4::field1(wb, sb, ones);
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma_f16(o[n][i], a0, a1, a2, a3, p[x][n][0], p[x][n][1]);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_f16(l[n], 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, p[x][n][0], p[x][n][1]);
            }
        };
        do {
            const int seg_tile = c.tile;
            const int hk = c.u / chunks, g0 = (c.u % chunks) * R;
            {
                const __nv_bfloat16* qp = a.q + (int64_t)c.b * a.q_stride + (int64_t)(hk * a.G + g0) * D + t * (D / 4);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    uint32_t w[4 * W];
#pragma unroll
                    for (int i = 0; i < W; ++i) {
                        const uint4 x = 8 * n + g < a.G - g0 ? *reinterpret_cast<const uint4*>(qp + (8 * n + g) * D + i * 8) : make_uint4(0u, 0u, 0u, 0u);
                        w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
                    }
                    // the largest magnitude's power of two goes to 2^13; a row that is not finite stays as it is
                    uint32_t top = 0;
#pragma unroll
                    for (int i = 0; i < 4 * W; ++i) top = max(top, max(w[i] & 0x7FFFu, w[i] >> 16 & 0x7FFFu));
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    const uint32_t e = top >= 0x7F80u ? 140u : max(top >> 7, 14u);
                    const float by = __uint_as_float((267u - e) << 23), back = __uint_as_float((e - 13u) << 23);
#pragma unroll
                    for (int i = 0; i < 4 * W; ++i) qf[n][i / 2][i % 2] = pack_f16(bf16_lo(w[i]) * by, bf16_hi(w[i]) * by);
                    factor[n][0] = a.scale_log2 * __shfl_sync(0xffffffffu, back, 8 * t);
                    factor[n][1] = a.scale_log2 * __shfl_sync(0xffffffffu, back, 8 * t + 4);
#pragma unroll
                    for (int i = 0; i < MT; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
                    l[n][0] = l[n][1] = l[n][2] = l[n][3] = 0.f;
                    m[n][0] = m[n][1] = kLowest;
                }
            }
#pragma unroll 1
            for (; c.tile < c.end; ++c.tile) {
                prefetch();
                cp_async_wait<S::kStages - 1>();
                __syncwarp();
                const uint8_t* const stage = ring + got * S::kStage;
                if (++got == S::kStages) got = 0;
                const int base = c.k.base(c.tile);
                if (c.k.whole(base)) tile(std::true_type(), stage, base);
                else tile(std::false_type(), stage, base);
                __syncwarp();
            }
            // the unit, or this warp's part of it, is done; the lane has dims D / 8 g ... of heads 8 n + 2 t, + 1
            const bool open_start = seg_tile > 0, open_end = c.end < c.tiles;
            if (open_start || open_end) {
                // one that began before is kept beside the ring, the last one (no
                // tile follows it) in the ring
                if (!open_start) cp_async_wait<0>();
                __syncwarp();
                float* part = open_start ? head_part : tail_part;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int r = 8 * n + 2 * t + i;
#pragma unroll
                        for (int w = 0; w < W; ++w)
                            *reinterpret_cast<float4*>(part + r * D + g * (D / 8) + 4 * w) =
                                make_float4(o[n][2 * w][i], o[n][2 * w][2 + i], o[n][2 * w + 1][i], o[n][2 * w + 1][2 + i]);
                        if (g == 0) *reinterpret_cast<float2*>(part + R * D + 2 * r) = make_float2(m[n][i], l[n][i]);
                    }
                if (lane == 0) note_open(sh, line, c, open_start, open_end);
            } else if (!ROWS || c.k.len >= 0) {            // (a row of no request is one tile, whole: it ends here)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int r = g0 + 8 * n + 2 * t + i;
                        if (r >= a.G) continue;
#pragma unroll
                        for (int w = 0; w < W; ++w)
                            finish<D>(a, buf, c.b, hk, r, g * (D / 8) + 4 * w, m[n][i], l[n][i],
                                      make_float4(o[n][2 * w][i], o[n][2 * w][2 + i], o[n][2 * w + 1][i], o[n][2 * w + 1][2 + i]));
                    }
            }
        } while (next_unit(a, sh.kept, line, c, units));
        cp_async_wait<0>();
    }
    __syncthreads();

    join_open<D, R>(a, buf, sh, line, chunks, [&](int k) {
        return reinterpret_cast<const float*>(smem + (k % 2 ? k / 2 * S::kRing : S::kWarps * S::kRing + k / 2 * S::kPart));
    });
}

template <int D, int R, bool ROWS>
bd_status launch_shape4(const Args& a, const Cache& cache, const DecodeBuffers& buf, cudaStream_t stream) {
    using S = Shape4<D, R>;
    const void* kernel = reinterpret_cast<const void*>(decode4_kernel<D, R, ROWS>);
    if (!set_smem_attr(kernel, S::kSmem, 11 + (D == 64) * 2 + (R == 16) + ROWS * 4)) return BD_ERR_CUDA;
    // (a launch that is set up while the kernel before it ends: 3 us less of calls that follow one another)
    return launch_close(decode4_kernel<D, R, ROWS>, decode_blocks(), S::kWarps * 32, S::kSmem, stream, a, cache, buf);
}

}  // namespace

namespace {
template <bool ROWS>
bd_status launch_rows(const Args& a, const cache4::Cache& cache, int head_dim, const DecodeBuffers& buf, cudaStream_t stream) {
    if (a.G <= 8) return head_dim == 128 ? launch_shape4<128, 8, ROWS>(a, cache, buf, stream) : launch_shape4<64, 8, ROWS>(a, cache, buf, stream);
    return head_dim == 128 ? launch_shape4<128, 16, ROWS>(a, cache, buf, stream) : launch_shape4<64, 16, ROWS>(a, cache, buf, stream);
}
}  // namespace

bd_status launch_decode4(const Args& a, const cache4::Cache& cache, int head_dim, const DecodeBuffers& buf, cudaStream_t stream) {
    return a.cu_q ? launch_rows<true>(a, cache, head_dim, buf, stream) : launch_rows<false>(a, cache, head_dim, buf, stream);
}

}  // namespace attn
}  // namespace bd
