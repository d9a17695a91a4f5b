// bd_cache4.cu -- rows of keys and values into the 4-bit cache and out of it.
//
// Both directions move 4 bytes of bf16 for 17/16 of a byte of cache and do a few
// operations a value, so the bytes bound them.  A warp takes a block (16 tokens of one
// head, K and V) at a time: a row's D values lie on D / 8 lanes, 16 bytes each, so a
// group's largest value is two shuffles away and a lane's eight numbers are one word of K.  A
// word of V holds four dims of two tokens; the lanes of the two swap halves, so that
// whole words are written wherever both tokens are.
// Measured (8 heads of 128): 131,080 tokens of 16 requests written in 125 us and read in 117, 680 MB
// each way = 5.4 and 5.8 TB/s, 81% and 86% of a copy's rate; prompts of 9,525 tokens 13.6 and 10.9 us (7.3 for the bytes),
// one token 3.6 and 3.2, most of it lengths and slots, then rows, that wait for one another.  Writing is bound by its
// instructions: without a path for whole halves of a block, which needs no predicates, it took 159.
#include <math.h>

#include <type_traits>

#include "bd_attn_math.cuh"
#include "bd_cache4.cuh"
#include "bd_cache4_host.cuh"

namespace bd {
namespace cache4 {
namespace {

using attn::Args;
using attn::Request;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// The rows' side: bf16, heads of a row one after the other.
struct Rows {
    __nv_bfloat16 *k, *v;
    int64_t k_stride, v_stride;
};

// The attention's scratch for prompts: keys in their places, [B, kv_heads, length, D] bf16.
struct Scratch {
    __nv_bfloat16 *k, *v;
    int64_t length;
};

// Which blocks of a request a call touches: `head` from the first on, and those from
// block `from` to its end; of them the tokens [first, len).
struct Span {
    int first, len, row0, head, from, n;
};

__device__ __forceinline__ Span rows_span(const Request& r) {
    Span s;
    s.first = r.len - r.rows;
    s.len = r.len;
    s.row0 = r.row0;
    s.head = 0;
    s.from = s.first / kBlock;
    s.n = (r.len + kBlock - 1) / kBlock - s.from;
    return s;
}

// What the queries of a prompt see: all but what lies before the first one's window and
// behind the first tokens.
__device__ __forceinline__ Span seen_span(const Args& a, const Request& r) {
    Span s;
    const int lo = attn::window_lo(a, r.len - r.rows), sinks = min(a.sinks, r.len);
    s.first = 0;
    s.len = r.len;
    s.row0 = 0;
    s.head = (sinks + kBlock - 1) / kBlock;
    s.from = lo / kBlock;
    if (s.from <= s.head) s.head = s.from = 0;
    s.n = s.head + (r.len + kBlock - 1) / kBlock - s.from;
    return s;
}

// Blocks of the requests before each thread's run of requests; of a call of no more requests
// than threads the requests themselves.
struct Items {
    int64_t before[kThreads + 1];
    int64_t warp[kWarps];
    Span span[kThreads];
    int slot[kThreads];
    int served;
};

// Request b as this call sees it; false if nothing of it is touched.
template <bool SCRATCH>
__device__ __forceinline__ bool span_of(const Args& a, int b, int served, Span& s) {
    if (b >= served) return false;
    const Request r = attn::read_request(a, b);
    if (r.rows == 0) return false;
    if (r.len < r.rows) {   // (one that is out of range has no length)
        report(a.status, BD_ERR_SLOT);
        return false;
    }
    s = SCRATCH ? seen_span(a, r) : rows_span(r);
    return true;
}

template <bool SCRATCH>
__device__ __forceinline__ int64_t lay_items(const Args& a, Items& items) {
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int run = (a.B + kThreads - 1) / kThreads;
    if (tid == 0) items.served = a.B;
    Span one;
    bool in_one = false;                        // what a call of few requests reads in one go
    __syncthreads();
    for (int b = tid * run; b < min(a.B, (tid + 1) * run); ++b) {
        if (a.cu_q) {
            // requests from the first whose offsets do not ascend on are not served
            const int lo = a.cu_q[b], hi = a.cu_q[b + 1];
            if (lo < 0 || hi < lo || hi > a.T) {
                atomicMin(&items.served, b);
                report(a.status, BD_ERR_SLOT);
                break;
            }
        }
        if (run == 1) in_one = span_of<SCRATCH>(a, b, a.B, one);
    }
    __syncthreads();
    const int served = items.served;
    int64_t mine = 0;
    for (int b = tid * run; b < min(a.B, (tid + 1) * run); ++b) {
        Span s = one;
        const bool in = run == 1 ? in_one && b < served : span_of<SCRATCH>(a, b, served, s);
        if (in) mine += s.n;
        if (run == 1) {
            items.span[b] = s;
            items.slot[b] = a.slots ? a.slots[b] : b;
        }
    }
    int64_t incl = mine;
    for (int x = 1; x < 32; x <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, incl, x);
        if (lane >= x) incl += o;
    }
    if (lane == 31) items.warp[warp] = incl;
    __syncthreads();
    int64_t before = 0;
    for (int w = 0; w < warp; ++w) before += items.warp[w];
    items.before[tid + 1] = before + incl;
    if (tid == 0) items.before[0] = 0;
    __syncthreads();
    return items.before[kThreads];
}

// The request that holds block i of all, which becomes the block's number within it, and its slot.  (Of more requests than
// threads a thread's run is walked again for every block: one token of each of 256, 512, 1024, 2048 and 8192 requests is
// written in 4.3, 6.6, 11.5, 22 and 149 us.)
template <bool SCRATCH>
__device__ __forceinline__ int find(const Args& a, const Items& items, int64_t& i, Span& s, int& slot) {
    int t = 0;
    for (int step = kThreads / 2; step; step /= 2)
        if (items.before[t + step] <= i) t += step;
    i -= items.before[t];
    const int run = (a.B + kThreads - 1) / kThreads;
    if (run == 1) {
        s = items.span[t];
        slot = items.slot[t];
        return t;
    }
    for (int b = t * run;; ++b) {
        if (!span_of<SCRATCH>(a, b, items.served, s)) continue;
        if (i < s.n) {
            slot = a.slots ? a.slots[b] : b;
            return b;
        }
        i -= s.n;
    }
}

// ---- values into numbers ---------------------------------------------------------------

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The bits of the largest |x| (bf16) of a group of keys, and of values in the upper half; a
// group's 32 values lie on four lanes.
__device__ __forceinline__ uint32_t largest(const uint4& k, const uint4& v) {
    auto four = [](const uint4& x) {
        return max_u16x2(max_u16x2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu), max_u16x2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
    };
    const uint32_t a = four(k), b = four(v);
    uint32_t m = max_u16x2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
    m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    return max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, 2));
}

// A group's scale as its byte, from the bits of the largest |x| (bf16).  The quotient by 7 is a product with
// 1 / 7, off by 2^-23 of itself, rounded to 12 bits, which a tie between two scales (5 bits; 7 times it has 8) is
// itself and other quotients are 2^-9 or more from, and then to the scale's 4, ties to even.
__device__ __forceinline__ uint32_t scale_code(uint32_t top) {
    if (top >= 0x7F80u) return kNanScale;
    const uint32_t bits = (__float_as_uint(__uint_as_float(top << 16) * (1.f / 7.f)) + 0x400u) & ~0x7FFu;
    if (bits < 0x38800000u) return (uint32_t)__float2int_rn(__uint_as_float(bits) * 131072.f);      // below 2^-14: units of 2^-17
    return min(((bits + 0x7FFFFu + (bits >> 20 & 1u)) >> 20) - (112u << 3), kTopScale);
}

__device__ __forceinline__ float scale_value(uint32_t code) { return __half2float(__ushort_as_half((unsigned short)(code << 7))); }

// 1 / s, off by 2^-23 of itself; 0 for 0.
__device__ __forceinline__ float inverse_scale(uint32_t code) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(scale_value(code)));
    return code ? r : 0.f;
}

// Eight values as n + 8, two fields of a unit each: (n0 + 8) 2^6 + (n1 + 8) 2^2 in the low bits.  x / s is a product with 1 /
// s, off by 2^-23 of itself, to the nearest multiple of 2^-10 (that many of 1.5 2^13's last places), which
// a tie x = (n + 1/2) s is itself, and then to whole numbers.  Other x lie 2^-9 or more from a tie (8 bits of
// x against 4 of s), so this is the exact quotient's rounding, ties to even.  Only quotients by the largest scale, and by
// those below 2^-14, which have fewer bits, can lie outside [-7.5, 7.5].
// (All in f32, at twice the rate of shifts and of minima; prompts of 9,525 tokens 21.4 -> 18.2 us, with the scales found once.)
__device__ __forceinline__ void fields(const uint4& x, uint32_t code, float inv, uint32_t (&pairs)[4], const int (&order)[8]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = i % 2 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
    if (code >= kTopScale || code < 8) {
        const float s = scale_value(code);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = fminf(fmaxf(y[i], -7.f * s), 7.f * s);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = (fmaf(y[i], inv, 12288.f) + 12570632.f) - 12582912.f;     // 1.5 2^23 - 12288 + 8
#pragma unroll
    for (int i = 0; i < 4; ++i) pairs[i] = __float_as_uint(fmaf(y[order[2 * i]], 64.f, fmaf(y[order[2 * i + 1]], 4.f, 8388608.f)));
}

// A word of two units: their first two fields, and the other two with swapped bytes.
__device__ __forceinline__ uint32_t word_of(uint32_t first0, uint32_t last0, uint32_t first1, uint32_t last1) {
    return __byte_perm(first0, first1, 0x5410) | __byte_perm(last0, last1, 0x4501);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 4) write_kernel(const Args a, const Cache c, const Rows rows) {
    using Lay = Layout<D>;
    constexpr int L = D / 8;                    // lanes of a row
    constexpr int R = 32 / L;                   // rows of a step
    constexpr int kHalf = kBlock / R / 2;       // steps of half a block
    __shared__ Items items;
    __shared__ __align__(4) uint8_t codes[kWarps][D];
    const int tid = threadIdx.x, lane = tid % 32, col = lane % L;
    attn::grid_wait();
    const int64_t total = lay_items<false>(a, items) * a.Hk;
    for (int64_t at = (int64_t)blockIdx.x * kWarps + tid / 32; at < total; at += (int64_t)gridDim.x * kWarps) {
        int64_t i = at / a.Hk;
        const int h = (int)(at - i * a.Hk);
        Span s;
        int slot;
        find<false>(a, items, i, s, slot);
        const int block = s.from + (int)i, t0 = block * kBlock;
        uint8_t* const to = c.data + slot * c.ss + h * c.sh + (int64_t)block * Lay::kBytes;
        const int lo = max(s.first - t0, 0), hi = min(s.len - t0, kBlock);      // tokens of the block
        const int64_t row0 = (int64_t)s.row0 - s.first + t0;
        const int row = lane / L;
        // a row may hold 2^31 values and more (2^32 times eight of them, and a block of each of its heads, no GPU)
        const unsigned eights = (unsigned)h * L + col;
        const __nv_bfloat16* k_from = rows.k + (row0 + row) * rows.k_stride + (uint64_t)eights * 8;
        const __nv_bfloat16* v_from = rows.v + (row0 + row) * rows.v_stride + (uint64_t)eights * 8;
        uint8_t* const k_to = to + row * (D / 2) + col * 4;
        uint8_t* const v_to = to + Lay::kV + row / 2 * D + col * 8;
        uint8_t* const code_to = codes[tid / 32] + (col % 4 ? 0 : row * (D / 32) + col / 4);
        // half a block from step u0 on; of one that is not WHOLE some tokens are none of the call's
        auto half = [&](auto all, int u0) {
            constexpr bool WHOLE = decltype(all)::value;
            uint4 k[kHalf], v[kHalf];
#pragma unroll
            for (int u = 0; u < kHalf; ++u) {
                const int j = (u0 + u) * R + row;
                if (!WHOLE) k[u] = v[u] = make_uint4(0u, 0u, 0u, 0u);
                if (!WHOLE && (j < lo || j >= hi)) continue;
                k[u] = *reinterpret_cast<const uint4*>(k_from + (u0 + u) * R * rows.k_stride);
                v[u] = *reinterpret_cast<const uint4*>(v_from + (u0 + u) * R * rows.v_stride);
            }
#pragma unroll
            for (int u = 0; u < kHalf; ++u) {
                if (!WHOLE && ((u0 + u + 1) * R <= lo || (u0 + u) * R >= hi)) continue;
                const int j = (u0 + u) * R + row;
                // a group's even lanes find the keys' scale, its odd ones the values'
                const uint32_t top = largest(k[u], v[u]), code = scale_code(lane % 2 ? top >> 16 : top & 0xFFFFu);
                const float inv = inverse_scale(code);
                const uint32_t code_k = __shfl_sync(0xffffffffu, code, lane & ~1), code_v = __shfl_sync(0xffffffffu, code, lane | 1);
                const float inv_k = __shfl_sync(0xffffffffu, inv, lane & ~1), inv_v = __shfl_sync(0xffffffffu, inv, lane | 1);
                const bool in = WHOLE || (j >= lo && j < hi), other = WHOLE || ((j ^ 1) >= lo && (j ^ 1) < hi);
                uint32_t n[4];
                constexpr int by_twos[8] = {0, 2, 4, 6, 1, 3, 5, 7}, in_order[8] = {0, 1, 2, 3, 4, 5, 6, 7};
                fields(k[u], code_k, inv_k, n, by_twos);
                if (in) {
                    // a group that is not finite holds zeros beside its scale
                    *reinterpret_cast<uint32_t*>(k_to + (u0 + u) * (R * D / 2)) = code_k == kNanScale ? 0x22222222u : word_of(n[0], n[1], n[2], n[3]);
                    if (col % 4 == 0) {
                        code_to[(u0 + u) * (R * D / 32)] = (uint8_t)code_k;
                        codes[tid / 32][D / 2 + col / 4 * kBlock + j] = (uint8_t)code_v;
                    }
                }
                fields(v[u], code_v, inv_v, n, in_order);
                // this token's two units, the first in the low half; of the word that both tokens share the other lane has one
                const uint32_t both = code_v == kNanScale ? 0x22222222u : word_of(n[0], n[1], n[2], n[3]);
                const uint32_t got = __shfl_xor_sync(0xffffffffu, both, L);
                uint8_t* const pair = v_to + (u0 + u) * (R * D / 2);
                if (in && other) {
                    *reinterpret_cast<uint32_t*>(pair + row % 2 * 4) = __byte_perm(both, got, row % 2 ? 0x3276 : 0x5410);
                } else if (in) {
                    *reinterpret_cast<uint16_t*>(pair + row % 2 * 2) = (uint16_t)both;
                    *reinterpret_cast<uint16_t*>(pair + row % 2 * 2 + 4) = (uint16_t)(both >> 16);
                }
            }
        };
#pragma unroll 1
        for (int u0 = lo / R / kHalf * kHalf; u0 * R < hi; u0 += kHalf) {
            if (u0 * R >= lo && (u0 + kHalf) * R <= hi) half(std::true_type(), u0);
            else half(std::false_type(), u0);
        }
        // the scales as they lie, four bytes a lane
        __syncwarp();
        if (lane * 4 < D) {
            bool all = true, seen[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int at = lane * 4 + y, j = at < D / 2 ? at / (D / 32) : at % kBlock;
                seen[y] = j >= lo && j < hi;
                all = all && seen[y];
            }
            uint8_t* const scales = to + Lay::kScaleK + lane * 4;
            if (all) {
                *reinterpret_cast<uint32_t*>(scales) = *reinterpret_cast<const uint32_t*>(&codes[tid / 32][lane * 4]);
            } else {
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    if (seen[y]) scales[y] = codes[tid / 32][lane * 4 + y];
            }
        }
        __syncwarp();
    }
}

// ---- and out again ---------------------------------------------------------------------

__device__ __forceinline__ uint32_t to_bf16(uint32_t h2) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
    return attn::pack_bf16(f.x, f.y);           // exact
}

template <int D, bool SCRATCH>
__global__ void __launch_bounds__(kThreads) read_kernel(const Args a, const Cache c, const Rows rows, const Scratch scratch) {
    using Lay = Layout<D>;
    constexpr int L = D / 8, R = 32 / L, kSteps = kBlock / R;
    __shared__ Items items;
    const Ones ones;
    const int tid = threadIdx.x, lane = tid % 32, col = lane % L;
    if (!SCRATCH) attn::grid_wait();
    const int64_t total = lay_items<SCRATCH>(a, items) * a.Hk;
    for (int64_t at = (int64_t)blockIdx.x * kWarps + tid / 32; at < total; at += (int64_t)gridDim.x * kWarps) {
        int64_t i = at / a.Hk;
        const int h = (int)(at - i * a.Hk);
        Span s;
        int slot;
        const int b = find<SCRATCH>(a, items, i, s, slot);
        const int block = (i < s.head ? 0 : s.from - s.head) + (int)i, t0 = block * kBlock;
        const uint8_t* const from = c.data + slot * c.ss + h * c.sh + (int64_t)block * Lay::kBytes;
        const int lo = max(s.first - t0, 0), hi = min(s.len - t0, kBlock);
        __nv_bfloat16 *k_to, *v_to;
        int64_t k_next, v_next;                 // from token to token
        if constexpr (SCRATCH) {
            const int64_t first = (((int64_t)b * a.Hk + h) * scratch.length + t0) * D;
            k_to = scratch.k + first;
            v_to = scratch.v + first;
            k_next = v_next = D;
        } else {
            const int64_t row0 = (int64_t)s.row0 - s.first + t0;
            k_to = rows.k + row0 * rows.k_stride + (uint64_t)(uint32_t)h * D;
            v_to = rows.v + row0 * rows.v_stride + (uint64_t)(uint32_t)h * D;
            k_next = rows.k_stride;
            v_next = rows.v_stride;
        }
        uint32_t k[kSteps], codes[kSteps];
        uint2 v[kSteps];
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
            const int j = u * R + lane / L;
            if (j < lo || j >= hi) continue;
            k[u] = *reinterpret_cast<const uint32_t*>(from + j * (D / 2) + col * 4);
            v[u] = *reinterpret_cast<const uint2*>(from + Lay::kV + j / 2 * D + col * 8);
            codes[u] = from[Lay::kScaleK + j * (D / 32) + col / 4] | from[Lay::kScaleV + col / 4 * kBlock + j] << 8;
        }
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
            const int j = u * R + lane / L;
            if (j < lo || j >= hi) continue;
            const Scales sk = scale_of(codes[u] & 255u), sv = scale_of(codes[u] >> 8);
            uint32_t w = k[u], x = swap_bytes(w);
            *reinterpret_cast<uint4*>(k_to + j * k_next + col * 8) =
                make_uint4(to_bf16(field0(w, sk, ones)), to_bf16(field1(w, sk, ones)), to_bf16(field0(x, sk, ones)), to_bf16(field1(x, sk, ones)));
            w = __byte_perm(v[u].x, v[u].y, j % 2 ? 0x7632 : 0x5410);       // this token's two units
            x = swap_bytes(w);
            const uint32_t f0 = to_bf16(field0(w, sv, ones)), f1 = to_bf16(field1(w, sv, ones)), f2 = to_bf16(field0(x, sv, ones)), f3 = to_bf16(field1(x, sv, ones));
            *reinterpret_cast<uint4*>(v_to + j * v_next + col * 8) =
                make_uint4(__byte_perm(f0, f1, 0x5410), __byte_perm(f2, f3, 0x5410), __byte_perm(f0, f1, 0x7632), __byte_perm(f2, f3, 0x7632));
        }
    }
    // the plan, for those that wait for this (they begin at its end: letting them in earlier took 4 us more of windowed prompts)
    if (SCRATCH) attn::grid_wait();
}

// Thread blocks for at most `blocks` cache blocks, up to `each` a SM.
unsigned grid_for(int64_t blocks, int heads, int each) {
    const int64_t want = (blocks * heads + kWarps - 1) / kWarps, most = each * (int64_t)sm_count();
    return (unsigned)(want < most ? (want < 1 ? 1 : want) : most);
}

// A call's rows: checks, and the arguments as the kernels see them.
bd_status rows_call(bool write, void* k, int64_t k_stride, void* v, int64_t v_stride, int64_t T, int64_t B, const bd_kv_cache4* cache,
                    const int32_t* slots, const int32_t* cu_q, const int32_t* lens, void* workspace, size_t ws_bytes, cudaStream_t stream) {
    bd_status st;
    if (bad_cache4(cache, &st)) return st;
    const int64_t row = (int64_t)cache->kv_heads * cache->head_dim;
    if (T < 0 || T > (int64_t)1 << 30 || B < 0 || B > 65535 || (!cu_q && T != B) || k_stride < row || v_stride < row || k_stride > attn::kMaxStride ||
        v_stride > attn::kMaxStride)
        return BD_ERR_SHAPE;
    if (T == 0 || B == 0) return BD_OK;
    if (!k || !v || !lens) return BD_ERR_NULL;
    if (!aligned(k, 16) || !aligned(v, 16) || k_stride % 8 || v_stride % 8 || !aligned(slots, 4) || !aligned(cu_q, 4) || !aligned(lens, 4))
        return BD_ERR_ALIGN;
    if (!workspace || ws_bytes < kHeaderBytes) return BD_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return BD_ERR_ALIGN;
    const Args a = args_of(cache, T, B, slots, cu_q, lens, workspace);
    const Cache c = kernel_cache(cache);
    const Rows rows{static_cast<__nv_bfloat16*>(k), static_cast<__nv_bfloat16*>(v), k_stride, v_stride};
    const unsigned grid = grid_for(T < T / kBlock + 2 * B ? T : T / kBlock + 2 * B, cache->kv_heads, write ? 4 : 8);
    const Scratch none{};
    if (write)
        return cache->head_dim == 128 ? attn::launch_close(write_kernel<128>, grid, kThreads, 0, stream, a, c, rows)
                                      : attn::launch_close(write_kernel<64>, grid, kThreads, 0, stream, a, c, rows);
    return cache->head_dim == 128 ? attn::launch_close(read_kernel<128, false>, grid, kThreads, 0, stream, a, c, rows, none)
                                  : attn::launch_close(read_kernel<64, false>, grid, kThreads, 0, stream, a, c, rows, none);
}

}  // namespace

bool bad_cache4(const bd_kv_cache4* c, bd_status* st) {
    if (!c || !c->data) { *st = BD_ERR_NULL; return true; }
    if (c->slots < 1 || c->slots > attn::kMaxTokens || c->capacity < 1 || c->capacity > attn::kMaxTokens || c->capacity % kBlock ||
        c->kv_heads < 1 || (c->head_dim != 64 && c->head_dim != 128) || c->stride_slot < 1 || c->stride_head < 1 ||
        c->stride_slot > 2 * attn::kMaxStride || c->stride_head > 2 * attn::kMaxStride) {
        *st = BD_ERR_SHAPE;
        return true;
    }
    if (!aligned(c->data, 16) || c->stride_slot % 16 || c->stride_head % 16) { *st = BD_ERR_ALIGN; return true; }
    return false;
}

attn::Args args_of(const bd_kv_cache4* cache, int64_t T, int64_t B, const int32_t* slots, const int32_t* cu_q, const int32_t* lens, void* workspace) {
    Args a{};
    a.n_slots = (int32_t)cache->slots;
    a.capacity = (int32_t)cache->capacity;
    a.T = (int32_t)T;
    a.B = (int32_t)B;
    a.Hk = cache->kv_heads;
    a.slots = slots;
    a.cu_q = cu_q;
    a.lens = lens;
    a.status = static_cast<unsigned*>(workspace);
    return a;
}

Cache kernel_cache(const bd_kv_cache4* c) { return Cache{static_cast<uint8_t*>(c->data), c->stride_slot, c->stride_head}; }

bd_status launch_seen(const Args& a, const Cache& c, int head_dim, __nv_bfloat16* k, __nv_bfloat16* v, int64_t length, cudaStream_t stream) {
    const Scratch scratch{k, v, length};
    const unsigned grid = grid_for((int64_t)a.B * (length / kBlock + 1), a.Hk, 8);
    const Rows none{};
    return head_dim == 128 ? attn::launch_close(read_kernel<128, true>, grid, kThreads, 0, stream, a, c, none, scratch)
                           : attn::launch_close(read_kernel<64, true>, grid, kThreads, 0, stream, a, c, none, scratch);
}

}  // namespace cache4
}  // namespace bd

extern "C" size_t bitdelta_cache4_bytes(int64_t slots, int64_t capacity, int32_t kv_heads, int32_t head_dim) {
    bd_kv_cache4 c{reinterpret_cast<void*>(16), slots, capacity, kv_heads, head_dim, 16, 16};
    bd_status st;
    if (bd::cache4::bad_cache4(&c, &st)) return 0;
    // (slots, capacity up to 2^24, heads up to 2^31: what does not fit 63 bits is no size)
    const double bytes = (double)slots * (double)kv_heads * (double)(capacity / bd::cache4::kBlock) * (17.0 * head_dim);
    return bytes < 9e18 ? (size_t)slots * (size_t)kv_heads * (size_t)(capacity / bd::cache4::kBlock) * (size_t)(17 * head_dim) : 0;
}

extern "C" bd_status bitdelta_cache4_write(const void* k, int64_t k_stride, const void* v, int64_t v_stride, int64_t T, int64_t B, const bd_kv_cache4* cache,
                                           const int32_t* slots, const int32_t* cu_q, const int32_t* lens, void* workspace, size_t ws_bytes, void* stream) {
    return bd::cache4::rows_call(true, const_cast<void*>(k), k_stride, const_cast<void*>(v), v_stride, T, B, cache, slots, cu_q, lens, workspace, ws_bytes,
                                 static_cast<cudaStream_t>(stream));
}

extern "C" bd_status bitdelta_cache4_read(void* k, int64_t k_stride, void* v, int64_t v_stride, int64_t T, int64_t B, const bd_kv_cache4* cache,
                                          const int32_t* slots, const int32_t* cu_q, const int32_t* lens, void* workspace, size_t ws_bytes, void* stream) {
    return bd::cache4::rows_call(false, k, k_stride, v, v_stride, T, B, cache, slots, cu_q, lens, workspace, ws_bytes, static_cast<cudaStream_t>(stream));
}
