// bd_attn_decode.cu -- attention of one query row a request on its own keys.
//
// o = sum_j p_j v_j with p the softmax of q.k_j: 4 head_dim flops a head and key for
// 4 head_dim bytes a key, one flop a byte of cache for each head of a group (8 for a
// group of 8), so the cache's bytes bound it.  One launch of one block
// a SM; the visible keys of all (request, key/value head) units, in tiles of 16,
// form one line that is cut into equal parts for the blocks and again for their
// warps: ragged lengths, one long request and thousands of short ones all keep
// every SM reading.  A warp works alone: it streams its tiles through a ring of
// its own in shared memory (cp.async, 16 bytes a lane; keys that are not visible
// are never read, their rows are filled with zeros), multiplies with mma.sync
// (m16n8k16: a group's heads are the rows) and keeps a running maximum, sum and
// output in registers.  tcgen05 has nothing to give here: its tiles are 128 rows
// high where a group has 1 to 16, and the tensor work is a tenth of the time.
// Units that several warps or blocks share are joined in their order from shared
// memory and, across blocks, from the workspace by the block that finishes last,
// so the result does not depend on timing.
// Measured (64 query heads on 8 of 128, GPU time): 128 requests of 1 to 16,384 keys
// seeing 4 + 4,096 of them 284 us = 6.6 TB/s, 98% of a copy's rate; 4 requests of
// 90,001 to 131,072 keys 270 us = 6.7 TB/s; one of 300 keys 7.9 us, which is the
// way through loads that wait for one another (lengths, query, keys, joining).
// Groups of 16 heads: 64 requests of 8000 keys on 2 heads 103 us, 77 for the bytes.
// Larger groups read (from L2, mostly) and multiply the keys once for every 16 heads:
// 8 requests of 32,000 keys on one head 72 us for 64 query heads and 113 for 128, 19 for the bytes.
#include <math.h>

#include "bd_attn_line.cuh"
#include "bd_tc_common.cuh"

namespace bd {
namespace attn {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 16;                 // keys of a tile
// R: rows of a unit (8 or 16 query heads).  A probability is multiplied as two
// bf16 terms, so that it keeps 16 significant bits and the result is rounded once,
// at its end.  With up to 8 heads the second term costs nothing (it takes rows 8 to
// 15 of the product), with more a second product.
// An infinite value times the second term, which may be zero or of the other sign,
// would make a NaN of an infinite result.  With 8 rows the second terms' sum stands
// by itself and is added to a finite first one only; with 16 both go to one sum, so the first
// term is rounded towards zero and the second takes 2^-23 of the probability more, so that it is never zero.
// Two stages a warp: of the 64 KB that 8 warps then load ahead nothing is missed, and
// a third makes the reads of large calls slower (284 -> 294 us on the 128 requests).
// 16 rows for up to 8 heads: one request of 300 keys 7.9 -> 9.3 us.
template <int D, int R>
struct Shape {
    static constexpr int kStage = 2 * kTile * D * 2;                        // K and V of a tile
    static constexpr int kStages = 2 * (128 / D);
    static constexpr int kRing = kStage * kStages;                          // of one warp
    static constexpr int kPart = R * D * 4 + R * 8;                         // an open unit: O, then (m, l)
    static constexpr int kSmem = kWarps * (kRing + kPart);
    static_assert(kRing >= kPart, "a warp's last open unit reuses its ring");
};

// Where the visible own keys of a request lie: the first `head` and, behind a
// gap, the window.  Key x of the n visible ones is key x + (x >= head ? gap : 0).
// Measured on both sides: kUnitCost 0 / 3 / 8 on 128 requests over 14 prefixes (own
// parts of 1 to 700 keys) 108 / 99 / 99 us, one request of 8000 keys 17.5 / 17.4 /
// 16.8; kLeast 16 / 64 on the latter 17.4 / 18.3; a block for each short unit, with /
// without, one request of 300 keys 7.8 / 10.3 us, 16 of 200 to 900 12.5 / 15.6.
struct Keys {
    static constexpr int kUnitCost = 3, kLeast = 16, kShort = 64, kJoin = 4;
    int n, head, gap;
    static constexpr bool kAllKept = false;
    static __device__ __forceinline__ Keys of(const Args& a, const Request& r) {
        Keys k;
        const int lo = min(max(window_lo(a, r.plen + r.len - 1) - r.plen, 0), r.len);
        const int sinks = min(max(a.sinks - r.plen, 0), r.len);
        k.gap = max(lo - sinks, 0);
        k.head = k.gap ? sinks : r.len;
        k.n = r.len - k.gap;
        return k;
    }
    __device__ __forceinline__ int tiles() const { return max(1, (n + kTile - 1) / kTile); }
};

template <int D>
__device__ __forceinline__ void load_tile(const Args& a, const Cursor<Keys>& c, int chunks, uint32_t stage, int lane) {
    constexpr int L = D / 8;               // lanes of a row
    constexpr int rows = 32 / L;           // rows of one step
    const int h = c.u / chunks, x0 = c.tile * kTile, row = lane / L;
    const __nv_bfloat16* k = a.k + (int64_t)c.r.slot * a.ss + (int64_t)h * a.sh + (lane % L) * 8;
    const int64_t v = a.v - a.k;
    const uint32_t to = stage + row * (D * 2);
    if (x0 + kTile <= c.k.n && (x0 >= c.k.head || x0 + kTile <= c.k.head)) {
        k += (int64_t)(x0 + (x0 >= c.k.head ? c.k.gap : 0) + row) * a.st;
#pragma unroll
        for (int i = 0; i < kTile / rows; ++i) {
            const uint32_t at = to + i * rows * (D * 2) + (((lane % L) ^ ((i * rows + row) & 7)) << 4);
            cp_async16(at, k, true);
            cp_async16(at + kTile * D * 2, k + v, true);
            k += rows * a.st;
        }
        return;
    }
#pragma unroll 1
    for (int i = 0; i < kTile / rows; ++i) {
        const int x = x0 + i * rows + row;
        const bool in = x < c.k.n;
        const __nv_bfloat16* from = in ? k + (int64_t)(x + (x >= c.k.head ? c.k.gap : 0)) * a.st : a.k;
        const uint32_t at = to + i * rows * (D * 2) + (((lane % L) ^ ((i * rows + row) & 7)) << 4);
        cp_async16(at, from, in);
        cp_async16(at + kTile * D * 2, from + v, in);
    }
}

template <int D, int R>
__global__ void __launch_bounds__(kThreads, 1) decode_kernel(const Args a, const DecodeBuffers buf, const TilePlan plan) {
    using S = Shape<D, R>;
    constexpr int NT = D / 8;              // 8-wide column tiles of the output
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ LineBlock<kWarps> sh;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int chunks = (a.G + R - 1) / R;  // a group of more than 16 heads is read once a 16
    const int units = a.Hk * chunks;

    grid_go_on();
    const Line<Keys> line = lay_line<Keys>(a, sh, units, [&](int b) { return read_request<true>(a, b); });
    const uint32_t ring = smem_addr(smem) + warp * S::kRing;
    float* const tail_part = reinterpret_cast<float*>(smem + warp * S::kRing);
    float* const head_part = reinterpret_cast<float*>(smem + kWarps * S::kRing + warp * S::kPart);

    Cursor<Keys> c;
    if (first_unit(a, sh, line, c, units)) {
        Cursor<Keys> ahead = c;
        bool more = true;
        int put = 0;
        auto prefetch = [&]() {
            if (more) {
                load_tile<D>(a, ahead, chunks, ring + put * S::kStage, lane);
                if (++ahead.tile == ahead.end) more = next_unit(a, sh.kept, line, ahead, units);
            }
            cp_async_commit();
            if (++put == S::kStages) put = 0;
        };
#pragma unroll 1
        for (int i = 0; i < S::kStages - 1; ++i) prefetch();

        int got = 0;
        uint32_t qf[D / 16][R == 8 ? 2 : 4];
        float o[NT][4], m[R / 8], l[R / 8];
        const int row = lane / 4, col = 2 * (lane % 4);
        do {
            const int seg_tile = c.tile;
            {
                const int hk = c.u / chunks, head0 = hk * a.G + (c.u % chunks) * R;
                const int rows = min(R, a.G - (c.u % chunks) * R);
                const __nv_bfloat16* qp = a.q + (int64_t)c.b * a.q_stride + (int64_t)head0 * D;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                    for (int j = 0; j < (R == 8 ? 2 : 4); ++j) {
                        const int r = R == 8 ? row : row + 8 * (j % 2), half = R == 8 ? j : j / 2;
                        qf[kk][j] = r < rows ? *reinterpret_cast<const uint32_t*>(qp + r * D + kk * 16 + half * 8 + col) : 0u;
                    }
#pragma unroll
                for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
#pragma unroll
                for (int i = 0; i < R / 8; ++i) { m[i] = -INFINITY; l[i] = 0.f; }
            }
#pragma unroll 1
            for (; c.tile < c.end; ++c.tile) {
                prefetch();
                cp_async_wait<S::kStages - 1>();
                __syncwarp();
                const uint32_t ks = ring + got * S::kStage, vs = ks + kTile * D * 2;
                if (++got == S::kStages) got = 0;
                float s[2][4] = {}, odd[2][4] = {};    // two chains of products each
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const int key = (lane / 16) * 8 + lane % 8, chunk = 2 * kk + (lane / 8) % 2;
                    uint32_t kf[4];
                    ldmatrix4(kf, ks + key * (D * 2) + ((chunk ^ (key & 7)) << 4));
                    if constexpr (R == 8) {
                        mma16816(kk % 2 ? odd[0] : s[0], qf[kk][0], 0u, qf[kk][1], 0u, kf[0], kf[1]);
                        mma16816(kk % 2 ? odd[1] : s[1], qf[kk][0], 0u, qf[kk][1], 0u, kf[2], kf[3]);
                    } else {
                        mma16816(kk % 2 ? odd[0] : s[0], qf[kk][0], qf[kk][1], qf[kk][2], qf[kk][3], kf[0], kf[1]);
                        mma16816(kk % 2 ? odd[1] : s[1], qf[kk][0], qf[kk][1], qf[kk][2], qf[kk][3], kf[2], kf[3]);
                    }
                }
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[t][i] += odd[t][i];
                const int x0 = c.tile * kTile + col;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const bool in = x0 + 8 * t + i < c.k.n;
                        s[t][i] = in ? s[t][i] * a.scale_log2 : -INFINITY;
                        if (R == 16) s[t][2 + i] = in ? s[t][2 + i] * a.scale_log2 : -INFINITY;
                    }
                if (a.weights) {
                    // the scores, for the weights' pass over them (rows have room for whole tiles)
                    const int hk = c.u / chunks, g0 = (c.u % chunks) * R;
#pragma unroll
                    for (int i = 0; i < R / 8; ++i) {
                        const int r = g0 + row + 8 * i;
                        if (r >= a.G) continue;
                        float* to = buf.scores + ((int64_t)c.b * a.Hq + hk * a.G + r) * buf.score_stride + x0;
                        *reinterpret_cast<float2*>(to) = make_float2(s[0][2 * i], s[0][2 * i + 1]);
                        *reinterpret_cast<float2*>(to + 8) = make_float2(s[1][2 * i], s[1][2 * i + 1]);
                    }
                }
                uint32_t pf[4], pl[4];
                float top[R / 8];
                bool grows = false;
#pragma unroll
                for (int i = 0; i < R / 8; ++i) {
                    float t = fmaxf(fmaxf(s[0][2 * i], s[0][2 * i + 1]), fmaxf(s[1][2 * i], s[1][2 * i + 1]));
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
                    top[i] = fmaxf(m[i], t);
                    grows = grows || top[i] > m[i];
                }
                if (__any_sync(0xffffffffu, grows)) {
                    float f[R / 8];
#pragma unroll
                    for (int i = 0; i < R / 8; ++i) {
                        f[i] = top[i] > m[i] ? exp2_approx(m[i] - top[i]) : 1.f;
                        l[i] *= f[i];
                        m[i] = top[i];
                    }
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        o[i][0] *= f[0];
                        o[i][1] *= f[0];
                        o[i][2] *= f[R / 8 - 1];
                        o[i][3] *= f[R / 8 - 1];
                    }
                }
#pragma unroll
                for (int i = 0; i < R / 8; ++i) {
                    const float use = m[i] == -INFINITY ? 0.f : m[i];
                    float p[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) p[e] = exp2_approx(s[e / 2][2 * i + e % 2] - use);
                    l[i] += (p[0] + p[1]) + (p[2] + p[3]);
                    if constexpr (R == 8) {
                        const uint32_t h0 = pack_bf16(p[0], p[1]), h1 = pack_bf16(p[2], p[3]);
                        pf[0] = h0;
                        pf[1] = pack_bf16(p[0] - bf16_lo(h0), p[1] - bf16_hi(h0));
                        pf[2] = h1;
                        pf[3] = pack_bf16(p[2] - bf16_lo(h1), p[3] - bf16_hi(h1));
                    } else {
                        const uint32_t h0 = pack_bf16_down(p[0], p[1]), h1 = pack_bf16_down(p[2], p[3]);
                        constexpr float more = 1.f + 1.f / (1 << 23);
                        pf[i] = h0;
                        pf[2 + i] = h1;
                        pl[i] = pack_bf16(fmaf(p[0], more, -bf16_lo(h0)), fmaf(p[1], more, -bf16_hi(h0)));
                        pl[2 + i] = pack_bf16(fmaf(p[2], more, -bf16_lo(h1)), fmaf(p[3], more, -bf16_hi(h1)));
                    }
                }
#pragma unroll
                for (int cc = 0; cc < D / 16; ++cc) {
                    const int key = ((lane / 8) % 2) * 8 + lane % 8, chunk = 2 * cc + lane / 16;
                    uint32_t vf[4];
                    ldmatrix4_trans(vf, vs + key * (D * 2) + ((chunk ^ (key & 7)) << 4));
                    mma16816(o[2 * cc], pf[0], pf[1], pf[2], pf[3], vf[0], vf[1]);
                    mma16816(o[2 * cc + 1], pf[0], pf[1], pf[2], pf[3], vf[2], vf[3]);
                    if constexpr (R == 16) {
                        mma16816(o[2 * cc], pl[0], pl[1], pl[2], pl[3], vf[0], vf[1]);
                        mma16816(o[2 * cc + 1], pl[0], pl[1], pl[2], pl[3], vf[2], vf[3]);
                    }
                }
                __syncwarp();
            }
            // the unit, or this warp's part of it, is done
#pragma unroll
            for (int i = 0; i < R / 8; ++i) {
                l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
                l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
            }
            if constexpr (R == 8) {
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    o[i][0] += isfinite(o[i][0]) ? o[i][2] : 0.f;
                    o[i][1] += isfinite(o[i][1]) ? o[i][3] : 0.f;
                }
            }
            const bool open_start = seg_tile > 0, open_end = c.end < c.tiles;
            if (open_start || open_end) {
                // one that began before is kept beside the ring, the last one (no
                // tile follows it) in the ring
                if (!open_start) cp_async_wait<0>();
                __syncwarp();
                float* part = open_start ? head_part : tail_part;
#pragma unroll
                for (int i = 0; i < R / 8; ++i) {
                    const int r = row + 8 * i;
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        *reinterpret_cast<float2*>(part + r * D + t * 8 + col) = make_float2(o[t][2 * i], o[t][2 * i + 1]);
                    if (lane % 4 == 0) *reinterpret_cast<float2*>(part + R * D + 2 * r) = make_float2(m[i], l[i]);
                }
                if (lane == 0) note_open(sh, line, c, open_start, open_end);
            } else {
                const int hk = c.u / chunks, g0 = (c.u % chunks) * R;
#pragma unroll
                for (int i = 0; i < R / 8; ++i) {
                    const int r = g0 + row + 8 * i;
                    if (r >= a.G) continue;
                    const int64_t row_at = (int64_t)c.b * a.Hq + hk * a.G + r;
                    if (buf.with_prefix) {
                        float* to = buf.own + row_at * D + col;
#pragma unroll
                        for (int t = 0; t < NT; ++t)
                            *reinterpret_cast<float2*>(to + t * 8) = make_float2(o[t][2 * i], o[t][2 * i + 1]);
                        if (lane % 4 == 0) buf.own_ml[row_at] = make_float2(m[i], l[i]);
                        continue;
                    }
                    const float inv = inverse(l[i]);
                    __nv_bfloat16* to = a.out + row_at * D + col;
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        *reinterpret_cast<uint32_t*>(to + t * 8) = pack_bf16(o[t][2 * i] * inv, o[t][2 * i + 1] * inv);
                    if (a.weights && lane % 4 == 0) buf.lse[row_at] = log_sum(m[i], l[i]);
                }
            }
        } while (next_unit(a, sh.kept, line, c, units));
        cp_async_wait<0>();
    }
    __syncthreads();

    join_open<D, R>(a, buf, sh, line, chunks, [&](int k) {
        return reinterpret_cast<const float*>(smem + (k % 2 ? k / 2 * S::kRing : kWarps * S::kRing + k / 2 * S::kPart));
    });
    if (buf.with_prefix) {
        // the plan is there: the queries in the order of the prefixes, for the tiles
        grid_wait();
        const int sorted = plan.head->sorted, chunks_q = a.Hq * D / 8;
        for (int i = blockIdx.x; i < sorted; i += gridDim.x) {
            const uint4* from = reinterpret_cast<const uint4*>(a.q + (int64_t)plan.order[i].x * a.q_stride);
            uint4* to = reinterpret_cast<uint4*>(plan.sorted_q + (int64_t)i * a.Hq * D);
            for (int j = tid; j < chunks_q; j += kThreads) to[j] = from[j];
        }
    }
}

// weights[slot, h, key] += sum over the group's heads of exp(score - log of the
// row's denominator).  Reads the scores that the decode kernel left (in L2, up
// to its size) instead of the keys: 4 bytes a head and key for 2 head_dim a key.
// A pass of its own because the denominator is only known when all parts of a row
// are joined.  32 requests of 2,049 to 4,608 keys: 74 us without weights, 87 with the
// scores' stores and this pass (four keys a thread; with two 89, with one 90, where two
// requests of some hundred keys take 13.1, 12.2 and 11.7).
__global__ void __launch_bounds__(256) weigh_kernel(const Args a, const DecodeBuffers buf) {
    const int b = blockIdx.z, hk = blockIdx.y;
    grid_wait();
    const Request r = read_request<true>(a, b);
    const Keys k = Keys::of(a, r);
    const int64_t row = (int64_t)b * a.Hq + (int64_t)hk * a.G;
    float* w = a.weights + ((int64_t)r.slot * a.Hk + hk) * a.capacity;
    // four keys a thread (rows of scores have room for whole tiles)
    for (int x = (blockIdx.x * 256 + threadIdx.x) * 4; x < k.n; x += gridDim.x * 1024) {
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int g = 0; g < a.G; ++g) {
            const float4 s = *reinterpret_cast<const float4*>(buf.scores + (row + g) * buf.score_stride + x);
            const float lse = buf.lse[row + g];
            sum.x += exp2_approx(s.x - lse);
            sum.y += exp2_approx(s.y - lse);
            sum.z += exp2_approx(s.z - lse);
            sum.w += exp2_approx(s.w - lse);
        }
        const float v[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (x + i < k.n) w[x + i + (x + i >= k.head ? k.gap : 0)] += v[i];
    }
}

template <int D, int R>
bd_status launch_shape(const Args& a, const DecodeBuffers& buf, const TilePlan& plan, cudaStream_t stream) {
    const void* kernel = reinterpret_cast<const void*>(decode_kernel<D, R>);
    if (!set_smem_attr(kernel, Shape<D, R>::kSmem, D == 128 ? (R == 8 ? 4 : 5) : (R == 8 ? 6 : 7))) return BD_ERR_CUDA;
    if (buf.with_prefix)       // beside the one block that lays out the prefixes' tiles
        return launch_close(decode_kernel<D, R>, decode_blocks() > 1 ? decode_blocks() - 1 : 1, kThreads, Shape<D, R>::kSmem, stream, a, buf, plan);
    decode_kernel<D, R><<<decode_blocks(), kThreads, Shape<D, R>::kSmem, stream>>>(a, buf, plan);
    return launch_status();
}

}  // namespace

int decode_blocks() { return sm_count() < kMaxBlocks ? sm_count() : kMaxBlocks; }

size_t decode_parts_bytes(int head_dim) { return (size_t)2 * decode_blocks() * (16 * head_dim + 32) * sizeof(float); }

bd_status launch_decode(const Args& a, int head_dim, const DecodeBuffers& buf, const TilePlan& plan, cudaStream_t stream) {
    if (a.G <= 8) return head_dim == 128 ? launch_shape<128, 8>(a, buf, plan, stream) : launch_shape<64, 8>(a, buf, plan, stream);
    return head_dim == 128 ? launch_shape<128, 16>(a, buf, plan, stream) : launch_shape<64, 16>(a, buf, plan, stream);
}

bd_status launch_weigh(const Args& a, const DecodeBuffers& buf, cudaStream_t stream) {
    const int64_t heads = (int64_t)a.B * a.Hk, most = (a.capacity + 1023) / 1024;
    int64_t x = (16 * (int64_t)sm_count() + heads - 1) / heads;
    x = x < most ? x : most;
    return launch_close(weigh_kernel, dim3((unsigned)x, (unsigned)a.Hk, (unsigned)a.B), 256, 0, stream, a, buf);
}

}  // namespace attn
}  // namespace bd
