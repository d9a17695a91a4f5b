// bd_attn.cu -- attention over a key/value cache: the C entry points (checks
// of the arguments, workspace) and the kernels' launches.
#include <math.h>

#include "bd_attn.cuh"

namespace bd {
namespace attn {

bool bad_cache(const bd_kv_cache* c, bd_status* st) {
    if (!c || !c->k || !c->v) { *st = BD_ERR_NULL; return true; }
    if (c->slots < 1 || c->slots > kMaxTokens || c->capacity < 1 || c->capacity > kMaxTokens || c->kv_heads < 1 ||
        (c->head_dim != 64 && c->head_dim != 128) || c->stride_slot < 1 || c->stride_token < 1 || c->stride_head < 1) {
        *st = BD_ERR_SHAPE;
        return true;
    }
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || c->stride_slot % 8 || c->stride_token % 8 || c->stride_head % 8) {
        *st = BD_ERR_ALIGN;
        return true;
    }
    return false;
}

namespace {

// One warp a (row, query head), the softmax in one pass over the keys with a
// running maximum and sum: lane i holds head_dim / 32 neighbouring values.
template <int D>
__global__ void __launch_bounds__(256) rows_kernel(const Args a) {
    constexpr int E = D / 32;
    const int64_t id = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    const int b = blockIdx.y;
    const Request rq = read_request(a, b);
    const int64_t i = id / a.Hq;
    const int h = id % a.Hq;
    if (i >= rq.rows) return;
    const int64_t row = rq.row0 + i;
    float q[E], o[E] = {};
    for (int e = 0; e < E; ++e)
        q[e] = __bfloat162float(a.q[row * a.q_stride + (int64_t)h * D + lane * E + e]) * a.scale_log2;
    const int end = rq.plen + rq.len;
    const int t = end - rq.rows + (int)i;
    const int lo = window_lo(a, t);
    float m = -INFINITY, l = 0.f;
    for (int p = 0; p <= t && p < end; ++p) {
        if (p >= a.sinks && p < lo) continue;
        const bool own = p >= rq.plen;
        const int64_t at = (int64_t)(own ? rq.slot : rq.pslot) * a.ss + (int64_t)(own ? p - rq.plen : p) * a.st +
                           (int64_t)(h / a.G) * a.sh + lane * E;
        float s = 0.f;
        for (int e = 0; e < E; ++e) s = fmaf(q[e], __bfloat162float(a.k[at + e]), s);
        for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        const float mn = fmaxf(m, s);
        if (mn == -INFINITY) continue;
        const float f = exp2f(m - mn), w = exp2f(s - mn);
        l = l * f + w;
        for (int e = 0; e < E; ++e) o[e] = o[e] * f + w * __bfloat162float(a.v[at + e]);
        m = mn;
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    for (int e = 0; e < E; ++e)
        a.out[(row * a.Hq + h) * D + lane * E + e] = __float2bfloat16(o[e] * inv);
    if (a.weights) {
        const int kv = h / a.G;
        const int first = 0;
        for (int p = max(first, rq.plen); p <= t && p < end; ++p) {
            if (p >= a.sinks && p < lo) continue;
            const int64_t at = (int64_t)rq.slot * a.ss + (int64_t)(p - rq.plen) * a.st + (int64_t)kv * a.sh + lane * E;
            float s = 0.f;
            for (int e = 0; e < E; ++e) s = fmaf(q[e], __bfloat162float(a.k[at + e]), s);
            for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
            if (lane == 0)
                atomicAdd(a.weights + ((int64_t)rq.slot * a.Hk + kv) * a.capacity + p - rq.plen, exp2f(s - m) * inv);
        }
    }
}

bool sizes_ok(int64_t tokens, int64_t batch, int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
    return tokens >= 0 && tokens <= (int64_t)1 << 30 && batch >= 0 && batch <= 65535 && kv_heads >= 1 &&
           q_heads >= kv_heads && q_heads % kv_heads == 0 && q_heads / kv_heads <= kMaxGroup && q_heads <= 65535 &&
           (head_dim == 64 || head_dim == 128);
}

bd_status attention(const void* q, int64_t q_stride, int64_t T, int64_t B, int32_t q_heads, const bd_kv_cache* c,
                    const int32_t* slots, const int32_t* cu_q, const int32_t* lens, const int32_t* prefix_ids,
                    const int32_t* prefix_slots, const int32_t* prefix_lens, int32_t P, int32_t window, int32_t sinks,
                    float scale, float* weights, void* out, void* workspace, size_t ws_bytes, cudaStream_t stream) {
    bd_status st;
    if (bad_cache(c, &st)) return st;
    if (!sizes_ok(T, B, q_heads, c->kv_heads, c->head_dim) || window < 0 || sinks < 0 || P < 0 || !isfinite(scale) ||
        q_stride < (int64_t)q_heads * c->head_dim)
        return BD_ERR_SHAPE;
    if (T == 0 || B == 0) return BD_OK;
    if (!q || !out || !lens) return BD_ERR_NULL;
    if (P > 0 && (!prefix_ids || !prefix_slots || !prefix_lens)) return BD_ERR_NULL;
    if (!aligned(q, 16) || !aligned(out, 16) || q_stride % 8 || !aligned(slots, 4) || !aligned(cu_q, 4) ||
        !aligned(lens, 4) || !aligned(prefix_ids, 4) || !aligned(prefix_slots, 4) || !aligned(prefix_lens, 4) ||
        !aligned(weights, 4))
        return BD_ERR_ALIGN;
    const size_t need =
        bitdelta_attn_workspace(T, B, q_heads, c->kv_heads, c->head_dim, weights ? c->capacity : 0);
    if (!workspace || ws_bytes < need) return BD_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return BD_ERR_ALIGN;
    Args a{};
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.q_stride = q_stride;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.k = static_cast<const __nv_bfloat16*>(c->k);
    a.v = static_cast<const __nv_bfloat16*>(c->v);
    a.ss = c->stride_slot;
    a.st = c->stride_token;
    a.sh = c->stride_head;
    a.n_slots = (int32_t)c->slots;
    a.capacity = (int32_t)c->capacity;
    a.T = (int32_t)T;
    a.B = (int32_t)B;
    a.Hq = q_heads;
    a.Hk = c->kv_heads;
    a.G = q_heads / c->kv_heads;
    a.slots = slots;
    a.lens = lens;
    a.cu_q = cu_q;
    a.prefix_ids = P > 0 ? prefix_ids : nullptr;
    a.prefix_slots = prefix_slots;
    a.prefix_lens = prefix_lens;
    a.P = P;
    a.window = window;
    a.sinks = sinks;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.weights = weights;
    a.status = static_cast<unsigned*>(workspace);
    const int64_t most = cu_q ? T : 1;
    const dim3 grid((unsigned)((most * q_heads + 7) / 8), (unsigned)B);
    if (c->head_dim == 128)
        rows_kernel<128><<<grid, 256, 0, stream>>>(a);
    else
        rows_kernel<64><<<grid, 256, 0, stream>>>(a);
    return launch_status();
}

}  // namespace
}  // namespace attn
}  // namespace bd

extern "C" size_t bitdelta_attn_workspace(int64_t tokens, int64_t batch, int32_t q_heads, int32_t kv_heads,
                                          int32_t head_dim, int64_t weigh_len) {
    if (!bd::attn::sizes_ok(tokens, batch, q_heads, kv_heads, head_dim) || weigh_len < 0 ||
        weigh_len > bd::attn::kMaxTokens)
        return 0;
    return bd::kHeaderBytes;
}

extern "C" bd_status bitdelta_attn_decode(const void* q, int64_t q_stride, int64_t B, int32_t q_heads,
                                          const bd_kv_cache* cache, const int32_t* slots, const int32_t* lens,
                                          int32_t window, int32_t sinks, float scale, float* weights, void* out,
                                          void* workspace, size_t ws_bytes, void* stream) {
    return bd::attn::attention(q, q_stride, B, B, q_heads, cache, slots, nullptr, lens, nullptr, nullptr, nullptr, 0,
                               window, sinks, scale, weights, out, workspace, ws_bytes,
                               static_cast<cudaStream_t>(stream));
}

extern "C" bd_status bitdelta_attn_decode_prefix(const void* q, int64_t q_stride, int64_t B, int32_t q_heads,
                                                 const bd_kv_cache* cache, const int32_t* slots, const int32_t* lens,
                                                 const int32_t* prefix_ids, const int32_t* prefix_slots,
                                                 const int32_t* prefix_lens, int32_t P, int32_t window, int32_t sinks,
                                                 float scale, float* weights, void* out, void* workspace,
                                                 size_t ws_bytes, void* stream) {
    return bd::attn::attention(q, q_stride, B, B, q_heads, cache, slots, nullptr, lens, prefix_ids, prefix_slots,
                               prefix_lens, P, window, sinks, scale, weights, out, workspace, ws_bytes,
                               static_cast<cudaStream_t>(stream));
}

extern "C" bd_status bitdelta_attn_prefill(const void* q, int64_t q_stride, int64_t T, int64_t B, int32_t q_heads,
                                           const bd_kv_cache* cache, const int32_t* slots, const int32_t* cu_q,
                                           const int32_t* lens, const int32_t* prefix_ids, const int32_t* prefix_slots,
                                           const int32_t* prefix_lens, int32_t P, int32_t window, int32_t sinks,
                                           float scale, void* out, void* workspace, size_t ws_bytes, void* stream) {
    if (B > 0 && !cu_q) return BD_ERR_NULL;
    return bd::attn::attention(q, q_stride, T, B, q_heads, cache, slots, cu_q, lens, prefix_ids, prefix_slots,
                               prefix_lens, P, window, sinks, scale, nullptr, out, workspace, ws_bytes,
                               static_cast<cudaStream_t>(stream));
}
