// bd_attn.cu -- attention over a key/value cache: the C entry points (checks
// of the arguments, workspace) and the kernels' launches.
#include <math.h>

#include "bd_attn_math.cuh"

namespace bd {
namespace attn {

bool bad_cache(const bd_kv_cache* c, bd_status* st) {
    if (!c || !c->k || !c->v) { *st = BD_ERR_NULL; return true; }
    if (c->slots < 1 || c->slots > kMaxTokens || c->capacity < 1 || c->capacity > kMaxTokens || c->kv_heads < 1 ||
        (c->head_dim != 64 && c->head_dim != 128) || c->stride_slot < 1 || c->stride_token < 1 || c->stride_head < 1 ||
        c->stride_slot > kMaxStride || c->stride_token > kMaxStride || c->stride_head > kMaxStride) {
        *st = BD_ERR_SHAPE;
        return true;
    }
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || c->stride_slot % 8 || c->stride_token % 8 || c->stride_head % 8) {
        *st = BD_ERR_ALIGN;
        return true;
    }
    return false;
}

bool sizes_ok(int64_t tokens, int64_t batch, int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
    return tokens >= 0 && tokens <= (int64_t)1 << 30 && batch >= 0 && batch <= 65535 && kv_heads >= 1 &&
           q_heads >= kv_heads && q_heads % kv_heads == 0 && q_heads / kv_heads <= kMaxGroup && q_heads <= 65535 &&
           (head_dim == 64 || head_dim == 128);
}

Workspace layout(void* base, int64_t tokens, int64_t batch, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                 int64_t weigh_len) {
    Workspace w{};
    char* p = static_cast<char*>(base);
    size_t at = kHeaderBytes;
    auto take = [&](size_t bytes) {
        char* r = p ? p + at : nullptr;
        at += round_up(bytes, kAlign);
        return r;
    };
    w.decode.tickets = reinterpret_cast<unsigned*>(p ? p + kTicketsAt : nullptr);
    w.decode.parts = reinterpret_cast<float*>(take(decode_parts_bytes(head_dim)));
    w.decode.own = reinterpret_cast<float*>(take((size_t)batch * q_heads * head_dim * sizeof(float)));
    w.decode.own_ml = reinterpret_cast<float2*>(take((size_t)batch * q_heads * sizeof(float2)));
    if (weigh_len > 0) {
        w.decode.score_stride = (int64_t)round_up((size_t)weigh_len, 16);   // whole tiles
        w.decode.lse = reinterpret_cast<float*>(take((size_t)batch * q_heads * sizeof(float)));
        w.decode.scores = reinterpret_cast<float*>(take((size_t)batch * q_heads * w.decode.score_stride * sizeof(float)));
    }
    const int64_t tiles = most_tiles(tokens, batch, q_heads / kv_heads);
    w.plan.head = reinterpret_cast<PlanHead*>(take(sizeof(PlanHead)));
    w.plan.tiles = reinterpret_cast<RowTile*>(take((size_t)tiles * sizeof(RowTile)));
    w.plan.starts = reinterpret_cast<int4*>(take((size_t)tile_blocks() * sizeof(int4)));
    w.plan.order = reinterpret_cast<int2*>(take((size_t)batch * sizeof(int2)));
    w.plan.req_tile = reinterpret_cast<int32_t*>(take((size_t)batch * sizeof(int32_t)));
    w.plan.req_row = reinterpret_cast<int32_t*>(take((size_t)batch * sizeof(int32_t)));
    w.plan.sorted_q = reinterpret_cast<__nv_bfloat16*>(take((size_t)batch * q_heads * head_dim * sizeof(__nv_bfloat16)));
    // parts: every row once, and one unit's rows more for each thread block; a prefill
    // of so many rows that it is not split leaves none
    int64_t rows = split_below() * kPartRows;
    rows = rows < batch * q_heads ? batch * q_heads : rows;
    rows = (rows < tokens * q_heads ? rows : tokens * q_heads) + (int64_t)tile_blocks() * kPartRows;
    w.plan.o = reinterpret_cast<float*>(take((size_t)rows * head_dim * sizeof(float)));
    w.plan.ml = reinterpret_cast<float2*>(take((size_t)rows * sizeof(float2)));
    w.total = at;
    return w;
}

namespace {

bd_status attention(const void* q, int64_t q_stride, int64_t T, int64_t B, int32_t q_heads, const bd_kv_cache* c,
                    const int32_t* slots, const int32_t* cu_q, const int32_t* lens, const int32_t* prefix_ids,
                    const int32_t* prefix_slots, const int32_t* prefix_lens, int32_t P, int32_t window, int32_t sinks,
                    float scale, float* weights, void* out, void* workspace, size_t ws_bytes, cudaStream_t stream) {
    bd_status st;
    if (bad_cache(c, &st)) return st;
    if (!sizes_ok(T, B, q_heads, c->kv_heads, c->head_dim) || window < 0 || sinks < 0 || P < 0 || P > kMaxPrefixes || !isfinite(scale) ||
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
    const Workspace w = layout(workspace, T, B, q_heads, c->kv_heads, c->head_dim, weights ? c->capacity : 0);
    if (cu_q) return launch_prefill(a, c->head_dim, w.plan, stream);
    DecodeBuffers buf = w.decode;
    buf.with_prefix = P > 0;
    if (P > 0) {
        const bd_status done = launch_plan(a, w.plan, stream);
        if (done != BD_OK) return done;
    }
    bd_status done = launch_decode(a, c->head_dim, buf, w.plan, stream);
    if (done == BD_OK && P > 0) done = launch_prefixes(a, c->head_dim, w.plan, buf, stream);
    if (done == BD_OK && weights) done = launch_weigh(a, buf, stream);
    return done;
}

}  // namespace
}  // namespace attn
}  // namespace bd

extern "C" size_t bitdelta_attn_workspace(int64_t tokens, int64_t batch, int32_t q_heads, int32_t kv_heads,
                                          int32_t head_dim, int64_t weigh_len) {
    if (!bd::attn::sizes_ok(tokens, batch, q_heads, kv_heads, head_dim) || weigh_len < 0 ||
        weigh_len > bd::attn::kMaxTokens)
        return 0;
    return bd::attn::layout(nullptr, tokens, batch, q_heads, kv_heads, head_dim, weigh_len).total;
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
