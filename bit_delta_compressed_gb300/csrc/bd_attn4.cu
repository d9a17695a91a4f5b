// bd_attn4.cu -- attention over the 4-bit cache: the C entry points (checks of the
// arguments, workspace) and the kernels' launches.
//
// A prompt's keys are read back to bf16 first, what its queries see of them, and multiplied
// by the tile kernel of the bf16 cache: its products bound a prompt (2048 tokens behind
// 14,336 keys of 8 heads of 128: 540 us at the measured bf16 rate, where reading back is
// 18 MB in and 67 MB out, 12.6 us at a copy's rate, and the tiles' reading of those 67), and a tile made
// of 4 bits in shared memory would be made again by every row tile.  The plan, which goes by lengths alone, is laid out meanwhile (prompts of 1, 66 and 131 tokens 23 -> 17.4 us).
#include <math.h>

#include "bd_attn4.cuh"
#include "bd_attn_line.cuh"
#include "bd_cache4_host.cuh"

namespace bd {
namespace attn {
namespace {

// A prompt call of up to kFewRows rows, or four for each request, goes through the decode kernel, each row as a request of its
// own: its keys are then read, as they lie, once for every row, and not read back.  The host does not see how the rows lie, so
// of a call of more than kFewInAll rows this is so for the requests that have up to kFewEach; the others' keys are read back for the
// tiles, in launches of their own that find nothing where there are none.
// Measured (64 query heads on 8 of 128), row by row / read back: one request's 8 rows on 300 keys 7.7 / 17.2 us, on 16,000 32 / 49, on
// 100,000 142 / 186; 16 rows 8.5 / 17.4, 56 / 51, 270 / 187.  In a call that both kinds share, with 3 rows of each of 19
// other requests of 500 keys, one request's 16 rows on 4000, 16,000 and 100,000 keys: by rows 38 / 67 / 284 us, by tiles 44 / 66 / 199; 10 rows 33 / 52 /
// 188, 43 / 65 / 198; 20 rows by tiles 45 / 68 / 199, all by rows 32 / 72 / 348, all read back 52 / 78 / 220.
// All by rows / shared / all read back: 4 rows of each of 16 requests of 300, 4000 and 16,000 keys 16 / 22 / 21 us, 57 / 64 / 118, 180 / 188 /
// 401; one row of each of 64 of 300 keys 16 / 25 / 61, four of 4000 186 / 195 / 420; of 128 of 4000 keys one row - / 108 / 776,
// four - / 370 / 778.  49 of 64 rows in one request of 16,000 keys, the others on 300, 143 / 76 / 83; 193 of 256 528 / 136 / 227, of
// 100,000 keys 3163 / 555 / 1170.  Calls of up to kFewInAll: 4 rows of each of 8 requests of 300 and 4000 keys 13 / 20 / 19 and
// 34 / 41 / 70; 25 of 32 in one request of 4000, 16,000 and 100,000 keys 28 / 37 / 37, 77 / 61 / 61, 415 / 190 / 203.
constexpr int kFewRows = 8, kFewInAll = 32, kFewEach = 16;
// (Of calls of more than kKept rows or requests, which a block of the decode kernel does not keep on chip, all are read back.)

// The attention's workspace, and behind it the keys and values that prompts read back.
struct Workspace4 {
    Workspace w;
    __nv_bfloat16 *k, *v;
    int64_t length;                        // keys of a request that there is room for
    size_t total;
};

Workspace4 layout4(void* base, int64_t tokens, int64_t batch, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int64_t longest) {
    Workspace4 r{};
    r.w = layout(base, tokens, batch, q_heads, kv_heads, head_dim, 0);
    size_t at = r.w.total;
    char* p = static_cast<char*>(base);
    auto take = [&](size_t bytes) {
        char* q = p ? p + at : nullptr;
        at += round_up(bytes, kAlign);
        return q;
    };
    if (longest > 0) {
        r.length = (longest + cache4::kBlock - 1) / cache4::kBlock * cache4::kBlock;
        const size_t bytes = (size_t)batch * (size_t)kv_heads * (size_t)r.length * (size_t)head_dim * sizeof(__nv_bfloat16);
        r.k = reinterpret_cast<__nv_bfloat16*>(take(bytes));
        r.v = reinterpret_cast<__nv_bfloat16*>(take(bytes));
    }
    r.total = at;
    return r;
}

bd_status attention4(const void* q, int64_t q_stride, int64_t T, int64_t B, int32_t q_heads, const bd_kv_cache4* c, const int32_t* slots,
                     const int32_t* cu_q, const int32_t* lens, int64_t longest, int32_t window, int32_t sinks, float scale, void* out, void* workspace,
                     size_t ws_bytes, cudaStream_t stream) {
    bd_status st;
    if (cache4::bad_cache4(c, &st)) return st;
    if (!sizes_ok(T, B, q_heads, c->kv_heads, c->head_dim) || window < 0 || sinks < 0 || !isfinite(scale) || q_stride < (int64_t)q_heads * c->head_dim ||
        longest < 0 || longest > kMaxTokens)
        return BD_ERR_SHAPE;
    if (T == 0 || B == 0) return BD_OK;
    if (cu_q && longest < 1) return BD_ERR_SHAPE;
    if (!q || !out || !lens) return BD_ERR_NULL;
    if (!aligned(q, 16) || !aligned(out, 16) || q_stride % 8 || !aligned(slots, 4) || !aligned(cu_q, 4) || !aligned(lens, 4)) return BD_ERR_ALIGN;
    const size_t need = bitdelta_attn4_workspace(T, B, q_heads, c->kv_heads, c->head_dim, longest);
    if (!workspace || need == 0 || ws_bytes < need) return BD_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return BD_ERR_ALIGN;
    Args a = cache4::args_of(c, T, B, slots, cu_q, lens, workspace);
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.q_stride = q_stride;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.Hq = q_heads;
    a.G = q_heads / c->kv_heads;
    a.window = window;
    a.sinks = sinks;
    a.scale_log2 = scale * 1.4426950408889634f;
    const cache4::Cache cache = cache4::kernel_cache(c);
    const Workspace4 w = layout4(workspace, T, B, q_heads, c->kv_heads, c->head_dim, longest);
    if (!cu_q) return launch_decode4(a, cache, c->head_dim, w.w.decode, stream);
    a.longest = longest < a.capacity ? (int32_t)longest : a.capacity;
    if (T <= kKept && B <= kKept && (T <= kFewRows || T <= 4 * B)) {
        if (T > kFewInAll) a.few = kFewEach;
        Args rows = a;
        rows.R = a.B;
        rows.B = a.T;
        st = launch_decode4(rows, cache, c->head_dim, w.w.decode, stream);
        if (st != BD_OK || !a.few) return st;
    }
    // the plan (one block) and the reading beside it go by the cache's slots and lengths, the
    // tiles by the plan: request b's keys lie in slot b of what was read back
    a.stands_in = 1;
    st = launch_plan(a, w.w.plan, stream);
    if (st != BD_OK) return st;
    st = cache4::launch_seen(a, cache, c->head_dim, w.k, w.v, w.length, stream);
    if (st != BD_OK) return st;
    a.k = w.k;
    a.v = w.v;
    a.st = c->head_dim;
    a.sh = w.length * a.st;
    a.ss = a.Hk * a.sh;
    a.n_slots = a.B;
    a.capacity = (int32_t)w.length;
    return launch_tiles(a, c->head_dim, w.w.plan, stream);
}

}  // namespace
}  // namespace attn
}  // namespace bd

extern "C" size_t bitdelta_attn4_workspace(int64_t tokens, int64_t batch, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int64_t longest) {
    if (!bd::attn::sizes_ok(tokens, batch, q_heads, kv_heads, head_dim) || longest < 0 || longest > bd::attn::kMaxTokens) return 0;
    // a tensor map's strides end at 2^40 bytes, and a workspace of more is none
    if ((double)batch * kv_heads * (double)longest * head_dim * 4 > (double)((int64_t)1 << 40)) return 0;
    return bd::attn::layout4(nullptr, tokens, batch, q_heads, kv_heads, head_dim, longest).total;
}

extern "C" bd_status bitdelta_attn4_decode(const void* q, int64_t q_stride, int64_t B, int32_t q_heads, const bd_kv_cache4* cache, const int32_t* slots,
                                           const int32_t* lens, int32_t window, int32_t sinks, float scale, void* out, void* workspace, size_t ws_bytes,
                                           void* stream) {
    return bd::attn::attention4(q, q_stride, B, B, q_heads, cache, slots, nullptr, lens, 0, window, sinks, scale, out, workspace, ws_bytes,
                                static_cast<cudaStream_t>(stream));
}

extern "C" bd_status bitdelta_attn4_prefill(const void* q, int64_t q_stride, int64_t T, int64_t B, int32_t q_heads, const bd_kv_cache4* cache,
                                            const int32_t* slots, const int32_t* cu_q, const int32_t* lens, int64_t longest, int32_t window, int32_t sinks,
                                            float scale, void* out, void* workspace, size_t ws_bytes, void* stream) {
    if (B > 0 && !cu_q) return BD_ERR_NULL;
    return bd::attn::attention4(q, q_stride, T, B, q_heads, cache, slots, cu_q, lens, longest, window, sinks, scale, out, workspace, ws_bytes,
                                static_cast<cudaStream_t>(stream));
}
