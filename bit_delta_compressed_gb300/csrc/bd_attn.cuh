// bd_attn.cuh -- what the attention kernels share: the call's arguments as
// the kernels see them, the checks of what only the device can read, and the
// visible range of a row.
#pragma once

#include "bd_internal.cuh"

namespace bd {
namespace attn {

constexpr int kMaxGroup = 128;          // query heads of one key/value head
constexpr int64_t kMaxTokens = 1 << 24; // a slot's capacity: positions stay below 2^25
constexpr int64_t kMaxStride = (int64_t)1 << 38;   // elements: a tensor map's strides end at 2^40 bytes
constexpr int kMaxPrefixes = BITDELTA_MAX_PREFIXES;

struct Args {
    const __nv_bfloat16* q;
    int64_t q_stride;
    __nv_bfloat16* out;
    const __nv_bfloat16 *k, *v;
    int64_t ss, st, sh;                 // cache strides: slot, token, head
    int32_t n_slots, capacity;
    int32_t T, B, Hq, Hk, G;            // query rows, requests, heads, heads of a group
    const int32_t *slots, *lens, *cu_q; // cu_q NULL: one row a request
    const int32_t *prefix_ids, *prefix_slots, *prefix_lens;
    int32_t P;
    int32_t window, sinks;
    float scale_log2;                   // scale * log2(e): scores are kept as powers of two
    float* weights;
    unsigned* status;
};

// One request: where its keys lie and which rows of q are its own.
struct Request {
    int32_t slot, len, pslot, plen, row0, rows;
};

// Reads request b.  Anything out of range leaves the request without keys
// (its rows become zeros) and is reported.
__device__ __forceinline__ Request read_request(const Args& a, int b) {
    Request r;
    r.slot = a.slots ? a.slots[b] : b;
    r.len = a.lens[b];
    r.pslot = 0;
    r.plen = 0;
    bool ok = r.slot >= 0 && r.slot < a.n_slots && r.len >= 0 && r.len <= a.capacity;
    if (a.prefix_ids) {
        const int id = a.prefix_ids[b];
        if (id >= 0 && id < a.P) {
            r.pslot = a.prefix_slots[id];
            r.plen = a.prefix_lens[id];
            ok = ok && r.pslot >= 0 && r.pslot < a.n_slots && r.plen >= 0 && r.plen <= a.capacity;
        } else {
            ok = ok && id == -1;
        }
    }
    r.row0 = b;
    r.rows = 1;
    if (a.cu_q) {
        const int lo = a.cu_q[b], hi = a.cu_q[b + 1];
        r.row0 = min(max(lo, 0), a.T);
        r.rows = min(max(hi, r.row0), a.T) - r.row0;
        ok = ok && lo == r.row0 && hi == r.row0 + r.rows && r.len >= r.rows;
    }
    if (!ok) {
        report(a.status, BD_ERR_SLOT);
        r.slot = r.pslot = 0;
        r.len = r.plen = 0;
    }
    return r;
}

// Positions below lo (and not below sinks) are outside the window of a query at t.
__device__ __forceinline__ int window_lo(const Args& a, int t) {
    return a.window > 0 ? max(0, t - a.window + 1) : 0;
}

// Host check of a cache description: true, and the error in *st, if it is unfit.
bool bad_cache(const bd_kv_cache* c, bd_status* st);

}  // namespace attn
}  // namespace bd
