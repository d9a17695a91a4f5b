// bd_cache4_host.cuh -- what the entry points on the 4-bit cache share.
#pragma once

#include "bd_attn_math.cuh"
#include "bd_cache4.cuh"

namespace bd {
namespace cache4 {

// Host check of a cache description: true, and the error in *st, if it is unfit.
bool bad_cache4(const bd_kv_cache4* c, bd_status* st);

// The arguments that all of them have (heads of q, masks and results are the attention's).
attn::Args args_of(const bd_kv_cache4* cache, int64_t T, int64_t B, const int32_t* slots, const int32_t* cu_q, const int32_t* lens,
                   void* workspace);
Cache kernel_cache(const bd_kv_cache4* c);

// Reads what the queries of a prompt call see back to bf16, [B, Hk, length, head_dim], keys in
// their places.  It runs beside the launch before it, and ends after that.
bd_status launch_seen(const attn::Args& a, const Cache& c, int head_dim, __nv_bfloat16* k, __nv_bfloat16* v, int64_t length, cudaStream_t stream);

}  // namespace cache4
}  // namespace bd
