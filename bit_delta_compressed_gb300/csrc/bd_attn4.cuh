// bd_attn4.cuh -- the attention kernels of the 4-bit cache, for its entry points.
#pragma once

#include "bd_attn_math.cuh"
#include "bd_cache4.cuh"

namespace bd {
namespace attn {

bd_status launch_decode4(const Args& a, const cache4::Cache& cache, int head_dim, const DecodeBuffers& buf, cudaStream_t stream);

}  // namespace attn
}  // namespace bd
