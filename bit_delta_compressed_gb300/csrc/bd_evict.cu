// bd_evict.cu -- eviction from a key/value cache by accumulated weight.
//
// One thread block per (request, key/value head, part of the source's
// positions).  Every block finds the head's threshold itself -- the weights of
// one head are a few ten KB, cheap next to the rows, and blocks that need
// nothing from one another need one launch and no flags -- and then moves the
// kept rows of its own part.  The threshold is the c-th largest weight of the
// middle (neither first nor recent) keys, found exactly by a radix selection
// of 11 + 11 + 10 bits on the weights' ordered bit patterns; of the keys equal
// to it the earliest are kept, so the result does not depend on the split.
// Measured: 32 requests of 4,100 to 4,608 keys to 4,096 (8 heads of 128) 194 us for 1.09 GB
// = 5.6 TB/s, 83% of a copy's rate.  DRAM moves just those bytes (543 MB read, 488
// written); rows of 256 bytes, a tenth of them left out, read and written at once run no
// faster: selecting and moving in two launches 201 to 210 us, 2 to 12 parts a head 197 to 247.
#include "bd_attn.cuh"

namespace bd {
namespace attn {
namespace {

constexpr int kThreads = 256;
constexpr int kBins = 2048;

struct EvictArgs {
    __nv_bfloat16 *k, *v;
    int64_t ss, st, sh;
    int32_t n_slots, capacity, Hk;
    float* weights;
    int32_t *lens, *kept;
    const int32_t *src, *dst;
    int32_t n, budget, sinks, recent;
    unsigned* status;
};

// Order-preserving bits: a < b as floats iff key(a) < key(b); both zeros alike,
// NaN above everything.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0xFFFFFFFFu;
    const uint32_t u = w == 0.f ? 0u : __float_as_uint(w);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Sum over the block; every thread gets it.  `part`: one int a warp, free on entry.
__device__ __forceinline__ int block_sum(int v, int* part) {
    v = __reduce_add_sync(0xffffffffu, v);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    int s = 0;
    for (int w = 0; w < kThreads / 32; ++w) s += part[w];
    __syncthreads();
    return s;
}

// How many threads before this one have `flag`; `total` over the block.
__device__ __forceinline__ int block_rank(bool flag, int* part, int* total) {
    const unsigned mask = __ballot_sync(0xffffffffu, flag);
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    if (lane == 0) part[warp] = __popc(mask);
    __syncthreads();
    int before = __popc(mask & ((1u << lane) - 1)), all = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        before += w < warp ? part[w] : 0;
        all += part[w];
    }
    __syncthreads();
    *total = all;
    return before;
}

// The c-th largest key of w[lo, hi) (1 <= c <= hi - lo) and, of the keys equal
// to it, how many belong to the c largest.
__device__ uint32_t select_key(const float* w, int lo, int hi, int c, int* hist, int* part, int* equal) {
    __shared__ uint32_t found_bin;
    __shared__ int found_need;
    uint32_t prefix = 0;
    int need = c;
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        for (int i = threadIdx.x; i < kBins; i += kThreads) hist[i] = 0;
        __syncthreads();
        for (int base = lo; base < hi; base += kThreads) {
            const int p = base + threadIdx.x;
            const uint32_t key = p < hi ? weight_key(w[p]) : 0u;
            const bool in = p < hi && (pass == 0 || (key >> (shift + bits)) == prefix);
            const uint32_t bin = (key >> shift) & ((1u << bits) - 1);
            // many weights may share a bin (all zero, at first): a warp whose
            // counted lanes all do adds once
            const unsigned mask = __ballot_sync(0xffffffffu, in);
            if (mask == 0) continue;
            const int leader = __ffs(mask) - 1;
            const uint32_t first_bin = __shfl_sync(0xffffffffu, bin, leader);
            const bool same = __all_sync(0xffffffffu, !in || bin == first_bin);
            if (same) {
                if (threadIdx.x % 32 == (unsigned)leader) atomicAdd(hist + bin, __popc(mask));
            } else if (in) {
                atomicAdd(hist + bin, 1);
            }
        }
        __syncthreads();
        // from the top bin down: thread t owns bins [8 (255 - t), 8 (255 - t) + 8)
        const int first = (kThreads - 1 - (int)threadIdx.x) * (kBins / kThreads);
        int mine = 0;
        for (int i = 0; i < kBins / kThreads; ++i) mine += hist[first + i];
        int incl = mine;
        const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
        for (int x = 1; x < 32; x <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, x);
            if (lane >= x) incl += o;
        }
        if (lane == 31) part[warp] = incl;
        __syncthreads();
        for (int v = 0; v < warp; ++v) incl += part[v];
        if (incl - mine < need && incl >= need) {
            int above = incl - mine;
            int bin = first + kBins / kThreads - 1;
            while (above + hist[bin] < need) above += hist[bin--];
            found_bin = (uint32_t)bin;
            found_need = need - above;
        }
        __syncthreads();
        prefix = (prefix << bits) | found_bin;
        need = found_need;
        __syncthreads();
    }
    *equal = need;
    return prefix;
}

template <int D>
__global__ void __launch_bounds__(kThreads) evict_kernel(const EvictArgs a) {
    __shared__ int hist[kBins];
    __shared__ int part[kThreads / 32];
    __shared__ int list[kThreads];
    const int i = blockIdx.z, h = blockIdx.y, split = blockIdx.x, splits = gridDim.x;
    const int src = a.src[i], dst = a.dst[i];
    bool bad = src < 0 || src >= a.n_slots || dst < 0 || dst >= a.n_slots;
    for (int j = threadIdx.x; j < a.n; j += kThreads) bad = bad || a.src[j] == dst || (j != i && a.dst[j] == dst);
    const int len = bad ? -1 : a.lens[src];
    bad = bad || len < 0 || len > a.capacity;
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) report(a.status, BD_ERR_SLOT);
        return;
    }
    const int keep = min(len, a.budget);
    const float* w = a.weights + ((int64_t)src * a.Hk + h) * a.capacity;
    float* w_out = a.weights + ((int64_t)dst * a.Hk + h) * a.capacity;
    int32_t* kept = a.kept ? a.kept + ((int64_t)i * a.Hk + h) * a.budget : nullptr;

    // keys outside [lo, hi) stay; of those inside, the ones above the threshold
    // and the first `equal` ones at it
    int lo = len, hi = len, equal = 0;
    uint32_t threshold = 0xFFFFFFFFu;
    if (len > a.budget) {
        lo = a.sinks;
        hi = len - a.recent;
        const int c = a.budget - a.sinks - a.recent;
        if (c > 0) threshold = select_key(w, lo, hi, c, hist, part, &equal);
        // c == 0: nothing in the middle is above the largest pattern, and none equal is kept
    }
    const int p0 = (int)((int64_t)len * split / splits), p1 = (int)((int64_t)len * (split + 1) / splits);
    int above = 0, at = 0;
    for (int p = lo + threadIdx.x; p < min(hi, p0); p += kThreads) {
        const uint32_t key = weight_key(w[p]);
        above += key > threshold;
        at += key == threshold;
    }
    above = block_sum(above, part);
    int equal_before = block_sum(at, part);
    int out = min(p0, lo) + above + min(equal_before, equal) + max(0, p0 - hi);

    constexpr int L = D / 8;             // lanes that move one row, 16 bytes each
    constexpr int R = kThreads / L;      // rows in one round
    const int64_t s0 = (int64_t)src * a.ss + (int64_t)h * a.sh + (threadIdx.x % L) * 8;
    const int64_t d0 = (int64_t)dst * a.ss + (int64_t)h * a.sh + (threadIdx.x % L) * 8;
    for (int base = p0; base < p1; base += kThreads) {
        const int p = base + threadIdx.x;
        const bool in = p < p1;
        const float weight = in ? w[p] : 0.f;
        const bool middle = in && p >= lo && p < hi;
        const uint32_t key = weight_key(weight);
        int equals, count;
        const bool is_equal = middle && key == threshold;
        const int rank = equal_before + block_rank(is_equal, part, &equals);
        equal_before += equals;
        const bool keeps = in && (!middle || key > threshold || (is_equal && rank < equal));
        const int place = block_rank(keeps, part, &count);
        if (keeps) {
            list[place] = p;
            w_out[out + place] = weight;
            if (kept) kept[out + place] = p;
        }
        __syncthreads();
        for (int r = threadIdx.x / L; r < count; r += 4 * R) {
            uint4 kk[4], vv[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (r + u * R < count) {
                    const int64_t from = s0 + (int64_t)list[r + u * R] * a.st;
                    kk[u] = ld_stream(reinterpret_cast<const uint4*>(a.k + from));
                    vv[u] = ld_stream(reinterpret_cast<const uint4*>(a.v + from));
                }
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (r + u * R < count) {
                    const int64_t to = d0 + (int64_t)(out + r + u * R) * a.st;
                    *reinterpret_cast<uint4*>(a.k + to) = kk[u];
                    *reinterpret_cast<uint4*>(a.v + to) = vv[u];
                }
        }
        out += count;
        __syncthreads();
    }
    if (kept)
        for (int j = keep + split * kThreads + threadIdx.x; j < a.budget; j += splits * kThreads) kept[j] = -1;
    if (h == 0 && split == 0 && threadIdx.x == 0) a.lens[dst] = keep;
}

}  // namespace
}  // namespace attn
}  // namespace bd

extern "C" size_t bitdelta_evict_workspace(int64_t n, int32_t kv_heads, int64_t capacity) {
    if (n < 0 || n > 65535 || kv_heads < 1 || kv_heads > 65535 || capacity < 1 || capacity > bd::attn::kMaxTokens)
        return 0;
    return bd::kHeaderBytes;
}

extern "C" bd_status bitdelta_cache_evict(const bd_kv_cache* cache, float* weights, int32_t* lens, const int32_t* src,
                                          const int32_t* dst, int64_t n, int64_t budget, int64_t sinks, int64_t recent,
                                          int32_t* kept, void* workspace, size_t ws_bytes, void* stream) {
    using namespace bd;
    using namespace bd::attn;
    bd_status st;
    if (bad_cache(cache, &st)) return st;
    const size_t need = bitdelta_evict_workspace(n, cache->kv_heads, cache->capacity);
    if (need == 0 || budget < 1 || budget > cache->capacity || sinks < 0 || recent < 0 || sinks > budget ||
        recent > budget - sinks)
        return BD_ERR_SHAPE;
    if (n == 0) return BD_OK;
    if (!weights || !lens || !src || !dst) return BD_ERR_NULL;
    if (!aligned(weights, 4) || !aligned(lens, 4) || !aligned(src, 4) || !aligned(dst, 4) || !aligned(kept, 4))
        return BD_ERR_ALIGN;
    if (!workspace || ws_bytes < need) return BD_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return BD_ERR_ALIGN;
    EvictArgs a{};
    a.k = static_cast<__nv_bfloat16*>(cache->k);
    a.v = static_cast<__nv_bfloat16*>(cache->v);
    a.ss = cache->stride_slot;
    a.st = cache->stride_token;
    a.sh = cache->stride_head;
    a.n_slots = (int32_t)cache->slots;
    a.capacity = (int32_t)cache->capacity;
    a.Hk = cache->kv_heads;
    a.weights = weights;
    a.lens = lens;
    a.kept = kept;
    a.src = src;
    a.dst = dst;
    a.n = (int32_t)n;
    a.budget = (int32_t)budget;
    a.sinks = (int32_t)sinks;
    a.recent = (int32_t)recent;
    a.status = static_cast<unsigned*>(workspace);
    const int64_t heads = n * a.Hk;
    // parts: four blocks a SM in all, where the heads alone are fewer
    int64_t splits = (4 * (int64_t)sm_count() + heads - 1) / heads;
    splits = splits < 1 ? 1 : splits > 16 ? 16 : splits;
    const dim3 grid((unsigned)splits, (unsigned)a.Hk, (unsigned)n);
    if (cache->head_dim == 128)
        evict_kernel<128><<<grid, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
    else
        evict_kernel<64><<<grid, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
    return launch_status();
}
