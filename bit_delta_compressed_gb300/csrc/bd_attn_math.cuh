// bd_attn_math.cuh -- device pieces of the attention kernels: warp-level copies
// and matrix products, the softmax's exponential, and the interface between the
// kernels of one call (what lies where in the workspace).
#pragma once

#include <math.h>

#include "bd_attn.cuh"

namespace bd {
namespace attn {

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// 16 bytes from global to shared memory; where `in` is false nothing is read
// and zeros are written.
__device__ __forceinline__ void cp_async16(uint32_t to, const void* from, bool in) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(in ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// c (16 x 8, f32) += a (16 x 16, bf16) b (16 x 8, bf16)
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 2^x (2 units in the last place; -inf gives 0).
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// The same, rounded towards zero.
__device__ __forceinline__ uint32_t pack_bf16_down(float lo, float hi) {
    uint32_t r;
    asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// What a row's sum divides by: a row that saw nothing gives zeros, a NaN stays.
__device__ __forceinline__ float inverse(float l) { return l > 0.f ? 1.f / l : l; }

// log2 of a row's denominator; a row without keys weighs nothing.
__device__ __forceinline__ float log_sum(float m, float l) { return l > 0.f ? m + log2f(l) : (l == 0.f ? INFINITY : l); }

// ---- launches that follow one another closely ------------------------------------
// A kernel launched so may start while the one before it in the stream still runs;
// grid_wait() returns when that one has ended and its writes are visible.  Every
// kernel launched so calls it once at least, at its end if not before, so that its
// own end implies the end of all before it.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The next launch may begin as soon as blocks of this one leave room.
__device__ __forceinline__ void grid_go_on() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... Params, typename... Given>
bd_status launch_close(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       Given... given) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t config{};
    config.gridDim = grid;
    config.blockDim = block;
    config.dynamicSmemBytes = smem;
    config.stream = stream;
    config.attrs = &attr;
    config.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&config, kernel, Params(given)...);
    const bd_status st = launch_status();
    return e == cudaSuccess ? st : BD_ERR_CUDA;
}

// ---- the workspace -----------------------------------------------------------
// The header, then what one call needs.  The tickets of units that several blocks
// join have to be zero when a call begins, so they lie in the header, where no other
// entry point writes: a byte for each block, four to a word.  A unit has no more parts
// than there are blocks, so a byte never runs over.
constexpr size_t kTicketsAt = 64;
constexpr int kMaxBlocks = (int)(kHeaderBytes - kTicketsAt);
static_assert(kMaxBlocks < 256, "a ticket is a byte");

struct DecodeBuffers {
    float* parts;        // [2 * blocks] open units: O [R][D], (m, l) [R]
    unsigned* tickets;   // [kMaxBlocks / 4], a byte for each block
    float* scores;       // [B, Hq, score_stride] scaled scores of the visible own keys, by place among them
    float* lse;          // [B, Hq] log2 of the softmax's denominator
    int64_t score_stride;
    float* own;          // [B, Hq, D], and
    float2* own_ml;      // [B, Hq] with prefixes: what the own keys gave, not normalised
    int32_t with_prefix;
};

// Rows of a unit of the tile kernel, and the distance of its parts: part s of a
// unit's row lies kPartRows rows behind part s - 1.
constexpr int kPartRows = 256;

// ---- the tile kernel's plan (in the workspace) ---------------------------------
// A row tile: `tokens` tokens (their rows of q begin at row0; for prefixes row0 is
// a place in `order`) and the keys that any of them sees, as blocks of 128 of two
// sources, the prefix (0) and the request's own keys (1): of each `head` blocks from
// its first key on and `tail` blocks from key `from` on.
struct RowTile {
    int32_t slot[2], head[2], from[2], tail[2];
    int32_t off;             // keys of the prefix: the own keys' positions begin there
    int32_t own_hi;          // own keys that the last token sees
    int32_t lo_min;          // first position of the earliest window
    int32_t row0, tokens, t0;// t0: the first token's position (prefill)
    int32_t blocks, pad;
    int64_t line, rows_before;
};
struct PlanHead {
    int64_t tiles, line, per;// row tiles, blocks of all units, blocks of a thread block
    int32_t split;           // whether the blocks are cut into equal parts
    int32_t sorted;          // requests with a prefix
};
struct TilePlan {
    PlanHead* head;
    RowTile* tiles;
    int4* starts;            // of each thread block: row tile, head and block that its part begins with
    int2* order;             // requests sorted by prefix: request, position of its query
    int32_t* req_tile;       // prefixes: a request's row tile, -1 for none; prefill: its first one
    int32_t* req_row;        // prefixes: its first row of the unit
    __nv_bfloat16* sorted_q; // prefixes: the queries in the order of `order`
    float* o;                // unnormalised parts of rows,
    float2* ml;              // their maximum (log2) and sum
};

// Where a unit's parts lie: of thread blocks first .. first + n - 1, its row r in the
// first of them at row0 + r, each next one kPartRows further.
struct Parts {
    int64_t row0;
    int32_t n;
};
__device__ __forceinline__ Parts parts_of(const RowTile& t, const PlanHead& head, int Hk, int hk, int G) {
    const int64_t start = t.line * Hk + (int64_t)hk * t.blocks, first = start / head.per;
    Parts p;
    p.n = (int32_t)((start + t.blocks - 1) / head.per - first) + 1;
    p.row0 = t.rows_before * Hk + (int64_t)hk * t.tokens * G + first * kPartRows;
    return p;
}

// The workspace of one call: the header, which holds the tickets, lies where every
// call expects it, the rest is scratch.
struct Workspace {
    DecodeBuffers decode;
    TilePlan plan;
    size_t total;
};
bool sizes_ok(int64_t tokens, int64_t batch, int32_t q_heads, int32_t kv_heads, int32_t head_dim);
Workspace layout(void* base, int64_t tokens, int64_t batch, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int64_t weigh_len);

int tile_blocks();
int64_t split_below();       // units from which on a prefill is not split
int64_t most_tiles(int64_t tokens, int64_t batch, int G);
bd_status launch_prefill(const Args& a, int head_dim, const TilePlan& plan, cudaStream_t stream);   // plan and tiles
bd_status launch_tiles(const Args& a, int head_dim, const TilePlan& plan, cudaStream_t stream);
bd_status launch_plan(const Args& a, const TilePlan& plan, cudaStream_t stream);
bd_status launch_prefixes(const Args& a, int head_dim, const TilePlan& plan, const DecodeBuffers& buf, cudaStream_t stream);

int decode_blocks();
size_t decode_parts_bytes(int head_dim);
bd_status launch_decode(const Args& a, int head_dim, const DecodeBuffers& buf, const TilePlan& plan, cudaStream_t stream);
bd_status launch_weigh(const Args& a, const DecodeBuffers& buf, cudaStream_t stream);

}  // namespace attn
}  // namespace bd
