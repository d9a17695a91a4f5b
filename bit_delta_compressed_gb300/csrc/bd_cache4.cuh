// bd_cache4.cuh -- the 4-bit key/value cache: its blocks, and the arithmetic that takes
// values into them and out again.
//
// 32 consecutive values of a head of a token share a scale s, an unsigned float of 5
// exponent and 3 mantissa bits (bias 15): a byte that, 7 bits to the left, is an f16.
// s is the nearest one (ties to even) to max|x| / 7, at most 240, and a value is n s, n
// the nearest whole number (ties to even) to x / s in [-7, 7]; n + 8 is stored.
//
// A block holds 16 tokens of one head, 17 D bytes (D = head_dim), laid out for the
// fragments of mma.m16n8k16 that the attention multiplies:
//   [0, 8 D)       K, 16-bit units [token][D / 8][2]: unit (w, half) holds dims 8 w + 2 f + half
//   [8 D, 16 D)    V, 16-bit units [token / 2][D / 4][token % 2]: unit w holds dims 4 w + f
//   [16 D, +D / 2) scales of K [token][D / 32]
//   [.., 17 D)     scales of V [D / 32][token]
// Field f = 0, 1 of a unit lies at bits 9-6 and 5-2, and f = 2, 3 lies there once the
// unit's bytes are swapped.  So a field becomes an f16 in one logical operation, as the mantissa of 16 +
// q or of 256 + q, and (16 + q) s - 24 s, or (256 + q) s - 264 s, is one fma whose
// result is exact, as are 24 s and 264 s (2 and 6 bits more than s's 4; s <= 240 keeps
// 264 s finite).  With the nibbles in order, three shifts in place of one byte swap a word.
// Tokens share no byte, so any of them can be written by itself.
#pragma once

#include "bd_attn.cuh"

namespace bd {
namespace cache4 {

constexpr int kBlock = 16;                      // tokens of a block
constexpr uint32_t kTopScale = 0xB7;            // 240
constexpr uint32_t kNanScale = 0xFF;            // a group that holds a NaN or an infinity

template <int D>
struct Layout {
    static constexpr int kV = 8 * D, kScaleK = 16 * D, kScaleV = 16 * D + D / 2, kBytes = 17 * D;
};

// One layer's cache as the kernels see it (slots, capacity and heads are the call's).
struct Cache {
    uint8_t* data;
    int64_t ss, sh;                             // strides in bytes: slot, head
};

__device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t swap_bytes(uint32_t w) { return __byte_perm(w, 0, 0x2301); }

// Two scales (f16x2) and what they take away.
struct Scales {
    uint32_t s, c0, c1;
};
__device__ __forceinline__ Scales scales(uint32_t s) {
    return Scales{s, mul2(s, 0xCE00CE00u), mul2(s, 0xDC20DC20u)};      // -24 s, -264 s
}
__device__ __forceinline__ Scales scale_of(uint32_t byte) { return scales(byte * 0x00800080u); }   // one scale twice
__device__ __forceinline__ uint32_t scale_pair(uint32_t two) { return __byte_perm(two, 0, 0x1404) >> 1; }

// What the fields' masks are joined with: 16 and 256 twice.  A logical operation takes one
// constant at most, so these two are registers.
struct Ones {
    uint32_t f0, f1;
    __device__ __forceinline__ Ones() {
        asm volatile("mov.u32 %0, 0x4C004C00;" : "=r"(f0));
        asm volatile("mov.u32 %0, 0x5C005C00;" : "=r"(f1));
    }
};

// (w & mask) | ones
template <uint32_t MASK>
__device__ __forceinline__ uint32_t cut(uint32_t w, uint32_t ones) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "n"(MASK), "r"(ones));
    return r;
}

// The first and second field of a word's two units as values, f16x2; with the word's
// bytes swapped, the third and fourth.
__device__ __forceinline__ uint32_t field0(uint32_t w, const Scales& s, const Ones& k) { return fma2(cut<0x03C003C0u>(w, k.f0), s.s, s.c0); }
__device__ __forceinline__ uint32_t field1(uint32_t w, const Scales& s, const Ones& k) { return fma2(cut<0x003C003Cu>(w, k.f1), s.s, s.c1); }

}  // namespace cache4
}  // namespace bd
