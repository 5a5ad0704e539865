// The 4-bit cache's block of 16 tokens of a head (include/mlora.h): where its atoms lie, and
// codes and scales as numbers.
//
// An atom, 8 bytes, holds 16 adjacent elements of a token: element e in nibble e, as code + 8.  A
// block of D elements is D atoms of keys, D atoms of values, then a byte of scale (e4m3) per atom
// in the same order; all of it 18 D bytes, one copy.  The orders are those in which the lanes of
// mma.sync fragments take them (attend4_split.cu): a lane's two atoms of 16 bytes lie together, a
// warp's 512 bytes in its lanes' order, so that neither copies nor reads of shared memory meet a
// bank conflict.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

namespace mlora {

__host__ __device__ __forceinline__ int block4_bytes(int dim) { return 18 * dim; }

// Keys, in units of 4 groups (of 16 elements): [token % 8][group of the unit][token / 8].
__device__ __forceinline__ int key_atom(int t, int group, int groups) {
    const int u = group >> 2, n = min(4, groups - 4 * u);
    return u * 64 + ((t & 7) * n + (group & 3)) * 2 + (t >> 3);
}
// Values, in units of 8 groups: [token / 8][group of the unit][token % 8].
__device__ __forceinline__ int value_atom(int t, int group, int groups) {
    const int u = group >> 3, n = min(8, groups - 8 * u);
    return u * 128 + ((t >> 3) * n + (group & 7)) * 8 + (t & 7);
}

// d = a b + c on halves
__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// A code times its scale has 3 + 4 significant bits and lies in 2^-9 .. 3136: fp16 and bf16 hold it
// exactly, and one fused operation makes it.  A nibble n = code + 8 goes into the mantissa of a
// constant, whose multiple of the scale, exact as well, is taken off again:
//   bf16, n in bits 6..3 under 0x4300: ( 128 +  8 n) (s / 8)  - 24 s   = (n - 8) s
//   fp16, n in bits 7..4 under 0x6400: (1024 + 16 n) (s / 16) - 72 s   = (n - 8) s
//         n in bits 3..0:              (1024 +    n) (s / 16) - 64.5 s = (n - 8) s / 16
// (64.5 s has 129 * 15 < 2^11 at most.)  In fp16 even nibbles are left over 16, so that a word needs
// one shift for its two halves of nibbles: the other operand, or the sum, takes the 16.
struct Scale2 {
    uint32_t mul, add;         // s / 8 and -24 s, on both halves
};
struct Scale3 {
    uint32_t mul, even, odd;   // s / 16, -64.5 s, -72 s
};
// e4m3 bytes (without a sign) in the low byte of each half.  Bits moved into the wider type's
// exponent and mantissa are the value times 2^-8 (fp16) or 2^-120 (bf16), numbers below the least
// normal one included.  (Any byte becomes a finite bf16, any of 7 bits a finite fp16, so that
// tokens nothing was written to cost nothing under a weight of zero.)
__device__ __forceinline__ Scale3 scale_f16(uint32_t bytes) {
    const uint32_t raw = bytes << 7;
    return Scale3{fma_f16x2(raw, 0x4C004C00u, 0x80008000u),    // * 2^4
                  fma_f16x2(raw, 0xF408F408u, 0x80008000u),    // * -64.5 * 2^8
                  fma_f16x2(raw, 0xF480F480u, 0x80008000u)};   // * -72 * 2^8
}
__device__ __forceinline__ Scale2 scale_bf16(uint32_t bytes) {
    const uint32_t raw = bytes << 4;
    return Scale2{fma_bf16x2(raw, 0x7A007A00u, 0x80008000u),    // * 2^117
                  fma_bf16x2(raw, 0xFDC0FDC0u, 0x80008000u)};   // * -24 * 2^120
}
// (a & b) | c in one instruction.  (The compiler makes two of it: attention over 32 sequences of 32k tokens
// 272 us, 228 us so, when measured.)
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
// Nibble k of each half of w, times the scale of each half.
template <int K>
__device__ __forceinline__ uint32_t codes_f16(uint32_t w, const Scale3& s) {
    const uint32_t x = K >= 2 ? w >> 8 : w;
    return K & 1 ? fma_f16x2(and_or(x, 0x00F000F0u, 0x64006400u), s.mul, s.odd)
                 : fma_f16x2(and_or(x, 0x000F000Fu, 0x64006400u), s.mul, s.even);
}
template <int K>
__device__ __forceinline__ uint32_t codes_bf16(uint32_t w, const Scale2& s) {
    const uint32_t x = K == 0 ? w << 3 : w >> (4 * K - 3);
    return fma_bf16x2(and_or(x, 0x00780078u, 0x43004300u), s.mul, s.add);
}
// A scale in fp32.
__device__ __forceinline__ float scale_f32(uint32_t byte) { return __uint_as_float(byte << 20) * 0x1p120f; }

}  // namespace mlora
