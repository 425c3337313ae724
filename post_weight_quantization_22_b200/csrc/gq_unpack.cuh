// Unpacking of b-bit codes into pairs of 16-bit floats (packed layers, gq_linear*.cu).
//
// Eight consecutive codes (8 b bits of a row's stream) become four 32-bit registers; register i
// holds code i in its low half and code i + 4 in its high half, which for 4 bits costs one shift
// and one mask a pair.  A code c is made a float by writing it into the mantissa of a constant
// (bf16: 128 + c from 0x4300, 7 bits of room; fp16: 1024 + c from 0x6400, 10 bits) and
// subtracting that constant and the zero point at once: c - z, an integer of at most 8 bits and a
// sign, is exact in both types.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace gq {

// (a & b) | c in one instruction (left to itself the compiler takes two).
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// The eight codes of v (bits 0 .. 8B-1; higher bits are ignored) as pairs (i, i + 4) in bits
// 0..B-1 and 16..16+B-1, the other bits those of `other` (which has none there).
template <int B>
__device__ __forceinline__ void code_pairs(uint32_t lo, uint32_t hi, uint32_t other,
                                           uint32_t (&p)[4]) {
  constexpr uint32_t m = ((1u << B) - 1) * 0x00010001u;
  if constexpr (B <= 4) {
    uint32_t t;
    if constexpr (B == 2) t = __byte_perm(lo, 0, 0x4140);
    if constexpr (B == 3) t = __byte_perm(lo, lo << 4, 0x7610);
    if constexpr (B == 4) t = lo;
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = and_or(t >> (i * B), m, other);
  } else if constexpr (B == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = and_or(__byte_perm(lo, hi, 0x0400 + 0x0101 * i), m, other);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // codes 2h, 2h + 1 in the low bits of a, 2h + 4, 2h + 5 in those of b (2B <= 14 bits each)
      const uint32_t a = h == 0 ? lo : __funnelshift_r(lo, hi, 2 * B);
      const uint32_t b = h == 0 ? __funnelshift_r(lo, hi, 4 * B)
                                : 6 * B >= 32 ? hi >> (6 * B >= 32 ? 6 * B - 32 : 0)
                                              : __funnelshift_r(lo, hi, 6 * B);
      const uint32_t t = __byte_perm(a, b, 0x5410);
      p[2 * h] = and_or(t, m, other);
      p[2 * h + 1] = and_or(t >> B, m, other);
    }
  }
}

__device__ __forceinline__ uint32_t bf16x2_sub(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hsub2(reinterpret_cast<const __nv_bfloat162&>(a),
                                   reinterpret_cast<const __nv_bfloat162&>(b));
  return reinterpret_cast<const uint32_t&>(r);
}
__device__ __forceinline__ uint32_t f16x2_sub(uint32_t a, uint32_t b) {
  const __half2 r = __hsub2(reinterpret_cast<const __half2&>(a),
                            reinterpret_cast<const __half2&>(b));
  return reinterpret_cast<const uint32_t&>(r);
}

// What pair_value subtracts for a zero point z (0 <= z <= 2^B - 1), in both halves.
template <int B, bool kHalf>
__device__ __forceinline__ uint32_t zero_pair(uint32_t z) {
  uint32_t v;
  if constexpr (kHalf) {
    v = 0x6400u + z;  // 1024 + z
  } else if constexpr (B < 8) {
    v = 0x4300u + z;  // 128 + z
  } else {
    v = (uint32_t)__bfloat16_as_ushort(__float2bfloat16((float)z));
  }
  return v * 0x00010001u;
}

// What code_pairs puts around the codes for pair_value: the constant of the type.
template <int B, bool kHalf>
__device__ __forceinline__ constexpr uint32_t pair_other() {
  return kHalf ? 0x64006400u : B < 8 ? 0x43004300u : 0u;
}

// code - zero of a pair from code_pairs with pair_other, exact, in bf16 or fp16.
template <int B, bool kHalf>
__device__ __forceinline__ uint32_t pair_value(uint32_t p, uint32_t zp) {
  if constexpr (kHalf) {
    return f16x2_sub(p, zp);
  } else if constexpr (B < 8) {
    return bf16x2_sub(p, zp);
  } else {
    // 128 + (c mod 128), then minus 128 where c < 128: every step exact in 8 bits
    const uint32_t v = and_or(p, 0x007F007Fu, 0x43004300u);
    const uint32_t low = ((~p >> 7) & 0x00010001u) * 0x4300u;
    return bf16x2_sub(bf16x2_sub(v, low), zp);
  }
}

// Three bf16 parts of an fp32 value, by truncation: their sum is the value (8 + 8 + 8 bits).
__device__ __forceinline__ void split3(float v, uint32_t& h, uint32_t& mid, uint32_t& low) {
  h = __float_as_uint(v) & 0xFFFF0000u;
  const float r = fabsf(v) == __int_as_float(0x7F800000) ? 0.f : v - __uint_as_float(h);
  mid = __float_as_uint(r) & 0xFFFF0000u;
  low = __float_as_uint(r - __uint_as_float(mid));
}

// Words of a row's stream.
__host__ __device__ __forceinline__ int64_t row_words(int64_t n, int bits) {
  return (n * bits + 31) / 32;
}

}  // namespace gq
