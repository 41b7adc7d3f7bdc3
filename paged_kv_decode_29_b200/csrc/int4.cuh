// int4.cuh -- the INT4 cache format (DECATTN_KV_INT4) and its decoding, shared by the append, decode
// and prefill kernels.
//
// A row is the head_dim elements of one (page, KV head, slot) of K or V: head_dim / 2 bytes of codes,
// element 2 i in the low and 2 i + 1 in the high four bits of byte i, and one 16-bit word: the word
// without its four low bits is the scale s as a bf16 bit pattern, so s has at most four significant
// bits, and the four low bits are the zero point z. Element value: s (c - z). c - z has at most four
// significant bits and a sign, so s (c - z) has at most eight: every value is a bf16 number exactly.
#pragma once
#include "common.cuh"

namespace decattn {

// The scale of a row word as fp32 (the zero point's bits cleared).
__device__ __forceinline__ float int4_scale(uint32_t word) { return __uint_as_float((word & 0xfff0u) << 16); }

// Eight codes -> f16 pairs. Pair i holds the codes at bits 4 i .. 4 i + 3 of the low and of the high
// half of x, minus the zero points of those halves, exactly. A code under f16's 1024 is the number
// 1024 + c (even i), sixteen times it under 1024 + 16 c (odd i): one AND-OR per pair, then one
// addition of -(1024 + z), or one multiply-add (1024 + 16 c) / 16 - (64 + z). One shift serves two pairs.
//   nlo = -(1024 + z), nhi = -(64 + z) as f16 pairs (int4_nlo / int4_nhi).
__device__ __forceinline__ uint32_t int4_and_or(uint32_t x, uint32_t mask) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(x), "r"(mask), "r"(0x64006400u));  // (x & mask) | 1024's bits
  return r;
}
__device__ __forceinline__ uint32_t int4_add(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t int4_fma16(uint32_t a, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(0x2c002c00u), "r"(c));  // a / 16 + c
  return r;
}
__device__ __forceinline__ void int4_to_f16(uint32_t x, uint32_t nlo, uint32_t nhi, uint32_t (&o)[4]) {
  const uint32_t y = x >> 8;
  o[0] = int4_add(int4_and_or(x, 0x000f000fu), nlo);
  o[1] = int4_fma16(int4_and_or(x, 0x00f000f0u), nhi);
  o[2] = int4_add(int4_and_or(y, 0x000f000fu), nlo);
  o[3] = int4_fma16(int4_and_or(y, 0x00f000f0u), nhi);
}
// The zero points of two rows, one in each half of `pair` (bits 0..3 and 16..19; other bits are ignored).
__device__ __forceinline__ uint32_t int4_nlo(uint32_t pair) { return (pair & 0x000f000fu) | 0xe400e400u; }
__device__ __forceinline__ uint32_t int4_nhi(uint32_t pair) { return ((pair << 4) & 0x00f000f0u) | 0xd400d400u; }

// The eight elements of a word of codes, as bf16 pairs in order (element 2 i in the low half of pair i).
__device__ __forceinline__ uint4 int4_to_bf16(uint32_t x, uint32_t word) {
  const float s = int4_scale(word);
  const int z = (int)(word & 15u);
  uint32_t o[4];
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = __float_as_uint(s * (float)((int)((x >> (8 * i)) & 15u) - z));      // exact: 8
    const uint32_t hi = __float_as_uint(s * (float)((int)((x >> (8 * i + 4)) & 15u) - z));  // significant bits
    o[i] = (lo >> 16) | (hi & 0xffff0000u);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace decattn
