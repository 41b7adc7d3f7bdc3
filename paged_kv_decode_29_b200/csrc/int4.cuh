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

// Its zero point as fp32: the four bits under 2^23's pattern are 2^23 + z.
__device__ __forceinline__ float int4_zero(uint32_t word) { return __uint_as_float((word & 15u) | 0x4b000000u) - 8388608.f; }

// Eight codes -> f16 pairs: pair i holds the codes at bits 4 i .. 4 i + 3 of the low and of the high half of x as
// subnormal f16 numbers, c 2^-24 for even i and c 2^-20 for odd i (exact, five instructions for eight codes).
__device__ __forceinline__ void int4_to_f16_codes(uint32_t x, uint32_t (&o)[4]) {
  const uint32_t y = x >> 8;
  o[0] = x & 0x000f000fu;
  o[1] = x & 0x00f000f0u;
  o[2] = y & 0x000f000fu;
  o[3] = y & 0x00f000f0u;
}

// The eight elements of a word of codes, as bf16 pairs in order (element 2 i in the low half of pair i). A code under
// 128's bf16 pattern (step 1) is 128 + c; less 128 + z it is c - z, and that times s has at most eight significant
// bits: both operations are exact. No conversions: fp32 with one a code took 2 us more for 47 MB of bf16.
__device__ __forceinline__ uint4 int4_to_bf16(uint32_t x, uint32_t word) {
  const __nv_bfloat162 s = __bfloat162bfloat162(__ushort_as_bfloat16((unsigned short)(word & 0xfff0u)));
  const __nv_bfloat162 z = __bfloat162bfloat162(__ushort_as_bfloat16((unsigned short)(0x4300u | (word & 15u))));
  const uint32_t y = x >> 4;
  uint32_t o[4];
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    // byte i of x under the low half, of x >> 4 under the high half; the mask keeps the codes alone
    const uint32_t c = (__byte_perm(x, y, (uint32_t)(i | (4 + i) << 8)) & 0x000f000fu) | 0x43004300u;
    const __nv_bfloat162 v = __hmul2(__hsub2(reinterpret_cast<const __nv_bfloat162&>(c), z), s);
    o[i] = reinterpret_cast<const uint32_t&>(v);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace decattn
