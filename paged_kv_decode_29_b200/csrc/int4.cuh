// int4.cuh -- the INT4 cache format (DECATTN_KV_INT4): its decoding, shared by the append, decode and prefill kernels,
// and the launches over it.
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

// ------------------------------------------------------------------ launches
// The split kernel over an INT4 cache (split_int4.cu): out_bf16 in place of out.
struct SplitInt4Params : SplitParams {
  const uint8_t* k_codes;   // [num_pages][Hkv][P][D / 2]
  const uint8_t* v_codes;
  const uint16_t* kv_words; // row words [2][num_pages][Hkv][P]
  uint16_t* out_bf16;       // bf16 [B][T][Hq][D]
  int over_q;               // out and q share memory
};
bool split_int4_supported(int D, int GT);                         // split_int4.cu
cudaError_t launch_split_int4(const SplitInt4Params& p, int D, int device, cudaStream_t st);  // split_int4.cu

// The combine kernel with a bf16 output in place of out.
struct CombineBf16Params : CombineParams {
  uint16_t* out_bf16;
};
cudaError_t launch_combine_bf16(const CombineBf16Params& p, int device, cudaStream_t st);  // combine.cu

// The pages each request uses, expanded to a bf16 scratch pool (prefill_int4.cu).
struct WidenInt4Params {
  const uint8_t* k_codes;     // [num_pages][Hkv][P][D / 2]
  const uint8_t* v_codes;
  const uint16_t* kv_words;   // [2][num_pages][Hkv][P]: K, then V
  const int32_t* page_table;  // [B][mpps]
  const int32_t* seq_lens;    // [B]
  uint16_t* k_out;            // bf16 [B * mpps][Hkv][P][D]: page i of request b at b * mpps + i
  uint16_t* v_out;
  int32_t* pt_out;            // [B][mpps]: b * mpps + i
  int32_t* status;            // optional device word
  int B, Hkv, P, num_pages, mpps;
};
cudaError_t launch_widen_int4(const WidenInt4Params& p, cudaStream_t st);  // prefill_int4.cu

// The prefill kernel with a bf16 output in place of out, the keys of a request split over up to `splits` CTAs.
struct PrefillPartsParams : PrefillParams {
  uint16_t* out_bf16;         // bf16 [total_rows][Hq][D]
  int splits;                 // prefill_splits
  int items;                  // packed rows: row-block steps in the grid (prefill_items); 0: every request has as many
  float* part_o;              // [splits][total_rows][Hq][D] normalised partials
  float* part_lse;            // [splits][total_rows][Hq]
};

// Key blocks of 128 that one CTA of a split prefill takes of a request with Lb keys; a row block that sees n
// key blocks has ceil(n / that) parts. Short requests are split less: a part has two blocks at least.
__host__ __device__ inline int prefill_part_blocks(int Lb, int splits) {
  const int n = (Lb + 127) / 128, per = (n + splits - 1) / splits;
  return per < 2 ? 2 : per;
}
// Row-block steps (a CTA each, per head or pair of heads and part) that B requests of up to T rows can come to with
// total_rows rows in all, and the parts that their keys are split into.   prefill.cu
int64_t prefill_items(int B, int T, int G, int64_t total_rows);
int prefill_splits(int B, int T, int Hq, int G, int64_t total_rows, int64_t max_keys);
cudaError_t launch_prefill_parts(const PrefillPartsParams& p, const CUtensorMap& tmQ, const CUtensorMap& tmK,
                                 const CUtensorMap& tmV, const CUtensorMap& tmO, const CUtensorMap& tmP,
                                 cudaStream_t st);                // prefill.cu

}  // namespace decattn
