// append_int4.cu -- dec_attn_append_rope_int4: rotary embedding of the new q and k rows and the
// quantising append of the new K/V rows into an INT4 cache (int4.cuh has the format), one kernel.
//
// A row x of d bf16 values (k rotated) becomes codes c, a scale s and a zero point z:
//   lo = min(0, min x), hi = max(0, max x);  s = the smallest number of four significant bits with
//   15 s >= hi - lo, at least 2^-126;  z = rint(-lo / s);  c_i = clamp(rint(x_i / s) + z, 0, 15);
// the cache gives back s (c_i - z), which lies within s / 2 of x_i. Zero lies in [lo, hi], so it is a
// code, 0 <= z <= 15, and |c - z| <= 15 keeps every value a bf16 number.
// A code must not depend on the order of roundings, so k is rotated in fp64 (B200 runs fp64 at half
// the fp32 rate; the rotation is four operations on two elements) and rounded to bf16 once by way of
// fp32, and everything after it is either exact in fp32 or one correctly rounded operation: hi and lo
// have 8 significant bits, s has 4, and x / s is a quotient of an 8-bit by a 4-bit number, which lies
// on a tie of rint exactly or at least 2^-5 of a step away from it.
//
// Work: a block takes tokens blockIdx.x, + gridDim.x / groups, ... of one group of the token's rows
// (Hq q rows, then Hkv k rows, then Hkv v rows), one warp per row; lane l holds elements [E l, E l + E)
// of both halves of its row (E = d / 64), so every rotation pair sits in one lane and, for d = 128,
// so do the two codes of a byte.
#include <cmath>

#include "common.cuh"
#include "host_errors.h"
#include "int4.cuh"

namespace decattn {

constexpr int kA4Warps = 8;
constexpr int kA4Threads = 32 * kA4Warps;
constexpr int kA4MaxHalf = 64;

struct AppendInt4Params {
  const uint16_t* q_new;   // bf16 [rows][Hq][D]
  const uint16_t* k_new;   // bf16 [rows][Hkv][D]
  const uint16_t* v_new;
  const int32_t* page_table;
  const int32_t* seq_lens;
  const int32_t* cu_q;     // [B + 1] row offsets, or null (T rows per request)
  uint16_t* q_out;
  uint8_t* k_pages;        // [num_pages][Hkv][P][D / 2]
  uint8_t* v_pages;
  uint16_t* words;         // [2][num_pages][Hkv][P]
  uint16_t* k_values;      // optional bf16 [rows][Hkv][D]
  uint16_t* v_values;
  int32_t* status;
  int64_t total_rows;
  int B, T, Hq, Hkv, P, num_pages, mpps;
  int groups;                     // blocks per token
  double theta[kA4MaxHalf];       // base^(-2i/d)
};

template <int E>
struct A4Vec;
template <>
struct A4Vec<1> { using T = uint16_t; };
template <>
struct A4Vec<2> { using T = uint32_t; };

__device__ __forceinline__ float a4_bf(uint32_t u) { return __uint_as_float(u << 16); }

// Quantises this warp's row: lane values x[0..E) (first half) and x[E..2E) (second half), bf16
// numbers. Returns the row word; c[] are the codes, as numbers 0..15.
template <int E>
__device__ __forceinline__ uint32_t a4_quantise(const float (&x)[2 * E], uint32_t (&c)[2 * E], float& s_out, int& z_out) {
  float lo = 0.f, hi = 0.f;
  bool fine = true;
  #pragma unroll
  for (int e = 0; e < 2 * E; ++e) {
    lo = fminf(lo, x[e]);
    hi = fmaxf(hi, x[e]);
    fine &= fabsf(x[e]) < 1.7014118e38f;  // 2^127; false for a NaN
  }
  #pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  if (!__all_sync(0xffffffffu, fine)) {  // the row is stored as a NaN row: scale NaN, zero point 0
    #pragma unroll
    for (int e = 0; e < 2 * E; ++e) c[e] = 0;
    s_out = __int_as_float(0x7fc00000);
    z_out = 0;
    return 0x7fc0u;
  }
  const float h = 0.5f * hi - 0.5f * lo;  // half the range: hi - lo itself may pass fp32
  uint32_t sb = __float_as_uint(h / 7.5f) & 0xfff00000u;
  if (7.5f * __uint_as_float(sb) < h) sb += 0x00100000u;
  sb = max(sb, 0x00800000u);  // 2^-126
  const float s = __uint_as_float(sb);
  const float z = rintf(-lo / s);
  #pragma unroll
  for (int e = 0; e < 2 * E; ++e) c[e] = (uint32_t)(int)fminf(fmaxf(rintf(x[e] / s) + z, 0.f), 15.f);
  s_out = s;
  z_out = (int)z;
  return (sb >> 16) | (uint32_t)z_out;
}

template <int D>
__global__ void __launch_bounds__(kA4Threads) append_int4_kernel(const AppendInt4Params p) {
  constexpr int HALF = D / 2;
  constexpr int E = D / 64;
  using V = typename A4Vec<E>::T;
  __shared__ double2 cs[HALF];  // (cos, sin) of pos * theta_i
  griddep_wait();  // the inputs are written by the previous kernel of the stream
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int grp = blockIdx.x % p.groups;
  const int64_t step = gridDim.x / p.groups;
  const int rows = p.Hq + 2 * p.Hkv;
  const int64_t n_rows = p.cu_q ? min((int64_t)p.cu_q[p.B], p.total_rows) : p.total_rows;
  for (int64_t tok = blockIdx.x / p.groups; tok < n_rows; tok += step) {
    // ---- the token's request, position and page slot
    int b, t, T;
    if (p.cu_q) {
      int a = 0, z = p.B - 1;  // last request with cu_q[b] <= tok
      while (a < z) {
        const int mid = (a + z + 1) >> 1;
        if (p.cu_q[mid] <= tok) a = mid; else z = mid - 1;
      }
      b = a;
      const int c0 = p.cu_q[b], c1 = p.cu_q[b + 1];
      if (c0 < 0 || tok < c0 || tok >= c1 || c1 > p.total_rows) {  // offsets that do not cover the row
        if (threadIdx.x == 0 && grp == 0) set_status(p.status, DECATTN_EDEVICE);
        continue;
      }
      t = (int)(tok - c0);
      T = c1 - c0;
    } else {
      T = p.T;
      b = (int)(tok / T);
      t = (int)(tok - (int64_t)b * T);
    }
    const int64_t pos = (int64_t)p.seq_lens[b] - T + t;
    int64_t slot_row = -1;  // (page * Hkv) * P + slot, before adding the head
    if (pos >= 0) {
      const int64_t pg = pos / p.P;
      int pid = -1;
      if (pg < p.mpps) pid = p.page_table[(int64_t)b * p.mpps + pg];
      if (pid >= 0 && pid < p.num_pages)
        slot_row = (int64_t)pid * p.Hkv * p.P + (pos - pg * p.P);
      else if (threadIdx.x == 0 && grp == 0)
        set_status(p.status, DECATTN_EDEVICE);
    }
    __syncthreads();  // the previous token's angles are no longer read
    for (int i = threadIdx.x; i < HALF; i += kA4Threads) {
      double s, c;
      sincos((pos < 0 ? 0.0 : (double)pos) * p.theta[i], &s, &c);
      cs[i] = make_double2(c, s);
    }
    __syncthreads();
    for (int r = grp * kA4Warps + warp; r < rows; r += p.groups * kA4Warps) {
      const bool is_q = r < p.Hq, is_k = !is_q && r < p.Hq + p.Hkv;
      const int h = is_q ? r : is_k ? r - p.Hq : r - p.Hq - p.Hkv;
      const uint16_t* src = is_q ? p.q_new + (tok * p.Hq + h) * D : (is_k ? p.k_new : p.v_new) + (tok * p.Hkv + h) * D;
      const V lo = reinterpret_cast<const V*>(src)[lane], hi = reinterpret_cast<const V*>(src + HALF)[lane];
      uint32_t b1[E], b2[E];  // the row's bf16 bits (q and k: rotated)
      #pragma unroll
      for (int e = 0; e < E; ++e) {
        b1[e] = (uint32_t)((lo >> (16 * e)) & 0xffffu);
        b2[e] = (uint32_t)((hi >> (16 * e)) & 0xffffu);
        if (is_q || is_k) {
          const double2 c = cs[E * lane + e];
          const double x1 = (double)a4_bf(b1[e]), x2 = (double)a4_bf(b2[e]);
          b1[e] = __bfloat16_as_ushort(__float2bfloat16_rn((float)(x1 * c.x - x2 * c.y)));
          b2[e] = __bfloat16_as_ushort(__float2bfloat16_rn((float)(x2 * c.x + x1 * c.y)));
        }
      }
      auto store = [&](uint16_t* dst, const uint32_t (&u1)[E], const uint32_t (&u2)[E]) {
        V o1 = 0, o2 = 0;
        #pragma unroll
        for (int e = 0; e < E; ++e) {
          o1 |= (V)(u1[e] << (16 * e));
          o2 |= (V)(u2[e] << (16 * e));
        }
        reinterpret_cast<V*>(dst)[lane] = o1;
        reinterpret_cast<V*>(dst + HALF)[lane] = o2;
      };
      if (is_q) {
        store(p.q_out + (tok * p.Hq + h) * D, b1, b2);
        continue;
      }
      // ---- quantise and store the row
      float x[2 * E], s;
      uint32_t c[2 * E];
      int z;
      #pragma unroll
      for (int e = 0; e < E; ++e) {
        x[e] = a4_bf(b1[e]);
        x[E + e] = a4_bf(b2[e]);
      }
      const uint32_t word = a4_quantise<E>(x, c, s, z);
      if (slot_row >= 0) {
        const int64_t row = slot_row + (int64_t)h * p.P;
        uint8_t* dst = (is_k ? p.k_pages : p.v_pages) + row * (D / 2);
        if (E == 2) {
          dst[lane] = (uint8_t)(c[0] | (c[E - 1] << 4));
          dst[D / 4 + lane] = (uint8_t)(c[E] | (c[2 * E - 1] << 4));
        } else {  // the byte's two codes sit in lanes 2 i and 2 i + 1
          const uint32_t n1 = __shfl_down_sync(0xffffffffu, c[0], 1), n2 = __shfl_down_sync(0xffffffffu, c[1], 1);
          if ((lane & 1) == 0) {
            dst[lane / 2] = (uint8_t)(c[0] | (n1 << 4));
            dst[D / 4 + lane / 2] = (uint8_t)(c[1] | (n2 << 4));
          }
        }
        if (lane == 0) p.words[(is_k ? 0 : (int64_t)p.num_pages * p.Hkv * p.P) + row] = (uint16_t)word;
      }
      uint16_t* vals = is_k ? p.k_values : p.v_values;
      if (vals) {
        uint32_t v1[E], v2[E];
        #pragma unroll
        for (int e = 0; e < E; ++e) {  // exact: see the format
          v1[e] = __float_as_uint(s * (float)((int)c[e] - z)) >> 16;
          v2[e] = __float_as_uint(s * (float)((int)c[E + e] - z)) >> 16;
        }
        store(vals + (tok * p.Hkv + h) * D, v1, v2);
      }
    }
  }
}

static cudaError_t launch_append_int4(const AppendInt4Params& p, int D, int64_t blocks, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kA4Threads);
  cfg.dynamicSmemBytes = 0;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // launched while the previous kernel drains
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return D == 128 ? cudaLaunchKernelEx(&cfg, append_int4_kernel<128>, p)
                  : cudaLaunchKernelEx(&cfg, append_int4_kernel<64>, p);
}

}  // namespace decattn

using namespace decattn;

extern "C" int dec_attn_append_rope_int4(const dec_attn_shape* shape, const void* q_new, const void* k_new,
                                         const void* v_new, const int32_t* page_table, const int32_t* seq_lens,
                                         const int32_t* cu_q_lens, int64_t total_q_rows, float rope_base, void* q_out,
                                         void* k_pages, void* v_pages, void* kv_words, void* k_values, void* v_values,
                                         int32_t* status, void* stream) {
  if (!shape) return DECATTN_EINVAL;
  const dec_attn_shape& s = *shape;
  if (s.batch < 0 || s.q_tokens <= 0 || s.n_q_heads <= 0 || s.n_kv_heads <= 0 || s.page_size <= 0 ||
      s.num_pages < 0 || s.max_pages_per_seq < 0 || s.n_q_heads % s.n_kv_heads != 0 || total_q_rows < 0)
    return DECATTN_EINVAL;
  if (!cu_q_lens && total_q_rows != (int64_t)s.batch * s.q_tokens) return DECATTN_EINVAL;
  if (!(rope_base > 0.f) || !std::isfinite(rope_base)) return DECATTN_EINVAL;
  if (s.kv_dtype != DECATTN_KV_INT4) return DECATTN_ENOTSUP;
  if (s.head_dim != 64 && s.head_dim != 128) return DECATTN_ENOTSUP;
  if (s.batch == 0 || total_q_rows == 0) return DECATTN_OK;
  if (!q_new || !k_new || !v_new || !page_table || !seq_lens || !q_out || !k_pages || !v_pages || !kv_words)
    return DECATTN_EINVAL;
  if ((k_values == nullptr) != (v_values == nullptr)) return DECATTN_EINVAL;
  const uintptr_t need = s.head_dim == 128 ? 3 : 1;  // 4-byte (d = 128) or 2-byte lane accesses
  for (const void* ptr : {q_new, k_new, v_new, (const void*)q_out, (const void*)k_values, (const void*)v_values})
    if (reinterpret_cast<uintptr_t>(ptr) & need) return DECATTN_EALIGN;
  if (reinterpret_cast<uintptr_t>(kv_words) & 1) return DECATTN_EALIGN;
  if (((reinterpret_cast<uintptr_t>(page_table) | reinterpret_cast<uintptr_t>(seq_lens) |
        reinterpret_cast<uintptr_t>(cu_q_lens) | reinterpret_cast<uintptr_t>(status)) & 3) != 0)
    return DECATTN_EALIGN;
  AppendInt4Params p;
  p.q_new = static_cast<const uint16_t*>(q_new);
  p.k_new = static_cast<const uint16_t*>(k_new);
  p.v_new = static_cast<const uint16_t*>(v_new);
  p.page_table = page_table;
  p.seq_lens = seq_lens;
  p.cu_q = cu_q_lens;
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_pages = static_cast<uint8_t*>(k_pages);
  p.v_pages = static_cast<uint8_t*>(v_pages);
  p.words = static_cast<uint16_t*>(kv_words);
  p.k_values = static_cast<uint16_t*>(k_values);
  p.v_values = static_cast<uint16_t*>(v_values);
  p.status = status;
  p.total_rows = total_q_rows;
  p.B = s.batch; p.T = s.q_tokens; p.Hq = s.n_q_heads; p.Hkv = s.n_kv_heads; p.P = s.page_size;
  p.num_pages = s.num_pages; p.mpps = s.max_pages_per_seq;
  for (int i = 0; i < s.head_dim / 2; ++i) p.theta[i] = std::pow((double)rope_base, -2.0 * i / s.head_dim);
  const int64_t rows = (int64_t)s.n_q_heads + 2 * (int64_t)s.n_kv_heads;
  const int64_t groups = (rows + kA4Warps - 1) / kA4Warps;
  if (groups > 0x7fffffff || total_q_rows > 0x7fffffff) return DECATTN_ENOTSUP;
  p.groups = (int)groups;
  const int64_t tokens = total_q_rows * groups <= 0x7fffffff ? total_q_rows : 0x7fffffff / groups;
  const cudaError_t e = launch_append_int4(p, s.head_dim, tokens * groups, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DECATTN_OK : cuda_fail("INT4 append kernel launch", e);
}
