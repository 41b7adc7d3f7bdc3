// append_int4.cu -- dec_attn_append_rope_int4: rotary embedding of the new q and k rows and the
// quantising append of the new K/V rows into an INT4 cache (int4.cuh has the format), one kernel.
//
// A row x of d bf16 values (k rotated) becomes codes c, a scale s and a zero point z:
//   lo = min(0, min x), hi = max(0, max x);  s = the smallest number of four significant bits with
//   15 s >= hi - lo, at least 2^-126;  z = rint(-lo / s);  c_i = clamp(rint(x_i / s) + z, 0, 15);
// the cache gives back s (c_i - z), which lies within s / 2 of x_i. Zero lies in [lo, hi], so it is a
// code, 0 <= z <= 15, and |c - z| <= 15 keeps every value a bf16 number.
// A code must not depend on the order of roundings, so k is rotated in fp64 (B200 runs fp64 at half
// the fp32 rate) and rounded to bf16 once by way of fp32, and everything after it is exact in fp32, or one
// correctly rounded operation, or harmless: hi and lo have 8 significant bits and s has 4, so x / s lies on
// a tie of rint or at least 1 / 960 away from it (s / 2 <= |x| < 16 s: x and (k + 1/2) s are multiples of
// 2^(b-6) where s = n 2^b, 8 <= n <= 15). x times the rounded 1 / s is off by less than 2^-19, and rounding
// it to a multiple of 2^-11 first puts it back on the tie, or leaves it on its side.
//
// Work: eight lanes take a row, lane l elements [E l, E l + E) of both halves (E = d / 16), so every rotation
// pair sits in one lane and so do the codes of its bytes; a warp has four rows at a time and loads the next
// four meanwhile. A block takes kA4Tokens tokens (their angles: 64 each, one thread an angle) or, where
// that leaves multiprocessors idle, 32 rows of one token.
//
// Measured: 10010 tokens of 32 + 8 + 8 rows of 128 (231 MB, 35.8 us at the copy rate) in 52 us, issue slots 66% busy and
// the conversion pipe (fp64 and back) 43%; one step's 8 tokens in 3.2 us, which is launch and latency.
#include <cmath>
#include <cstring>

#include "common.cuh"
#include "host_errors.h"
#include "int4.cuh"

namespace decattn {

constexpr int kA4Warps = 8;
constexpr int kA4Threads = 32 * kA4Warps;
constexpr int kA4MaxHalf = 64;
constexpr int kA4Tokens = 8;

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
  int tokens;                     // tokens per block: kA4Tokens or 1
  int groups;                     // blocks per `tokens` tokens: each takes every groups-th set of 32 rows
  double theta[kA4MaxHalf];       // base^(-2i/d)
};

template <int E>
struct A4Vec;  // E bf16 numbers
template <>
struct A4Vec<4> { using T = uint2; };
template <>
struct A4Vec<8> { using T = uint4; };

__device__ __forceinline__ float a4_bf(uint32_t u) { return __uint_as_float(u << 16); }

// rint(x / s) for the rows' numbers (see above), r = 1 / s rounded.
__device__ __forceinline__ int a4_code(float x, float r) {
  const float q = __fadd_rn(__fadd_rn(__fmul_rn(x, r), 6144.f), -6144.f);       // to a multiple of 2^-11
  return __float_as_int(__fadd_rn(q, 12582912.f)) - __float_as_int(12582912.f);  // to a whole number, ties to even
}

// Quantises the row of these eight lanes: x[] are bf16 numbers. Returns the row word; c[] are the codes.
template <int N>
__device__ __forceinline__ uint32_t a4_quantise(const float (&x)[N], int (&c)[N], float& s_out, int& z_out) {
  float lo = 0.f, hi = 0.f;
  bool fine = true;
  #pragma unroll
  for (int e = 0; e < N; ++e) {
    lo = fminf(lo, x[e]);
    hi = fmaxf(hi, x[e]);
    fine &= fabsf(x[e]) < 1.7014118e38f;  // 2^127; false for a NaN
  }
  int ok = fine;
  #pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    ok &= __shfl_xor_sync(0xffffffffu, ok, o);
  }
  // half the range, as hi - lo itself may pass fp32; where the sum is rounded, s must cover what it was: 7.5 s and the larger
  // half have eight significant bits each and lie within a factor of 4, so their difference is exact
  const float far = fmaxf(0.5f * hi, -0.5f * lo), near = fminf(0.5f * hi, -0.5f * lo);
  uint32_t sb = __float_as_uint((far + near) / 7.5f) & 0xfff00000u;
  if (7.5f * __uint_as_float(sb) - far < near) sb += 0x00100000u;
  sb = max(sb, 0x00800000u);  // 2^-126
  const float s = __uint_as_float(sb), r = 1.f / s;
  const int z = a4_code(-lo, r);
  #pragma unroll
  for (int e = 0; e < N; ++e) c[e] = min(max(a4_code(x[e], r) + z, 0), 15);
  s_out = s;
  z_out = z;
  if (!ok) {  // the row is stored as a NaN row: scale NaN, codes and zero point 0
    #pragma unroll
    for (int e = 0; e < N; ++e) c[e] = 0;
    s_out = __int_as_float(0x7fc00000);
    z_out = 0;
    return 0x7fc0u;
  }
  return (sb >> 16) | (uint32_t)z;
}

template <int D>
__global__ void __launch_bounds__(kA4Threads) append_int4_kernel(const AppendInt4Params p) {
  constexpr int HALF = D / 2;
  constexpr int E = D / 16;
  using V = typename A4Vec<E>::T;
  __shared__ double2 cs[kA4Tokens][E][8];   // (cos, sin) of pos * theta_i at [i % E][i / E]
  __shared__ int64_t slot_sm[kA4Tokens];    // the token's row in the pools before adding the head; -1: no slot, -2: no token
  __shared__ int pos_sm[kA4Tokens];
  griddep_wait();  // the inputs are written by the previous kernel of the stream
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & 7;
  const int rows = p.Hq + 2 * p.Hkv;
  const int64_t tile = blockIdx.x / p.groups;
  const int grp = (int)(blockIdx.x - tile * p.groups);
  const int64_t n_rows = p.cu_q ? min((int64_t)p.cu_q[p.B], p.total_rows) : p.total_rows;
  const int64_t tok0 = tile * p.tokens;
  const int nt = (int)min((int64_t)p.tokens, n_rows - tok0);
  if (nt <= 0) return;
  // This warp's sets of four rows: of token t, rows r0 .. r0 + 3 (one for every eight lanes).
  const int first = 4 * (grp * kA4Warps + warp), stride = 4 * kA4Warps * p.groups, sub = lane >> 3;
  const uint32_t q_row = (uint32_t)p.Hq * D, kv_row = (uint32_t)p.Hkv * D;  // elements of a token
  // this lane's 16 numbers of its row
  auto load = [&](int t, int r0, V& lo, V& hi) {
    const int r = r0 + sub;
    if (t >= nt || r >= rows) return;
    const uint64_t tok = tok0 + t;
    const int rk = r - p.Hq, rv = rk - p.Hkv;
    const uint16_t* src = rk < 0 ? p.q_new + tok * q_row + (uint32_t)r * D
                                 : (rv < 0 ? p.k_new + (uint32_t)rk * D : p.v_new + (uint32_t)rv * D) + tok * kv_row;
    lo = reinterpret_cast<const V*>(src)[l];
    hi = reinterpret_cast<const V*>(src + HALF)[l];
  };
  V lo_n = V(), hi_n = V();
  load(0, first, lo_n, hi_n);
  // ---- the tokens' requests, positions and page slots
  if (threadIdx.x < nt) {
    const int64_t tok = tok0 + threadIdx.x;
    int b, t, T;
    bool good = true;
    if (p.cu_q) {
      int a = 0, z = p.B - 1;  // last request with cu_q[b] <= tok
      while (a < z) {
        const int mid = (a + z + 1) >> 1;
        if (p.cu_q[mid] <= tok) a = mid; else z = mid - 1;
      }
      b = a;
      const int c0 = p.cu_q[b], c1 = p.cu_q[b + 1];
      good = c0 >= 0 && tok >= c0 && tok < c1 && c1 <= p.total_rows;  // else offsets that do not cover the row
      t = (int)(tok - c0);
      T = c1 - c0;
    } else {
      T = p.T;
      b = (int)(tok / T);
      t = (int)(tok - (int64_t)b * T);
    }
    int64_t slot = -2;
    int pos = -1;
    if (good) {
      slot = -1;
      const int64_t at = (int64_t)p.seq_lens[b] - T + t;
      if (at >= 0) {
        pos = (int)at;
        const int pg = pos / p.P;
        int pid = -1;
        if (pg < p.mpps) pid = p.page_table[(int64_t)b * p.mpps + pg];
        if (pid >= 0 && pid < p.num_pages) slot = (int64_t)pid * p.Hkv * p.P + (pos - pg * p.P);
        else good = false;
      }
    }
    if (!good && grp == 0) set_status(p.status, DECATTN_EDEVICE);
    slot_sm[threadIdx.x] = slot;
    pos_sm[threadIdx.x] = pos;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < nt * HALF; i += kA4Threads) {
    const int t = i / HALF, j = i - t * HALF;
    double sn, c;
    sincos((double)max(pos_sm[t], 0) * p.theta[j], &sn, &c);
    cs[t][j % E][j / E] = make_double2(c, sn);
  }
  __syncthreads();
  int t_n = 0, r_n = first;
  if (first >= rows) return;
  while (t_n < nt) {
    const V lo = lo_n, hi = hi_n;
    const int t = t_n, r = r_n + sub;
    r_n += stride;
    if (r_n >= rows) {
      r_n = first;
      ++t_n;
    }
    load(t_n, r_n, lo_n, hi_n);
    const int64_t slot = slot_sm[t];
    const uint64_t tok = tok0 + t;
    const bool is_q = r < p.Hq, is_k = !is_q && r < p.Hq + p.Hkv, has = r < rows && slot != -2;
    const uint32_t* lw = reinterpret_cast<const uint32_t*>(&lo);
    const uint32_t* hw = reinterpret_cast<const uint32_t*>(&hi);
    float x[2 * E];  // the row's bf16 numbers (q and k: rotated)
    #pragma unroll
    for (int e = 0; e < E; ++e) {
      x[e] = (e & 1) ? bf16_hi(lw[e / 2]) : bf16_lo(lw[e / 2]);
      x[E + e] = (e & 1) ? bf16_hi(hw[e / 2]) : bf16_lo(hw[e / 2]);
    }
    if (is_q || is_k) {
      #pragma unroll
      for (int e = 0; e < E; ++e) {
        const double2 c = cs[t][e][l];
        const double x1 = (double)x[e], x2 = (double)x[E + e];
        x[e] = (float)(x1 * c.x - x2 * c.y);
        x[E + e] = (float)(x2 * c.x + x1 * c.y);
      }
    }
    uint32_t y[E];  // as bf16 pairs
    #pragma unroll
    for (int e = 0; e < E; ++e) y[e] = pack_bf16(x[2 * e], x[2 * e + 1]);
    auto store = [&](uint16_t* dst, const uint32_t (&u)[E]) {
      V o1, o2;
      #pragma unroll
      for (int e = 0; e < E / 2; ++e) {
        reinterpret_cast<uint32_t*>(&o1)[e] = u[e];
        reinterpret_cast<uint32_t*>(&o2)[e] = u[E / 2 + e];
      }
      reinterpret_cast<V*>(dst)[l] = o1;
      reinterpret_cast<V*>(dst + HALF)[l] = o2;
    };
    if (is_q && has) store(p.q_out + tok * q_row + (uint32_t)r * D, y);
    if (__all_sync(0xffffffffu, is_q || !has)) continue;
    // ---- quantise and store the rows of k and v (the warp together: its shuffles)
    float s;
    int c[2 * E], z;
    #pragma unroll
    for (int e = 0; e < E; ++e) {
      x[2 * e] = bf16_lo(y[e]);
      x[2 * e + 1] = bf16_hi(y[e]);
    }
    const uint32_t word = a4_quantise<2 * E>(x, c, s, z);
    if (is_q || !has) continue;
    const int h = is_k ? r - p.Hq : r - p.Hq - p.Hkv;
    if (slot >= 0) {
      const int64_t row = slot + h * p.P;
      uint32_t n1 = 0, n2 = 0;
      #pragma unroll
      for (int e = 0; e < E; ++e) {
        n1 |= (uint32_t)c[e] << (4 * e);
        n2 |= (uint32_t)c[E + e] << (4 * e);
      }
      uint8_t* dst = (is_k ? p.k_pages : p.v_pages) + row * (D / 2) + l * (E / 2);
      if (E == 8) {
        *reinterpret_cast<uint32_t*>(dst) = n1;
        *reinterpret_cast<uint32_t*>(dst + D / 4) = n2;
      } else {
        *reinterpret_cast<uint16_t*>(dst) = (uint16_t)n1;
        *reinterpret_cast<uint16_t*>(dst + D / 4) = (uint16_t)n2;
      }
      if (l == 0) p.words[(is_k ? 0 : (int64_t)p.num_pages * p.Hkv * p.P) + row] = (uint16_t)word;
    }
    uint16_t* vals = is_k ? p.k_values : p.v_values;
    if (vals) {
      uint32_t v[E];
      #pragma unroll
      for (int e = 0; e < E; ++e)  // exact: see the format
        v[e] = (__float_as_uint(s * (float)(c[2 * e] - z)) >> 16) | (__float_as_uint(s * (float)(c[2 * e + 1] - z)) & 0xffff0000u);
      store(vals + tok * kv_row + (uint32_t)h * D, v);
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
  for (const void* ptr : {q_new, k_new, v_new, (const void*)q_out, (const void*)k_pages, (const void*)v_pages,
                          (const void*)k_values, (const void*)v_values})
    if (reinterpret_cast<uintptr_t>(ptr) & 15) return DECATTN_EALIGN;
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
  // 64 powers take as long as the launch: this host thread keeps the last base's
  static thread_local struct { float base = 0.f; int d = 0; double theta[kA4MaxHalf]; } angles;
  if (angles.base != rope_base || angles.d != s.head_dim) {
    for (int i = 0; i < s.head_dim / 2; ++i) angles.theta[i] = std::pow((double)rope_base, -2.0 * i / s.head_dim);
    angles.base = rope_base;
    angles.d = s.head_dim;
  }
  std::memcpy(p.theta, angles.theta, sizeof p.theta);
  // kA4Tokens tokens to a block, their angles worked out once, where that gives every multiprocessor two blocks;
  // else a block for 32 rows of a token. 8 tokens of 48 rows: 3.2 us; 10010 tokens of 48 rows, a block each: 201 us
  // (its 64 angles once for every 8 rows), 8 tokens a block: 52.
  const int64_t rows = (int64_t)s.n_q_heads + 2 * (int64_t)s.n_kv_heads;
  int dev = 0;
  if (const cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return cuda_fail("cudaGetDevice", e);
  const int sms = default_bins(dev) / split_ctas_per_sm();
  const bool wide = total_q_rows >= (int64_t)2 * kA4Tokens * sms;
  const int64_t groups = wide ? 1 : (rows + 4 * kA4Warps - 1) / (4 * kA4Warps);
  p.tokens = wide ? kA4Tokens : 1;
  const int64_t blocks = (total_q_rows + p.tokens - 1) / p.tokens * groups;
  if (rows * s.head_dim > 0x7fffffff || (int64_t)s.n_kv_heads * s.page_size > 0x7fffffff || blocks > 0x7fffffff) return DECATTN_ENOTSUP;
  p.groups = (int)groups;
  const cudaError_t e = launch_append_int4(p, s.head_dim, blocks, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DECATTN_OK : cuda_fail("INT4 append kernel launch", e);
}
