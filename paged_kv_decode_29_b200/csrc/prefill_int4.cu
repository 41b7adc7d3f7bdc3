// prefill_int4.cu -- prefill over an INT4 KV cache (int4.cuh has the format).
//
// Prefill is a dense contraction, and every element of an INT4 row is a bf16 number exactly. So one
// pass expands the pages that the requests use into a bf16 scratch pool (scratch page
// b * max_pages_per_seq + i holds page i of request b), and the bf16 prefill kernel runs on that with
// a bf16 output: the products see the cache's values without a rounding. The pass moves 66 + 256 bytes
// a row once; the prefill kernel then reads K and V many times over from L2, and would have to expand
// them once per query block and head if it did so itself.
//
// Measured: 4 x 2048 rows, 32 query heads to 8 KV heads: 170 us, of which the expansion of 9 MB into 34 MB about 8; the rest
// is the bf16 prefill kernel, bound by the chain of its two products and its softmax. 5 ragged chunks behind histories
// of up to 7000 keys: 90 us (134 with their keys not split over CTAs).
//
// A NaN row of V (scale not finite) becomes a NaN row of K and zeros in V: a tensor-core product would carry a
// NaN of V into rows that do not see the key (0 times NaN), while a NaN score is masked like any other.
#include "common.cuh"
#include "int4.cuh"

namespace decattn {

constexpr int kWiThreads = 128;
constexpr int kWiD = 128;
constexpr int kWiBatch = 4;  // 16-byte outputs of K and of V that a thread has in flight

// CTA (w, h): scratch page w = b * mpps + i (page i of request b), KV head h, K and V. A thread takes
// 8 codes (4 bytes) of a row at a time and writes 16 bytes, so a warp reads two rows' codes (128 bytes)
// and writes 512 bytes in a row. Pages past the request's keys are never read by the prefill kernel and
// are left unwritten; the rows past its last key, up to a multiple of 16, are zero. A page id outside
// the pool is reported (DECATTN_EDEVICE) and its scratch page is zero.
__global__ void __launch_bounds__(kWiThreads) widen_int4_kernel(const WidenInt4Params p) {
  griddep_wait();               // the pages were written by earlier kernels of the stream
  griddep_launch_dependents();  // the prefill kernel may be scheduled; it waits for this grid itself
  const int w = (int)blockIdx.x, h = (int)blockIdx.y;
  const int b = w / p.mpps, i = w - b * p.mpps;
  if (threadIdx.x == 0 && h == 0) p.pt_out[w] = w;
  const int Lb = p.seq_lens[b];
  if (Lb < 0) {
    if (threadIdx.x == 0 && i == 0 && h == 0) set_status(p.status, DECATTN_EDEVICE);
    return;
  }
  if ((int64_t)i * p.P >= Lb) return;
  const int pid = p.page_table[w];
  const bool good = pid >= 0 && pid < p.num_pages;
  if (!good && threadIdx.x == 0 && h == 0) set_status(p.status, DECATTN_EDEVICE);
  const int rows = min(p.P, (int)(Lb - i * p.P));  // rows of the page that hold a key
  const int64_t src = ((int64_t)(good ? pid : 0) * p.Hkv + h) * p.P;
  const int64_t dst = ((int64_t)w * p.Hkv + h) * p.P;
  const uint16_t* kw = p.kv_words + src;
  const uint16_t* vw = kw + (int64_t)p.num_pages * p.Hkv * p.P;
  const uint32_t* kc = reinterpret_cast<const uint32_t*>(p.k_codes) + src * (kWiD / 8);
  const uint32_t* vc = reinterpret_cast<const uint32_t*>(p.v_codes) + src * (kWiD / 8);
  uint4* ko = reinterpret_cast<uint4*>(p.k_out) + dst * (kWiD / 8);
  uint4* vo = reinterpret_cast<uint4*>(p.v_out) + dst * (kWiD / 8);
  const int n = (rows + 15) / 16 * 16 * (kWiD / 8);  // the prefill kernel copies groups of 16 rows
  for (int c0 = threadIdx.x; c0 < n; c0 += kWiBatch * kWiThreads) {
    uint32_t wk[kWiBatch], wv[kWiBatch], ck[kWiBatch], cv[kWiBatch];
    #pragma unroll
    for (int u = 0; u < kWiBatch; ++u) {  // all loads first
      const int c = c0 + u * kWiThreads, r = c / (kWiD / 8);
      wk[u] = wv[u] = ck[u] = cv[u] = 0;  // a row without a key: 0 (0 - 0)
      if (good && r < rows) {
        wk[u] = kw[r];
        wv[u] = vw[r];
        ck[u] = kc[c];
        cv[u] = vc[c];
      }
    }
    #pragma unroll
    for (int u = 0; u < kWiBatch; ++u) {
      const int c = c0 + u * kWiThreads;
      if (c >= n) break;
      const bool vnan = (wv[u] & 0x7f80u) == 0x7f80u;
      ko[c] = int4_to_bf16(ck[u], vnan ? 0x7fc0u : wk[u]);
      vo[c] = vnan ? make_uint4(0, 0, 0, 0) : int4_to_bf16(cv[u], wv[u]);
    }
  }
}

cudaError_t launch_widen_int4(const WidenInt4Params& p, cudaStream_t st) {
  const int64_t grid = (int64_t)p.B * p.mpps;
  if (grid <= 0) return cudaSuccess;
  if (grid > 0x7fffffff || p.Hkv > 65535) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, (unsigned)p.Hkv);
  cfg.blockDim = dim3(kWiThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // launched while the previous kernel drains
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, widen_int4_kernel, p);
}

}  // namespace decattn
