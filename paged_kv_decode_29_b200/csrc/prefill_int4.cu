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
// of up to 7000 keys: 89 us (134 with their keys not split over CTAs).
//
// A NaN row of V (scale not finite) becomes a NaN row of K and zeros in V: a tensor-core product would carry a
// NaN of V into rows that do not see the key (0 times NaN), while a NaN score is masked like any other.
#include "common.cuh"
#include "int4.cuh"

namespace decattn {

constexpr int kWiThreads = 128;
constexpr int kWiD = 128;
constexpr int kWiPerSm = 16;  // CTAs that a multiprocessor holds: 2048 threads
constexpr int kWiWaves = 4;
constexpr int kWiBatch = 4;  // 16-byte outputs of K and of V that a thread has in flight

// Scratch page w, which holds keys first .. of a request with Lb keys, of KV head h. A thread takes 8 codes (4 bytes)
// of a row at a time and writes 16 bytes, so a warp reads two rows' codes (128 bytes) and writes 512 bytes in a
// row. The rows past the last key, up to a multiple of 16, are zero. A page id outside the pool is reported
// (DECATTN_EDEVICE) and its scratch page is zero.
__device__ __forceinline__ void widen_page(const WidenInt4Params& p, int w, int h, int first, int Lb) {
  if (threadIdx.x == 0 && h == 0) p.pt_out[w] = w;
  const int pid = p.page_table[w];
  const bool good = pid >= 0 && pid < p.num_pages;
  if (!good && threadIdx.x == 0 && h == 0) set_status(p.status, DECATTN_EDEVICE);
  const int rows = min(p.P, Lb - first);  // rows of the page that hold a key
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

// CTA (x, h, b): pages x, x + gridDim.x, .. of request b, KV head h, K and V; page i goes to scratch page
// b * mpps + i. Pages past the request's keys are never read by the prefill kernel and are left unwritten.
__global__ void __launch_bounds__(kWiThreads) widen_int4_kernel(const WidenInt4Params p) {
  griddep_wait();               // the pages were written by earlier kernels of the stream
  griddep_launch_dependents();  // the prefill kernel may be scheduled; it waits for this grid itself
  const int h = (int)blockIdx.y, b = (int)blockIdx.z;
  const int Lb = p.seq_lens[b];
  if (Lb < 0 && threadIdx.x == 0 && blockIdx.x == 0 && h == 0) set_status(p.status, DECATTN_EDEVICE);
  for (int i = (int)blockIdx.x; i < p.mpps && (int64_t)i * p.P < Lb; i += (int)gridDim.x)
    widen_page(p, b * p.mpps + i, h, i * p.P, Lb);
}

cudaError_t launch_widen_int4(const WidenInt4Params& p, cudaStream_t st) {
  if (p.B <= 0 || p.mpps <= 0) return cudaSuccess;
  if (p.Hkv > 65535 || p.B > 65535) return cudaErrorInvalidValue;
  int dev = 0;
  if (const cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return e;
  const int sms = default_bins(dev) / split_ctas_per_sm();
  // A CTA a page, as the table allows for them, up to kWiWaves full GPUs: the host does not know the lengths, and
  // a server's table is as wide as its longest context may become. 5 chunks of 1 to 219 pages, 5 KV heads, all three
  // kernels: 83 us with a table of 219 pages, 86 with one of 4096 (181 with a CTA for each of its pages).
  const int64_t rows = (int64_t)p.B * p.Hkv, most = (int64_t)kWiWaves * kWiPerSm * sms;
  int64_t x = (most + rows - 1) / rows;
  if (x > p.mpps) x = p.mpps;
  if (x < 1) x = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)x, (unsigned)p.Hkv, (unsigned)p.B);
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
