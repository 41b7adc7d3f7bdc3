// split_int4.cu -- the split kernel over an INT4 cache (DECATTN_KV_INT4; int4.cuh has the format): one
// persistent CTA per bin of the plan walks its tiles, as split.cu does for bf16 and E4M3 pages.
//
// Mathematics, for the query rows r of a KV head and the keys j of a tile, with row scales s and zero
// points z of K and V:
//   S_jr = s^K_j <c^K_j - z^K_j, q_r>,  P_jr = 2^(S_jr sm_scale log2 e - m_r),  l_r = sum_j P_jr,
//   O_r  = sum_j (P_jr s^V_j) (c^V_j - z^V_j).
// Only small whole numbers c - z (exact in f16) and q or P s^V meet on the tensor cores; both scales
// multiply one score or one weight instead of head_dim elements.
//  * q_r is scaled by a power of two per row, so that its eight significant bits are exact in f16.
//  * P s^V is rounded once to f16, relative to the tile's largest s^V (a power of two near it is
//    divided out, and put back at the end): 2^-11 half a step, an eighth of the rounding that the
//    bf16 output gets anyway. m, l, O and the partials are fp32.
//
// CTA = 1 producer warp + RG x KG consumer warps. A stage of the ring is a block of 64 keys: K and V codes by
// TMA (64- or 32-byte swizzled rows) and their row words by 16-byte cp.async. Consumer warp (rg, kg)
// computes query rows 8 NQ rg .. + 8 NQ - 1 over every KG-th block, so one warp decodes a block's
// codes for all its rows; the KG warps' states of a tile are merged through shared memory.
//  * keys sit on the MMA's M side in both products (S^T = K Q^T, O^T = V^T P^T), as in split.cu.
//  * K: ldmatrix gives a lane 8 codes of a key; code pairs (i, i + 4) of such a word are one f16 pair
//    of the A operand (the order of head dims in the sum is free: q is laid out to match).
//  * V: ldmatrix.trans gives a lane 4 head dims of 2 neighbouring keys in a word, whose code pairs
//    (i, i + 4) are one f16 pair of V^T. So both operands come from the same 9 instructions per word.
#include "common.cuh"
#include "int4.cuh"

namespace decattn {

constexpr int kI4Block = 64;  // keys per stage
constexpr int kI4PExp = 14;   // P s^V <= 2^(kI4PExp + 1): f16's normal range goes 2^29 below the largest weight

template <int D, int NQ, int RG, int KG, int CPS>
struct I4Cfg {
  static constexpr int RB = D / 2;                            // bytes of a row's codes
  static constexpr int NCH = RB / 16;                         // 16-byte chunks of a row (32 head dims each)
  static constexpr int TILE = kI4Block * RB;                  // K (or V) codes of a stage
  static constexpr int WORDS = 2 * kI4Block;                  // bytes of K (or V) row words of a stage
  static constexpr int STAGE = 2 * TILE + 2 * WORDS;
  static constexpr int NCW = RG * KG;                         // consumer warps
  static constexpr int THREADS = 32 * (1 + NCW);
  static constexpr int QROWS = 8 * NQ * RG;
  static constexpr int QBYTES = QROWS * D * 2;
  static constexpr int NMERGE = KG - 1;                       // merge buffers per row group
  static constexpr int MREGS = NQ * (D / 16 * 4 + 4) + 1;     // O, m, l and the scale exponent, per lane
  static constexpr int MERGE = 32 * 4 * MREGS;
  static constexpr int NBAR_FIXED = 4 + 2 * RG * NMERGE;
  static constexpr int FIXED = 2 * QBYTES + RG * NMERGE * MERGE + 8 * NBAR_FIXED + 2 * (int)sizeof(Unit) + 1024;
  static constexpr int BUDGET = 227 * 1024 / CPS - 1024;      // per CTA, with the system's 1 KB
  static constexpr int FIT = (BUDGET - FIXED) / (STAGE + 16);
  // A multiple of KG: stage s belongs to key group s % KG for good. A warp that waited for other warps' stages
  // could reach a stage's next phase before its present one has begun, which a parity cannot tell apart.
  static constexpr int STAGES = (FIT > 8 ? 8 : FIT) / KG * KG;
  static_assert(STAGES >= 3 && STAGES >= KG, "the ring holds a block for every key group and one in flight");
  static constexpr int OFF_WORDS = STAGES * 2 * TILE;         // [stage][K, V][64] words
  static constexpr int OFF_Q = OFF_WORDS + STAGES * 2 * WORDS;
  static constexpr int OFF_MERGE = OFF_Q + 2 * QBYTES;
  static constexpr int OFF_BAR = OFF_MERGE + RG * NMERGE * MERGE;
  static constexpr int NBAR = 2 * STAGES + NBAR_FIXED;        // full, empty, qfull[2], qempty[2], mfull, mempty
  static constexpr int OFF_QMETA = OFF_BAR + 8 * NBAR;
  static constexpr int BYTES = OFF_QMETA + 2 * (int)sizeof(Unit);
  static constexpr int ALLOC = BYTES + 1024;                  // slack to align the base to 1024
  static_assert(CPS * (ALLOC + 1024) <= 228 * 1024, "the CTAs fit an SM's shared memory");
  // byte offset of (row r, 16-byte chunk c) in a stage's K or V codes: the TMA 64- or 32-byte swizzle
  __device__ static __forceinline__ uint32_t off(int r, int c) {
    return RB == 64 ? (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4)) : (uint32_t)(r * 32 + ((c ^ ((r >> 2) & 1)) << 4));
  }
};

__device__ __forceinline__ void cp_async_16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

template <int D, int NQ, int RG, int KG, int CPS>
__global__ void __launch_bounds__(I4Cfg<D, NQ, RG, KG, CPS>::THREADS, CPS)
split_int4_kernel(const SplitParams p, const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV) {
  using C = I4Cfg<D, NQ, RG, KG, CPS>;
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + C::OFF_BAR);
  uint64_t* empty = full + STAGES;
  uint64_t* qfull = empty + STAGES;
  uint64_t* qempty = qfull + 2;
  uint64_t* mfull = qempty + 2;           // [rg][buffer]
  uint64_t* mempty = mfull + RG * C::NMERGE;
  Unit* qmeta = reinterpret_cast<Unit*>(sm + C::OFF_QMETA);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t wl = p.wait_ns;  // every pipeline wait gives up after this long
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], RG); }
    for (int s = 0; s < 2; ++s) { mbar_init(&qfull[s], 1); mbar_init(&qempty[s], C::NCW); }
    for (int i = 0; i < RG * C::NMERGE; ++i) { mbar_init(&mfull[i], 1); mbar_init(&mempty[i], 1); }
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) { prefetch_tensormap(&tmK); prefetch_tensormap(&tmV); }
  // Everything below reads or writes what earlier kernels of the stream may still be working on: the
  // plan, the pages (a plan serves every layer of a step, so the kernel before this one can be the
  // append), the combine counters.
  griddep_wait();
  griddep_launch_dependents();  // the combine kernel may be scheduled; it waits for this grid itself
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < (int64_t)p.B * p.T * p.Hq;
       i += (int64_t)gridDim.x * blockDim.x)
    p.row_cnt[i] = 0;
  __syncthreads();

  if (warp == 0) {
    // ===================================================================== producer
    const PlanHeader hv = *reinterpret_cast<const PlanHeader*>(p.plan);
    int n_units = 0;
    if (hv.magic == kPlanMagic && hv.status == DECATTN_OK && hv.n_bins == (int)gridDim.x && hv.batch == p.B &&
        hv.n_kv_heads == p.Hkv && hv.tile_len == p.tile_len && hv.sparse == p.sparse)
      n_units = plan_bin_size(p.plan, hv, blockIdx.x);
    else if (lane == 0)
      set_status(p.status, hv.magic != kPlanMagic ? DECATTN_EINVAL : hv.status != DECATTN_OK ? hv.status : DECATTN_EINVAL);
    const int P = p.P, R = p.box_rows;  // R keys per TMA box: divides P and kI4Block
    const int nbox = kI4Block / R;
    int s = 0; uint32_t eph = 1;
    int qs = 0; uint32_t qeph = 1;
    bool ok = true;
    int64_t n_fill = 0, n_qfill = 0;  // ring stages and q slots whose copies were issued
    auto unit = [&](int j) {
      return hv.sparse ? plan_unit_sparse(p.plan, hv, p.seq_lens, blockIdx.x, j)
                       : plan_unit(p.plan, hv, p.seq_lens, blockIdx.x, j);
    };
    // page ids of logical pages pg0 + c .. + 31 of the request, one per lane
    auto page_ids = [&](const Unit& d, int pg0, int npg, int c) {
      return c + lane < npg ? p.page_table[(int64_t)d.b * p.mpps + min(pg0 + c + lane, p.mpps - 1)] : 0;
    };
    Unit dn = {};
    int pid_n0 = 0, pid_n1 = 0;
    if (n_units > 0) {
      dn = unit(0);
      const int npg = (dn.tok_end - dn.tok_begin + P - 1) / P;
      pid_n0 = page_ids(dn, dn.tok_begin / P, npg, 0);
      pid_n1 = page_ids(dn, dn.tok_begin / P, npg, 32);
    }
    for (int u = 0; u < n_units && ok; ++u) {
      const Unit d = dn;
      int pid0 = pid_n0, pid1 = pid_n1;  // pages c0 .. c0 + 31 and the 32 after them
      int c0 = 0;
      if (!warp_wait_lane0(&qempty[qs], qeph, p.status, wl)) { ok = false; break; }
      if (lane == 0) {  // q rows of this tile: T bulk copies of G consecutive heads each
        qmeta[qs] = d;
        const uint32_t bytes = (uint32_t)(p.G * D * 2);
        mbar_arrive_expect_tx(&qfull[qs], bytes * p.T);
        uint8_t* dst = sm + C::OFF_Q + qs * C::QBYTES;
        for (int t = 0; t < p.T; ++t)
          bulk_load(dst + t * bytes, p.q + (((int64_t)d.b * p.T + t) * p.Hq + (int64_t)d.h * p.G) * D, bytes, &qfull[qs]);
      }
      ++n_qfill;
      qs ^= 1; if (qs == 0) qeph ^= 1;
      const int pg0 = d.tok_begin / P;
      const int ntok = d.tok_end - d.tok_begin;
      const int npg = (ntok + P - 1) / P;
      if (lane == 0 && pg0 + npg > p.mpps) set_status(p.status, DECATTN_EDEVICE);  // row too short
      for (int k0 = 0; k0 < ntok && ok; k0 += kI4Block) {
        if (k0 / P >= c0 + 32) {
          c0 += 32;
          pid0 = pid1;
          pid1 = page_ids(d, pg0, npg, c0 + 32);
        }
        // lanes 0 .. 15: box lane of K; lanes 16 .. 31: box lane - 16 of V
        const int bx = lane & 15, kv = lane >> 4;
        const int key = k0 + bx * R;  // first key of the box, within the tile
        const bool has = bx < nbox && key < ntok;
        const int pi = min(key, ntok - 1) / P;  // the box's page: in the two chunks at hand
        const int a = __shfl_sync(0xffffffffu, pid0, (pi - c0) & 31), b2 = __shfl_sync(0xffffffffu, pid1, (pi - c0) & 31);
        int pid = pi - c0 < 32 ? a : b2;
        if (has && (pid < 0 || pid >= p.num_pages)) {
          set_status(p.status, DECATTN_EDEVICE);
          pid = 0;  // keeps the copy inside the pool; the result is flagged invalid
        }
        const int row = (pid * p.Hkv + d.h) * P + (key - pi * P);
        const uint32_t nb = (uint32_t)__popc(__ballot_sync(0xffffffffu, has));  // boxes of K and V together
        if (!warp_wait_lane0(&empty[s], eph, p.status, wl)) { ok = false; break; }
        // tests of the bounded waits leave one fill of CTA 0 out: nothing completes that stage
        if (!(blockIdx.x == 0 && n_fill == p.skip_fill)) {
          uint8_t* codes = sm + s * 2 * C::TILE;
          if (has) {
            uint8_t* wd = sm + C::OFF_WORDS + (s * 2 + kv) * C::WORDS + bx * R * 2;
            const uint16_t* ws = p.kv_words + (int64_t)kv * p.num_pages * p.Hkv * P + row;
            for (int i = 0; i < R; i += 8) cp_async_16(wd + 2 * i, ws + i);
            cp_async_mbar_arrive(&full[s]);  // before lane 0's arrival, so that the phase cannot end early
          }
          __syncwarp();
          if (lane == 0) mbar_arrive_expect_tx(&full[s], nb * (uint32_t)(R * C::RB));
          __syncwarp();
          if (has) tma_load_2d(codes + kv * C::TILE + bx * R * C::RB, kv ? &tmV : &tmK, 0, row, &full[s]);
        }
        ++n_fill;
        if (++s == STAGES) { s = 0; eph ^= 1; }
        if (k0 == 0 && u + 1 < n_units) {  // the next tile's descriptor and first page ids, ready long before use
          dn = unit(u + 1);
          const int npg1 = (dn.tok_end - dn.tok_begin + P - 1) / P;
          pid_n0 = page_ids(dn, dn.tok_begin / P, npg1, 0);
          pid_n1 = page_ids(dn, dn.tok_begin / P, npg1, 32);
        }
      }
    }
    if (ok) {
      // no more tiles: a unit with b = -1 tells the consumers to stop
      if (warp_wait_lane0(&qempty[qs], qeph, p.status, wl)) {
        if (lane == 0) {
          qmeta[qs].b = -1;
          mbar_arrive(&qfull[qs]);
        }
      } else {
        ok = false;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!ok && lane == 0) {  // a wait gave up: the copies already issued land before the CTA exits
      for (int64_t n = n_fill > STAGES ? n_fill - STAGES : 0; n < n_fill; ++n)
        mbar_wait(&full[n % STAGES], (uint32_t)((n / STAGES) & 1), nullptr, wl);
      for (int64_t n = n_qfill > 2 ? n_qfill - 2 : 0; n < n_qfill; ++n)
        mbar_wait(&qfull[n % 2], (uint32_t)((n / 2) & 1), nullptr, wl);
    }
    return;
  }

  // ======================================================================= consumer
  const int rg = (warp - 1) / KG, kg = (warp - 1) % KG;
  const int gid = lane >> 2, tig = lane & 3;
  const uint32_t smb = smem_u32(sm);
  // ldmatrix: lanes 0-7 / 8-15 address rows 0-7 / 8-15 of chunk c, lanes 16-31 the same rows of chunk c + 1
  const int ld_row = lane & 15, ld_c = lane >> 4;
  int s = kg; uint32_t fph = 0;   // this warp's next stage and its phase
  int cnt0 = 0;                   // (blocks before this tile) mod KG
  int qs = 0; uint32_t qfph = 0;
  uint32_t mph = 0;               // bit j: phase of merge buffer j's next use
  const float LN2 = 0.6931471805599453f;
  for (;;) {
    if (!__all_sync(0xffffffffu, mbar_wait(&qfull[qs], qfph, p.status, wl))) return;
    const Unit d = qmeta[qs];
    if (d.b < 0) return;  // the producer has no more tiles
    // ---- q fragments (B operand of S^T = K Q^T): column gid of tile nw = query row 8 (NQ rg + nw) + gid,
    //      scaled by 2^E per row (largest |q| in [2^14, 2^15)). Lane tig holds head dims 32 c + 8 tig .. + 7
    //      of chunk c; pair i is (i, i + 4) of those eight, as the codes of K's words pair up.
    uint32_t qf[NQ][C::NCH][4];
    float fcol[NQ][2];  // sm_scale log2(e) 2^-E of columns 2 tig, 2 tig + 1
    {
      const uint8_t* qsm = sm + C::OFF_Q + qs * C::QBYTES;
      #pragma unroll
      for (int nw = 0; nw < NQ; ++nw) {
        const int r = 8 * (NQ * rg + nw) + gid;
        const bool live = r < p.GT;
        uint4 x[C::NCH];
        float amax = 0.f;
        #pragma unroll
        for (int c = 0; c < C::NCH; ++c) {
          x[c] = live ? *reinterpret_cast<const uint4*>(qsm + ((size_t)r * D + 32 * c + 8 * tig) * 2) : make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
          #pragma unroll
          for (int i = 0; i < 4; ++i) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i]))));
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int ex = amax > 0.f ? ((__float_as_int(amax) >> 23) & 0xff) - 127 : 0;
        const int E = min(max(14 - ex, -100), 100);
        const float up = __int_as_float((127 + E) << 23), down = __int_as_float((127 - E) << 23);
        #pragma unroll
        for (int c = 0; c < C::NCH; ++c) {  // elements 0,1 | 2,3 | 4,5 | 6,7 in x, y, z, w
          qf[nw][c][0] = pack_f16(bf16_lo(x[c].x) * up, bf16_lo(x[c].z) * up);
          qf[nw][c][1] = pack_f16(bf16_hi(x[c].x) * up, bf16_hi(x[c].z) * up);
          qf[nw][c][2] = pack_f16(bf16_lo(x[c].y) * up, bf16_lo(x[c].w) * up);
          qf[nw][c][3] = pack_f16(bf16_hi(x[c].y) * up, bf16_hi(x[c].w) * up);
        }
        fcol[nw][0] = __shfl_sync(0xffffffffu, down, (2 * tig) * 4) * p.qk_scale_log2;
        fcol[nw][1] = __shfl_sync(0xffffffffu, down, (2 * tig + 1) * 4) * p.qk_scale_log2;
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&qempty[qs]);
    qs ^= 1; if (qs == 0) qfph ^= 1;

    // ---- per-column limits: key j is visible to query token t if j <= Lb - T + t
    int lim[NQ][2], lim_min = 0x7fffffff;
    #pragma unroll
    for (int nw = 0; nw < NQ; ++nw)
      #pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * (NQ * rg + nw) + 2 * tig + e;
        lim[nw][e] = r < p.GT ? d.seq_len - p.T + r / p.G : 0x7fffffff;
        lim_min = min(lim_min, lim[nw][e]);
      }
    lim_min = __reduce_min_sync(0xffffffffu, lim_min);
    const int safe_end = min(d.tok_end, lim_min + 1);  // keys below this need no mask

    float o[NQ][D / 16][4];
    float mrow[NQ][2], lrow[NQ][2];
    int eref = 16;  // biased exponent that P s^V is relative to (the largest s^V so far; at least 2^-111)
    #pragma unroll
    for (int nw = 0; nw < NQ; ++nw) {
      #pragma unroll
      for (int mt = 0; mt < D / 16; ++mt) o[nw][mt][0] = o[nw][mt][1] = o[nw][mt][2] = o[nw][mt][3] = 0.f;
      mrow[nw][0] = mrow[nw][1] = -INFINITY;
      lrow[nw][0] = lrow[nw][1] = 0.f;
    }

    const int nblk = (d.tok_end - d.tok_begin + kI4Block - 1) / kI4Block;
    const int first = kg >= cnt0 ? kg - cnt0 : kg - cnt0 + KG;  // this warp's first block of the tile
    for (int blk = first; blk < nblk; blk += KG) {
      if (!__all_sync(0xffffffffu, mbar_wait(&full[s], fph, p.status, wl))) return;
      const int kbase = d.tok_begin + blk * kI4Block;
      const uint32_t ks = smb + s * 2 * C::TILE, vs = ks + C::TILE;
      const uint32_t kwd = smb + C::OFF_WORDS + s * 2 * C::WORDS, vwd = kwd + C::WORDS;
      const bool need_mask = kbase + kI4Block > safe_end;  // warp-uniform
      const int nkey = d.tok_end - kbase;                  // keys of the block that exist
      // ---- S^T = K Q^T: four 16-key tiles
      float sv[4][NQ][4];
      #pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
        uint32_t w0 = lds_u16(kwd + 2 * (16 * mt + gid)), w1 = lds_u16(kwd + 2 * (16 * mt + 8 + gid));
        if (need_mask) {  // behind the last key the words are anything
          if (16 * mt + gid >= nkey) w0 = 0;
          if (16 * mt + 8 + gid >= nkey) w1 = 0;
        }
        const uint32_t z0 = (w0 & 15u) * 0x10001u, z1 = (w1 & 15u) * 0x10001u;
        const uint32_t nl0 = int4_nlo(z0), nh0 = int4_nhi(z0), nl1 = int4_nlo(z1), nh1 = int4_nhi(z1);
        float acc[NQ][4];
        #pragma unroll
        for (int nw = 0; nw < NQ; ++nw) acc[nw][0] = acc[nw][1] = acc[nw][2] = acc[nw][3] = 0.f;
        #pragma unroll
        for (int c = 0; c < C::NCH; c += 2) {
          uint32_t r[4];
          ldsm_x4(ks + C::off(16 * mt + ld_row, c + ld_c), r[0], r[1], r[2], r[3]);
          #pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t x0[4], x1[4];
            int4_to_f16(r[2 * h], nl0, nh0, x0);
            int4_to_f16(r[2 * h + 1], nl1, nh1, x1);
            const uint32_t a0[4] = {x0[0], x1[0], x0[1], x1[1]}, a1[4] = {x0[2], x1[2], x0[3], x1[3]};
            #pragma unroll
            for (int nw = 0; nw < NQ; ++nw) {
              mma_f16(acc[nw], a0, qf[nw][c + h][0], qf[nw][c + h][1]);
              mma_f16(acc[nw], a1, qf[nw][c + h][2], qf[nw][c + h][3]);
            }
          }
        }
        const float s0 = int4_scale(w0), s1 = int4_scale(w1);
        #pragma unroll
        for (int nw = 0; nw < NQ; ++nw) {
          #pragma unroll
          for (int i = 0; i < 4; ++i) {
            sv[mt][nw][i] = acc[nw][i] * (i < 2 ? s0 : s1);
            if (need_mask) {
              const int j = 16 * mt + gid + (i >> 1) * 8;
              if (j >= nkey || kbase + j > lim[nw][i & 1]) sv[mt][nw][i] = -INFINITY;
            }
          }
        }
      }
      // ---- the block's largest V scale (its bf16 exponent field, at bit 7 of a word); a NaN row does not count
      uint32_t vmax;
      {
        uint32_t w = lds_u32(vwd + 4 * lane);
        if (need_mask) {
          if (2 * lane >= nkey) w = 0;
          else if (2 * lane + 1 >= nkey) w &= 0xffffu;
        }
        const uint32_t e0 = (w >> 7) & 0xffu, e1 = (w >> 23) & 0xffu;
        vmax = __reduce_max_sync(0xffffffffu, max(e0 == 0xffu ? 0u : e0, e1 == 0xffu ? 0u : e1));
      }
      // ---- online softmax (log2 domain, fp32 state)
      const int enew = max(eref, (int)vmax);
      bool grew = enew > eref;
      float alpha[NQ][2], muse[NQ][2];
      #pragma unroll
      for (int nw = 0; nw < NQ; ++nw)
        #pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(sv[0][nw][e], sv[0][nw][e + 2]);
          #pragma unroll
          for (int mt = 1; mt < 4; ++mt) mx = fmax3(mx, sv[mt][nw][e], sv[mt][nw][e + 2]);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16)) * fcol[nw][e];  // the factor is positive
          const float mnew = fmaxf(mrow[nw][e], mx);
          grew |= mnew > mrow[nw][e];
          muse[nw][e] = mnew == -INFINITY ? 0.f : mnew;
          alpha[nw][e] = fast_exp2(mrow[nw][e] - muse[nw][e]);
          lrow[nw][e] *= alpha[nw][e];
          mrow[nw][e] = mnew;
        }
      if (__any_sync(0xffffffffu, grew)) {
        const int de = eref - enew;  // <= 0
        const float es = de < -126 ? 0.f : __int_as_float((127 + de) << 23);
        #pragma unroll
        for (int nw = 0; nw < NQ; ++nw) {
          const float a0 = alpha[nw][0] * es, a1 = alpha[nw][1] * es;
          #pragma unroll
          for (int mt = 0; mt < D / 16; ++mt) {
            o[nw][mt][0] *= a0; o[nw][mt][1] *= a1;
            o[nw][mt][2] *= a0; o[nw][mt][3] *= a1;
          }
        }
        eref = enew;
      }
      const float pf = __int_as_float((2 * 127 + kI4PExp - eref) << 23);  // 2^kI4PExp / 2^(eref - 127); eref <= 254
      // ---- O^T += V^T P^T, 16 keys at a time
      #pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
        uint32_t w0 = lds_u16(vwd + 2 * (16 * mt + gid)), w1 = lds_u16(vwd + 2 * (16 * mt + 8 + gid));
        uint32_t pa = lds_u32(vwd + 2 * (16 * mt + 2 * tig)), pb = lds_u32(vwd + 2 * (16 * mt + 8 + 2 * tig));
        if (need_mask) {  // zero points are whole numbers whatever the words hold; the scales must not be used
          if (16 * mt + gid >= nkey) w0 = 0;
          if (16 * mt + 8 + gid >= nkey) w1 = 0;
        }
        const float s0 = int4_scale(w0) * pf, s1 = int4_scale(w1) * pf;
        uint32_t bp[NQ][2];
        #pragma unroll
        for (int nw = 0; nw < NQ; ++nw) {
          float pv[4];
          #pragma unroll
          for (int i = 0; i < 4; ++i) pv[i] = fast_exp2(fmaf(sv[mt][nw][i], fcol[nw][i & 1], -muse[nw][i & 1]));
          lrow[nw][0] += pv[0] + pv[2];
          lrow[nw][1] += pv[1] + pv[3];
          float x[4] = {pv[0] * s0, pv[1] * s0, pv[2] * s1, pv[3] * s1};
          if (need_mask) {  // a NaN row stays out of the rows that do not see it
            #pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = sv[mt][nw][i] == -INFINITY ? 0.f : x[i];
          }
          bp[nw][0] = movmatrix_t(pack_f16(x[0], x[1]));
          bp[nw][1] = movmatrix_t(pack_f16(x[2], x[3]));
        }
        const uint32_t nla = int4_nlo(pa), nha = int4_nhi(pa), nlb = int4_nlo(pb), nhb = int4_nhi(pb);
        #pragma unroll
        for (int c = 0; c < C::NCH; c += 2) {
          uint32_t r[4];
          ldsm_x4_t(vs + C::off(16 * mt + ld_row, c + ld_c), r[0], r[1], r[2], r[3]);
          #pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t xa[4], xb[4];
            int4_to_f16(r[2 * h], nla, nha, xa);
            int4_to_f16(r[2 * h + 1], nlb, nhb, xb);
            // M-row gid of tile (c + h, jj): head dim 32 (c + h) + 4 gid + 2 jj, M-row gid + 8: the next one
            const uint32_t a0[4] = {xa[0], xa[1], xb[0], xb[1]}, a1[4] = {xa[2], xa[3], xb[2], xb[3]};
            #pragma unroll
            for (int nw = 0; nw < NQ; ++nw) {
              mma_f16(o[nw][2 * (c + h)], a0, bp[nw][0], bp[nw][1]);
              mma_f16(o[nw][2 * (c + h) + 1], a1, bp[nw][0], bp[nw][1]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
      s += KG;
      if (s >= STAGES) { s -= STAGES; fph ^= 1; }
    }

    // ---- the key groups' states of this tile: group 0 takes the others' (buffer j: written by group j + 1
    //      only and read by group 0 only, so that both sides see every phase of its barriers)
    #pragma unroll
    for (int j = 0; j < KG - 1; ++j) {
      const int fj = j + 1 >= cnt0 ? j + 1 - cnt0 : j + 1 - cnt0 + KG;  // that group's first block of the tile
      if (fj >= nblk) continue;
      const int mb = rg * C::NMERGE + j;
      float* buf = reinterpret_cast<float*>(sm + C::OFF_MERGE + mb * C::MERGE) + lane;
      const uint32_t ph = (mph >> j) & 1u;
      mph ^= 1u << j;
      if (kg == j + 1) {
        if (!__all_sync(0xffffffffu, mbar_wait(&mempty[mb], ph ^ 1u, p.status, wl))) return;
        int i = 0;
        #pragma unroll
        for (int nw = 0; nw < NQ; ++nw) {
          #pragma unroll
          for (int mt = 0; mt < D / 16; ++mt)
            #pragma unroll
            for (int k = 0; k < 4; ++k) buf[32 * i++] = o[nw][mt][k];
          #pragma unroll
          for (int e = 0; e < 2; ++e) {
            buf[32 * i++] = mrow[nw][e];
            buf[32 * i++] = lrow[nw][e];
          }
        }
        buf[32 * i] = __int_as_float(eref);
        __syncwarp();
        if (lane == 0) mbar_arrive(&mfull[mb]);
      } else if (kg == 0) {
        if (!__all_sync(0xffffffffu, mbar_wait(&mfull[mb], ph, p.status, wl))) return;
        const int eo = __float_as_int(buf[32 * (C::MREGS - 1)]), em = max(eref, eo);
        const float ea = eref - em < -126 ? 0.f : __int_as_float((127 + eref - em) << 23);
        const float eb = eo - em < -126 ? 0.f : __int_as_float((127 + eo - em) << 23);
        eref = em;
        int i = 0;
        #pragma unroll
        for (int nw = 0; nw < NQ; ++nw) {
          float wa[2], wb[2];
          const int im = i + D / 16 * 4;
          #pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float mo = buf[32 * (im + 2 * e)], lo = buf[32 * (im + 2 * e + 1)];
            const float m = fmaxf(mrow[nw][e], mo), mu = m == -INFINITY ? 0.f : m;
            wa[e] = fast_exp2(mrow[nw][e] - mu);
            wb[e] = fast_exp2(mo - mu);
            lrow[nw][e] = lrow[nw][e] * wa[e] + lo * wb[e];
            mrow[nw][e] = m;
            wa[e] *= ea;
            wb[e] *= eb;
          }
          #pragma unroll
          for (int mt = 0; mt < D / 16; ++mt)
            #pragma unroll
            for (int k = 0; k < 4; ++k) o[nw][mt][k] = o[nw][mt][k] * wa[k & 1] + buf[32 * i++] * wb[k & 1];
          i += 4;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&mempty[mb]);
      }
    }
    cnt0 = (cnt0 + nblk) % KG;
    if (kg != 0) continue;

    // ---- epilogue: row sums, normalise, store
    const float unref = __int_as_float((eref - kI4PExp) << 23);  // 2^(eref - 127) / 2^kI4PExp; eref >= 16
    #pragma unroll
    for (int nw = 0; nw < NQ; ++nw)
      #pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = lrow[nw][e];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        const int r = 8 * (NQ * rg + nw) + 2 * tig + e;
        if (r >= p.GT) continue;
        const float inv = l == 0.f ? 0.f : unref / l;
        const float lse_v = l == 0.f ? -INFINITY : (mrow[nw][e] + __log2f(l)) * LN2;
        const int t = r / p.G, g = r - t * p.G;
        if (d.slot < 0) {
          const int64_t row = ((int64_t)d.b * p.T + t) * p.Hq + (int64_t)d.h * p.G + g;
          uint16_t* dst = p.out_bf16 + row * D;
          #pragma unroll
          for (int c = 0; c < C::NCH; ++c)
            *reinterpret_cast<uint2*>(dst + 32 * c + 4 * gid) =
                make_uint2(pack_bf16(o[nw][2 * c][e] * inv, o[nw][2 * c][2 + e] * inv),
                           pack_bf16(o[nw][2 * c + 1][e] * inv, o[nw][2 * c + 1][2 + e] * inv));
          if (gid == 0) p.lse[row] = lse_v;
        } else {
          const int64_t row = (int64_t)d.slot * p.GT + r;
          float* dst = p.part_o + row * D;
          #pragma unroll
          for (int c = 0; c < C::NCH; ++c)
            *reinterpret_cast<float4*>(dst + 32 * c + 4 * gid) =
                make_float4(o[nw][2 * c][e] * inv, o[nw][2 * c][2 + e] * inv, o[nw][2 * c + 1][e] * inv,
                            o[nw][2 * c + 1][2 + e] * inv);
          if (gid == 0) p.part_lse[row] = lse_v;
        }
      }
  }
}

// ------------------------------------------------------------------ host side
template <int D, int NQ, int RG, int KG, int CPS>
static cudaError_t launch_i4(const SplitParams& p, const CUtensorMap& tmK, const CUtensorMap& tmV, cudaStream_t st) {
  using C = I4Cfg<D, NQ, RG, KG, CPS>;
  auto fn = split_int4_kernel<D, NQ, RG, KG, CPS>;
  if (!ensure_smem_attr((const void*)fn, C::ALLOC)) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.n_bins);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::ALLOC;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // overlaps our prologue with the planner
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, p, tmK, tmV);
}

template <int D>
static cudaError_t launch_i4_gt(const SplitParams& p, const CUtensorMap& tmK, const CUtensorMap& tmV, cudaStream_t st) {
  if (p.GT <= 8) return launch_i4<D, 1, 1, 2, 4>(p, tmK, tmV, st);
  if (p.GT <= 16) return launch_i4<D, 2, 1, 4, 2>(p, tmK, tmV, st);
  if (p.GT <= 32) return launch_i4<D, 2, 2, 2, 2>(p, tmK, tmV, st);
  return launch_i4<D, 2, 4, 1, 2>(p, tmK, tmV, st);
}

bool split_int4_supported(int D, int GT) { return GT >= 1 && GT <= kMaxGT && (D == 64 || D == 128); }

int split_int4_box_rows(int P) { return P % 64 == 0 ? 64 : P % 32 == 0 ? 32 : 16; }

cudaError_t launch_split_int4(const SplitParams& p, const CUtensorMap& tmK, const CUtensorMap& tmV, int D, cudaStream_t st) {
  if (!split_int4_supported(D, p.GT)) return cudaErrorInvalidValue;
  return D == 128 ? launch_i4_gt<128>(p, tmK, tmV, st) : launch_i4_gt<64>(p, tmK, tmV, st);
}

}  // namespace decattn
