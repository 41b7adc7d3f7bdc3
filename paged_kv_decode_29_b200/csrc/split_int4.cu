// split_int4.cu -- the split kernel over an INT4 cache (DECATTN_KV_INT4; int4.cuh has the format): persistent
// CTAs walk the bins of the plan, as split.cu does for bf16 and E4M3 pages.
//
// Mathematics, for the query rows r of a KV head and the keys j of a tile, with row scales s and zero
// points z of K and V:
//   S_jr = s^K_j (<c^K_j, q_r> - z^K_j <1, q_r>),  P_jr = 2^(S_jr sm_scale log2 e - m_r),  l_r = sum_j P_jr,
//   X_jr = P_jr s^V_j,  O_r = sum_j X_jr c^V_j - sum_j X_jr z^V_j.
// The tensor cores see codes, untouched but for a mask: a code in bits 0 .. 3 or 4 .. 7 of a half-word is the f16
// number c 2^-24 or c 2^-20 (a subnormal). Scales and zero points act on one score or one weight instead of on
// head_dim elements.
//  * q_r, of any magnitude, is scaled by a power of two per row, so that its eight significant bits are exact in f16 down
//    to 2^-24 of the row's largest element, and within 2^-35 of that below.
//  * X is rounded once to f16, relative to a reference of m and of s^V (a power of two near the largest s^V
//    is divided out, and put back at the end): off by at most 2^-11 of itself, an eighth of the rounding that the bf16
//    output gets anyway, or by 2^-22 of the row's largest X. That holds while a tile's V scales lie within 2^kI4Window of
//    one another; a tile with others has a reference of X for each row, the largest X that the row has seen, and new
//    references in every block ("wide": the key whose scale is far out may have no weight, or be hidden from the row).
//    Both sums of O take the rounded X, so a key's part of an element is off by that share of X (c - z), and a
//    channel of zeros stays one (but for the fp32 sums). m, l, the zero points' sum, O and the partials are fp32.
//
// CTA = W = head_dim / 32 warps, all alike. The KV stream is cut into blocks of 64 keys. Of every block warp w
// copies keys 64 w / W .. into the rings, computes their scores, and of O holds head dims 32 w .. 32 w + 31 over
// all keys: every code is decoded once, a lane holds 8 NQ numbers of O for 8 NQ query rows, and nothing is merged
// at a tile's end. X goes from the warps that have the scores to all warps through shared memory (stmatrix.trans
// turns it into the B operand's layout).
// More than 16 query rows go to several CTAs, 16 rows each, which walk the same bins side by side (neighbours in the
// grid: K and V come from L2 for all but one). They decode every code again, but run 16 warps a multiprocessor: 33 to
// 64 rows held by one CTA (8 warps a multiprocessor, 255 registers) took 46.3 us where this takes 29.7 (56 rows a KV
// head, 35 requests of 7602 keys together), 17 to 32 rows 31.0 against 27.3.
//  * One barrier per block, after its scores. It carries a vote whether a score passes its reference by more than
//    2^kI4Tau, or a V scale lies outside the window; if so the CTA takes the exact maxima, else they stay.
//    It also makes X of the block before visible, whose product comes next, beside the exponentials of this one.
//  * The same barrier paces the copies (cp.async): at block g, K (and the row words) of block g + kI4Stages and V
//    of block g + kI4Stages - 2 go into the places that it has freed, so that every copy has kI4Stages - 1 blocks'
//    time to land, across tiles too. No other signal is needed, and there is nothing to wait for without a bound.
//  * keys sit on the MMA's M side in the first product (S^T = K Q^T), head dims in the second (O^T = V^T X^T).
//  * K: ldmatrix gives a lane 8 codes of a key; code pairs (i, i + 4) of such a word are one f16 pair
//    of the A operand (the order of head dims in the sum is free: q is laid out to match).
//  * V: ldmatrix.trans gives a lane 4 head dims of 2 neighbouring keys in a word, whose code pairs
//    (i, i + 4) are one f16 pair of V^T. So both operands come from the same 5 instructions per word.
//
// Measured (kernel times; 32 requests of 4096 tokens, 4 query heads to a KV head: 139 MB, 21.5 us at the copy rate):
// 42.2 us with the combine. Bound by instruction issue and its latencies, not by DRAM: 290 instructions a warp and block,
// half the issue slots and 48% of the ALU pipe busy at 16 warps a multiprocessor; an earlier form without its
// copies took 38.5 us (41 with them), without its arithmetic 29. Other forms measured on the way, same case: a TMA producer warp with
// two consumer warps that split the keys 57; four warps that split the head dims behind a TMA producer 48.5 (16-key
// pages: the producer issues eight copies a block, each a loop over lanes); codes as E4M3 numbers for
// mma.m16n8k32 62.9 (warp MMAs on E4M3 convert their operands to f16: the conversion pipe was 77% busy).
#include "common.cuh"
#include "int4.cuh"

namespace decattn {

constexpr int kI4Block = 64;   // keys per block
constexpr int kI4Stages = 4;   // places of the K ring and of the V ring (a power of two)
constexpr int kI4Tau = 5;      // P <= 2^kI4Tau
constexpr int kI4XExp = 9;     // X < 2^(kI4Tau + 1 + kI4XExp) = 2^15
// V scales that a tile takes with one reference: up to 2^kI4Room above the largest of its first block, and 2^kI4Window in
// all. The largest X of a row is then 2^(kI4XExp - kI4Window) at least, and f16's subnormal rounding 2^-25.
constexpr int kI4Room = 4;
constexpr int kI4Window = 12;
constexpr int kI4Least = kI4XExp + 1;  // least exponent of X's reference: 2^(kI4Least - kI4XExp - 127) is a normal number
constexpr float kI4Far = 0x1p20f;  // |m| from which S - m is taken the other way: here m is off by up to 2^-4, and P by 2^(2^-4)
constexpr int kI4Queue = 64;   // tile descriptors at hand: 32 are fetched at a time

template <int D, int NQ>
struct I4Cfg {
  static constexpr int W = D / 32;                            // warps
  static constexpr int THREADS = 32 * W;
  static constexpr int MT = kI4Block / 16 / W;                // 16-key groups of a block per warp
  static constexpr int RB = D / 2;                            // bytes of a row's codes
  static constexpr int NCH = RB / 16;                         // 16-byte chunks of a row (32 head dims each)
  static constexpr int TILE = kI4Block * RB;                  // K (or V) codes of a block
  static constexpr int WORDS = 2 * kI4Block;                  // bytes of K (or V) row words of a block
  static constexpr int XBUF = 8 * NQ * 2 * kI4Block;          // X of a block: f16 [8 NQ rows][64 keys]
  static constexpr int QFRAG = NQ * NCH * 512;                // q as B operands: 16 bytes a lane, 8 rows and chunk
  static constexpr bool QREG = NQ == 1;                       // q operands held in registers, else read from QFRAG
  static constexpr int OFF_V = kI4Stages * TILE;              // after the K ring
  static constexpr int OFF_WORDS = 2 * kI4Stages * TILE;      // [stage][K, V][64] words
  static constexpr int OFF_X = OFF_WORDS + kI4Stages * 2 * WORDS;  // [buffer]
  static constexpr int OFF_QFRAG = OFF_X + 2 * XBUF;
  static constexpr int OFF_QUEUE = OFF_QFRAG + QFRAG;
  static constexpr int OFF_XCH = OFF_QUEUE + kI4Queue * (int)sizeof(Unit);
  static constexpr int XCH = 4 * (W * 5 * 8 * NQ + 4 * 8 * NQ + 2 * W + 3);  // see the pointers into it
  static constexpr int BYTES = (OFF_XCH + XCH + 15) / 16 * 16;
  static constexpr int ALLOC = BYTES + 128;                   // slack to align the base to 128
  // byte offset of (row r, 16-byte chunk c) in a block's K or V codes: the chunks of rows 64 or 32 bytes long are
  // permuted so that the 8 rows of an ldmatrix lie in 8 different bank groups
  __device__ static __forceinline__ uint32_t off(int r, int c) {
    return RB == 64 ? (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4)) : (uint32_t)(r * 32 + ((c ^ ((r >> 2) & 1)) << 4));
  }
};

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// ... by the lanes for which `does` holds
__device__ __forceinline__ void cp_async_16_if(uint32_t dst, const void* src, bool does) {
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %2, 0;\n @p cp.async.cg.shared.global [%0], [%1], 16;\n}" ::"r"(dst), "l"(src),
               "r"((uint32_t)does)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ void lds_128(uint32_t addr, uint32_t (&v)[4]) {
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr));
}
// A number that every lane of the warp holds, known to the compiler as such: branches on it need no
// reconvergence and it takes a uniform register.
__device__ __forceinline__ int uniform(int x) { return __reduce_max_sync(0xffffffffu, x); }
// stmatrix, transposed: matrix m's row i (8 f16) goes to the address that lane 8 m + i gives.
__device__ __forceinline__ void stsm_x2_t(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("stmatrix.sync.aligned.m8n8.x2.trans.shared.b16 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
// Barrier over the CTA, with a vote.
__device__ __forceinline__ bool bar_or(bool x) { return __syncthreads_or(x) != 0; }

// All tiles of the CTA. WIDE: with a reference of X for each row where the V scales of a tile need it, with queries of
// 2^104 and more, and with differences of scores taken before their factor where S and m are so large that their roundings
// differ. Without it such a tile is left wrong, and the return value asks the CTA for a second pass that has it. (One
// pass for both is slower where no tile needs it, as the hot loop is out of registers: 32 requests of 4096 tokens 42.2 ->
// 43.2 us, 16 query rows a KV head 105 -> 113. The second pass costs its CTAs the time once more, twice where every tile
// is wide: 44 -> 91 -> 123. Ending the first pass at its first wide tile, and starting the second one there, costs
// the ordinary case 0.7 us.)
template <int D, int NQ, bool WIDE>
__device__ __forceinline__ bool i4_pass(const SplitInt4Params& p) {
  using C = I4Cfg<D, NQ>;
  constexpr int W = C::W, MT = C::MT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  const int lane = threadIdx.x & 31, w = uniform((int)threadIdx.x >> 5);
  const int gid = lane >> 2, tig = lane & 3;
  const uint32_t smb = smem_u32(sm);
  Unit* queue = reinterpret_cast<Unit*>(sm + C::OFF_QUEUE);
  float* xmax = reinterpret_cast<float*>(sm + C::OFF_XCH);  // [warp][8 NQ]
  float* xsum = xmax + W * 8 * NQ;                          // [l, zero points][8 NQ][warp]
  float* qrow = xsum + W * 2 * 8 * NQ;                      // [score factor, <1, q>, one over the factor, 2^32 or 1][8 NQ]
  int* xexp = reinterpret_cast<int*>(qrow + 4 * 8 * NQ);    // [largest, least][warp]
  int* n_queued = xexp + 2 * W;                             // [2]: of every other refill
  int* redo = n_queued + 2;                                 // a second pass is needed
  float* xtop = reinterpret_cast<float*>(redo + 1);         // [8 NQ][warp]: of a wide tile, the largest X as an exponent
  int* xrow = redo + 1 + W * 8 * NQ + w * 8 * NQ;           // [warp][8 NQ]: of a wide tile, the references of X
  if (threadIdx.x == 0) *redo = 0;  // many barriers before its first use

  // ======================================================================= tiles
  // The CTA's query rows: r0 .. of every KV head. Its tiles: those of bins blockIdx.x / groups, + gridDim.x / groups,
  // ..., numbered through; descriptor u at queue[u % 64].
  const int groups = (p.GT + 8 * NQ - 1) / (8 * NQ);
  const int r0 = 8 * NQ * ((int)blockIdx.x % groups);
  int bin = (int)blockIdx.x / groups, bin_j = 0;  // warp 0: the next descriptor to fetch
  int total = 0;                         // descriptors fetched so far
  bool last = false;                     // there are no more
  int refills = 0;
  auto refill = [&] {                    // every warp calls it at the same point
    if (w == 0) {
      const PlanHeader* h = reinterpret_cast<const PlanHeader*>(p.plan);
      int n = 0;
      if (h->magic == kPlanMagic && h->status == DECATTN_OK && h->n_bins == p.n_bins && h->batch == p.B &&
          h->n_kv_heads == p.Hkv && h->tile_len == p.tile_len && h->sparse == p.sparse) {
        while (n == 0 && bin < p.n_bins) {
          n = min(plan_bin_size(p.plan, *h, bin) - bin_j, 32);
          if (lane < n) {
            const Unit u = h->sparse ? plan_unit_sparse(p.plan, *h, p.seq_lens, bin, bin_j + lane)
                                     : plan_unit(p.plan, *h, p.seq_lens, bin, bin_j + lane);
            if ((int64_t)u.tok_end > (int64_t)p.mpps * p.P) set_status(p.status, DECATTN_EDEVICE);  // table too short
            queue[(total + lane) % kI4Queue] = u;
          }
          bin_j += max(n, 0);
          if (n <= 0) {
            n = 0;
            bin += (int)gridDim.x / groups;
            bin_j = 0;
          }
        }
      } else if (lane == 0) {
        set_status(p.status, h->magic == kPlanMagic && h->status != DECATTN_OK ? h->status : DECATTN_EINVAL);
      }
      if (lane == 0) n_queued[refills & 1] = total + n;
    }
    __syncthreads();
    const int n = uniform(n_queued[refills & 1]);
    ++refills;
    last = n == total;
    total = n;
  };
  auto n_blocks = [&](const Unit& d) { return max((d.tok_end - d.tok_begin + kI4Block - 1) / kI4Block, 1); };

  // ======================================================================= copies
  // Page ids are read 32 blocks at a time, one chunk ahead: lane l holds, of block l of the chunk, the rows in the
  // pools of this warp's 16-key groups. Past a tile's end, and past the last tile, rows 0 .. 15 of the pools are
  // copied and masked or never looked at: a block's copies need no branch.
  int f_unit = -1, f_blk = 0, f_nblk = 0;  // the chunk after the next: of tile f_unit, from block f_blk
  int c_len = 0, c_at = 0, c_row[MT];      // the chunk that is being copied, its next block
  int n_len = 0, n_row[MT];                // the next one
  auto fetch_chunk = [&] {
    asm volatile("" ::: "memory");  // nothing of this is done ahead, in every block
    n_len = 0;
    if (f_blk >= f_nblk) {
      if (f_unit + 1 >= total && !last) refill();
      if (f_unit + 1 >= total) return;
      ++f_unit;
      f_blk = 0;
      f_nblk = uniform(n_blocks(queue[f_unit % kI4Queue]));
    }
    const Unit& u = queue[f_unit % kI4Queue];
    n_len = min(32, f_nblk - f_blk);
    #pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int key = u.tok_begin + kI4Block * (f_blk + lane) + 16 * (w * MT + m);
      n_row[m] = 0;
      if (lane < n_len && (uint32_t)key < (uint32_t)u.tok_end) {
        const int pg = key / p.P;
        int id = p.page_table[(int64_t)u.b * p.mpps + min(pg, p.mpps - 1)];
        if (id < 0 || id >= p.num_pages) {
          set_status(p.status, DECATTN_EDEVICE);
          id = 0;  // keeps the copies inside the pools; the result is flagged invalid
        }
        n_row[m] = (id * p.Hkv + u.h) * p.P + (key - pg * p.P);
      }
    }
    f_blk += n_len;
  };
  // Rows of the next block's groups.
  auto next_rows = [&](int (&row)[MT]) {
    if (c_at == c_len) {
      c_len = n_len > 0 ? n_len : -1;  // -1: no more blocks, and never again here
      c_at = 0;
      #pragma unroll
      for (int m = 0; m < MT; ++m) c_row[m] = n_len > 0 ? n_row[m] : 0;
      if (n_len > 0) fetch_chunk();
    }
    #pragma unroll
    for (int m = 0; m < MT; ++m) row[m] = __shfl_sync(0xffffffffu, c_row[m], c_at);
    ++c_at;
  };
  // A group's codes: 16 rows in a row in memory, 512 bytes per instruction
  constexpr int LPR = C::RB / 16, RPI = 32 / LPR;  // lanes per row, rows per instruction
  const uint32_t cp_off = C::off(16 * w * MT + lane / LPR, lane % LPR);
  const uint8_t* const k_src = p.k_codes + 16 * lane;
  const uint8_t* const v_src = p.v_codes + 16 * lane;
  auto copy_codes = [&](uint32_t ring, const uint8_t* pool, const int (&row)[MT]) {
    #pragma unroll
    for (int m = 0; m < MT; ++m) {
      const uint8_t* src = pool + (int64_t)row[m] * C::RB;
      #pragma unroll
      for (int i = 0; i < 16 / RPI; ++i) cp_async_16(ring + (16 * m + i * RPI) * C::RB, src + i * 512);
    }
  };
  // lanes 0, 1: K words of a group, lanes 2, 3: V words
  const uint16_t* w_src = p.kv_words + (int64_t)((lane >> 1) & 1) * p.num_pages * p.Hkv * p.P + 8 * (lane & 1);
  const uint32_t cpw_off = C::OFF_WORDS + ((lane >> 1) & 1) * C::WORDS + 32 * w * MT + 16 * (lane & 1);
  int row0[MT], row1[MT];        // rows of the two blocks whose K is copied and whose V is not
  #pragma unroll
  for (int m = 0; m < MT; ++m) row0[m] = row1[m] = 0;
  auto copy_step = [&](uint32_t place, bool with_v) {  // K into this place of its ring, V into the one two back
    int row[MT];
    next_rows(row);
    copy_codes(smb + cp_off + place * C::TILE, k_src, row);
    #pragma unroll
    for (int m = 0; m < MT; ++m)
      cp_async_16_if(smb + cpw_off + place * 2 * C::WORDS + 32 * m, w_src + row[m], lane < 4);
    if (with_v) copy_codes(smb + cp_off + C::OFF_V + ((place + kI4Stages - 2) % kI4Stages) * C::TILE, v_src, row0);
    cp_async_commit();
    #pragma unroll
    for (int m = 0; m < MT; ++m) {
      row0[m] = row1[m];
      row1[m] = row[m];
    }
  };

  // ======================================================================= compute
  // this lane's offsets: K rows (lanes 0-7 / 8-15 address rows 0-7 / 8-15 of a chunk, lanes 16-31 the same rows of
  // the next), V rows, its row words, and X written (lanes 0-7 / 8-15: rows 0-7 of 8 keys each) and read
  const uint32_t k_off = C::off(16 * w * MT + (lane & 15), lane >> 4), v_off = C::OFF_V + C::off(lane, w);
  const uint32_t w_off = C::OFF_WORDS + 2 * (16 * w * MT + gid);
  const uint32_t x_wr = C::OFF_X + (lane & 7) * 128 + (((2 * w * MT + ((lane >> 3) & 1)) ^ (lane & 7)) << 4);
  const uint32_t x_rd = C::OFF_X + (lane & 7) * 128 + (((lane >> 3) ^ (lane & 7)) << 4);
  const float LN2 = 0.6931471805599453f;

  // q of a tile: D / 8 lanes take a row, 8 head dims each
  constexpr int LPQ = D / 8, RPP = 32 / LPQ, PASSES = 8 * NQ / W / RPP;
  // query row r of a KV head is row (r / G) Hq + r % G behind the first one of (request, head); -1: no such row
  auto row_of = [&](int r) { return r < p.GT ? r / p.G * p.Hq + r % p.G : -1; };
  auto first_row = [&](const Unit& u) { return (int64_t)u.b * p.T * p.Hq + (int64_t)u.h * p.G; };
  uint4 qx[PASSES];
  int q_rows[PASSES];
  #pragma unroll
  for (int i = 0; i < PASSES; ++i) q_rows[i] = row_of(r0 + (w * PASSES + i) * RPP + lane / LPQ);
  auto load_q = [&](const Unit& u) {
    const uint16_t* src = p.q + first_row(u) * D + 8 * (lane % LPQ);
    #pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      qx[i] = make_uint4(0, 0, 0, 0);
      if (q_rows[i] >= 0) qx[i] = *reinterpret_cast<const uint4*>(src + (int64_t)q_rows[i] * D);
    }
  };
  int o_rows[NQ][2];  // of this lane's columns of O^T
  #pragma unroll
  for (int nw = 0; nw < NQ; ++nw)
    #pragma unroll
    for (int e = 0; e < 2; ++e) o_rows[nw][e] = row_of(r0 + 8 * nw + 2 * tig + e);

  fetch_chunk();
  if (f_unit < 0) return false;  // no tile
  load_q(queue[0]);        // beside the first copies
  #pragma unroll
  for (int i = 0; i < kI4Stages; ++i) copy_step(i, i >= 2);
  cp_async_wait<kI4Stages - 1>();
  __syncthreads();  // the first block's K is there

  uint32_t g = 0;   // blocks so far: block g is at place g % kI4Stages of the rings
  for (int unit = 0; unit <= f_unit; ++unit) {
    Unit d = queue[unit % kI4Queue];
    d.b = uniform(d.b);
    d.h = uniform(d.h);
    d.tok_begin = uniform(d.tok_begin);
    d.tok_end = uniform(d.tok_end);
    d.seq_len = uniform(d.seq_len);
    d.slot = uniform(d.slot);
    // ---- q as B operands of S^T = K Q^T, made by the warps together: column gid of tile nw = query row 8 nw + gid,
    //      scaled by 2^E per row (largest |q| in [2^14, 2^15)). Lane tig of the operand holds head dims
    //      32 c + 8 tig .. + 7 of chunk c: the pairs (i, i + 4) of those eight in register i, as the codes of K's
    //      words pair up, those that meet a code times 16 over 16. Here D / 8 lanes take a row, 8 head dims each.
    {
      #pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        const int row = (w * PASSES + i) * RPP + lane / LPQ, sg = lane % LPQ;
        // largest bit pattern without its sign: infinities and NaNs come out on top
        uint32_t amax = __vmaxu2(__vmaxu2(qx[i].x & 0x7fff7fffu, qx[i].y & 0x7fff7fffu),
                                 __vmaxu2(qx[i].z & 0x7fff7fffu, qx[i].w & 0x7fff7fffu));
        amax = max(amax & 0xffffu, amax >> 16);
        #pragma unroll
        for (int k = 1; k < LPQ; k <<= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, k));
        // largest element in [2^14, 2^15); below 2^-106 less, where 2^120 leaves every bf16 number exact all the same
        const int E = amax == 0 ? 0 : min(14 + 127 - (int)(amax >> 7), 120);
        const float up = __int_as_float((127 + E) << 23);
        float v[8] = {bf16_lo(qx[i].x), bf16_hi(qx[i].x), bf16_lo(qx[i].y), bf16_hi(qx[i].y),
                      bf16_lo(qx[i].z), bf16_hi(qx[i].z), bf16_lo(qx[i].w), bf16_hi(qx[i].w)};
        float sum = 0.f;
        #pragma unroll
        for (int k = 0; k < 8; ++k) {
          v[k] *= up;
          sum += v[k];
          if (k & 1) v[k] *= 0.0625f;
        }
        *reinterpret_cast<uint4*>(sm + C::OFF_QFRAG + (((row >> 3) * C::NCH + (sg >> 2)) * 32 + (row & 7) * 4 + (sg & 3)) * 16) =
            make_uint4(pack_f16(v[0], v[4]), pack_f16(v[1], v[5]), pack_f16(v[2], v[6]), pack_f16(v[3], v[7]));
        #pragma unroll
        for (int k = 1; k < LPQ; k <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
        if (sg == 0) {  // a row that is not finite has NaN scores where it sees a key; the mask comes after them
          const bool big = E < -90 && amax < 0x7f80u;  // 2^(24 - E) would leave fp32's range: 2^32 of it go to mask_block()
          const float f = amax >= 0x7f80u ? 1.f : __int_as_float((127 + (big ? -8 : 24) - E) << 23) * p.qk_scale_log2;
          if constexpr (WIDE) qrow[24 * NQ + row] = big ? 0x1p32f : 1.f;
          else if (big) *redo = 1;
          qrow[row] = f;
          qrow[8 * NQ + row] = amax >= 0x7f80u ? __int_as_float(0x7fc00000) : sum * 0x1p-24f;
          qrow[16 * NQ + row] = 1.f / f;
        }
      }
    }
    __syncthreads();
    const uint32_t qf = smb + C::OFF_QFRAG + 16 * lane;  // this lane's operands of q
    uint32_t qr[C::QREG ? C::NCH : 1][4];
    if (C::QREG)
      #pragma unroll
      for (int c = 0; c < C::NCH; ++c) lds_128(qf + 512 * c, qr[C::QREG ? c : 0]);
    float fcol[NQ][2], qsum[NQ][2];  // score factor sm_scale log2(e) 2^(24 - E) and <1, q> of columns 2 tig, 2 tig + 1
    float o[NQ][2][4];
    float nmu[NQ][2], thr[NQ][2];    // minus the reference m (0 for none yet), the score that moves it
    float lrow[NQ][2], zrow[NQ][2];  // this lane's keys' shares of l and of the zero points' sum
    // X's reference is 2^(eref - 127), in a wide tile xrow's for each row; the scales that it serves have bit
    // patterns from slow up to slow + swin (a negative or NaN scale never has one)
    int eref = kI4Least;
    uint32_t slow = 0, swin = 0;
    bool wide = false;
    [[maybe_unused]] float ref[NQ][2];  // WIDE: the references m as scores before their factor
    #pragma unroll
    for (int nw = 0; nw < NQ; ++nw)
      #pragma unroll
      for (int e = 0; e < 2; ++e) {
        fcol[nw][e] = qrow[8 * nw + 2 * tig + e];
        qsum[nw][e] = qrow[8 * NQ + 8 * nw + 2 * tig + e];
        #pragma unroll
        for (int i = 0; i < 4; ++i) o[nw][e][i] = 0.f;
        thr[nw][e] = -INFINITY;
        ref[nw][e] = -INFINITY;
        nmu[nw][e] = lrow[nw][e] = zrow[nw][e] = 0.f;
      }
    // key j is visible to query token t if j <= Lb - T + t: keys below this need no mask in any row
    int safe_end = min(d.tok_end, d.seq_len - p.T + r0 / p.G + 1);
    if constexpr (WIDE) {  // a row with a factor for mask_block() has it called in every block
      bool big = false;
      #pragma unroll
      for (int nw = 0; nw < NQ; ++nw)
        #pragma unroll
        for (int e = 0; e < 2; ++e) big |= qrow[24 * NQ + 8 * nw + 2 * tig + e] != 1.f;
      if (__any_sync(0xffffffffu, big)) safe_end = -kI4Block;
    }

    // O^T += V^T X^T over the 64 keys at a place of the V ring, X in buffer xs
    auto product = [&](uint32_t place, int xs) {
      const uint32_t vs = smb + place * C::TILE + v_off, xa = smb + xs * C::XBUF + x_rd;
      #pragma unroll
      for (int half = 0; half < 2; ++half) {  // 32 keys each
        uint32_t r[4], bx[NQ][4];
        ldsm_x4_t(vs + half * 32 * C::RB, r[0], r[1], r[2], r[3]);
        #pragma unroll
        for (int nw = 0; nw < NQ; ++nw)  // row n at 128 n, 16-byte chunk c at (c ^ n % 8) 16
          ldsm_x4((xa + nw * 1024) ^ (half * 64), bx[nw][0], bx[nw][1], bx[nw][2], bx[nw][3]);
        #pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t va[4], vb[4];
          int4_to_f16_codes(r[2 * h], va);
          int4_to_f16_codes(r[2 * h + 1], vb);
          // M-row gid of tile jj: head dim 32 w + 4 gid + 2 jj, M-row gid + 8: the next one, 16 times over
          const uint32_t a0[4] = {va[0], va[1], vb[0], vb[1]}, a1[4] = {va[2], va[3], vb[2], vb[3]};
          #pragma unroll
          for (int nw = 0; nw < NQ; ++nw) {
            mma_f16(o[nw][0], a0, bx[nw][2 * h], bx[nw][2 * h + 1]);
            mma_f16(o[nw][1], a1, bx[nw][2 * h], bx[nw][2 * h + 1]);
          }
        }
      }
    };
    float sv[MT][NQ][4];          // scores of this warp's keys of the block at hand
    float vsc[MT][2], vz[MT][2];  // V scale and zero point of keys gid, gid + 8
    // S^T = K Q^T of this warp's keys of block blk of the tile, at this place of the ring
    auto scores = [&](uint32_t place) {
      const uint32_t ks = smb + place * C::TILE + k_off, wd = smb + place * 2 * C::WORDS + w_off;
      #pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        uint32_t wk[2], wv[2];
        #pragma unroll
        for (int k = 0; k < 2; ++k) {
          wk[k] = lds_u16(wd + 32 * mt + 16 * k);
          wv[k] = lds_u16(wd + C::WORDS + 32 * mt + 16 * k);
          vsc[mt][k] = int4_scale(wv[k]);
          vz[mt][k] = int4_zero(wv[k]);
        }
        #pragma unroll
        for (int nw = 0; nw < NQ; ++nw) sv[mt][nw][0] = sv[mt][nw][1] = sv[mt][nw][2] = sv[mt][nw][3] = 0.f;
        #pragma unroll
        for (int c = 0; c < C::NCH; c += 2) {
          uint32_t r[4];
          ldsm_x4((ks + mt * 16 * C::RB) ^ (c * 16), r[0], r[1], r[2], r[3]);
          #pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t k0[4], k1[4];
            int4_to_f16_codes(r[2 * h], k0);
            int4_to_f16_codes(r[2 * h + 1], k1);
            const uint32_t a0[4] = {k0[0], k1[0], k0[1], k1[1]}, a1[4] = {k0[2], k1[2], k0[3], k1[3]};
            #pragma unroll
            for (int nw = 0; nw < NQ; ++nw) {
              uint32_t b[4];
              if (C::QREG) {
                #pragma unroll
                for (int i = 0; i < 4; ++i) b[i] = qr[C::QREG ? c + h : 0][i];
              } else {
                lds_128(qf + 512 * (nw * C::NCH + c + h), b);
              }
              mma_f16(sv[mt][nw], a0, b[0], b[1]);
              mma_f16(sv[mt][nw], a1, b[2], b[3]);
            }
          }
        }
        const float ksc[2] = {int4_scale(wk[0]), int4_scale(wk[1])}, kz[2] = {-int4_zero(wk[0]), -int4_zero(wk[1])};
        #pragma unroll
        for (int nw = 0; nw < NQ; ++nw)
          #pragma unroll
          for (int i = 0; i < 4; ++i)  // key gid + 8 (i / 2), column 2 tig + i % 2
            sv[mt][nw][i] = fmaf(kz[i >> 1], qsum[nw][i & 1], sv[mt][nw][i]) * ksc[i >> 1];
      }
    };
    // A NaN row of V moves into the scores of the query rows that see it: out and lse are NaN as for one of K, and 0
    // times its NaN reaches no other row. Its scale is in no window, so a block that all rows see comes to
    // new_references() for it.
    auto not_finite = [](float x) { return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u; };
    // A block that not every row sees to its end: scores of invisible keys become -inf, whatever their words
    // and codes hold.
    auto mask_block = [&](int kbase) {
      #pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int j0 = kbase + 16 * (w * MT + mt) + gid;
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool bad = not_finite(vsc[mt][i >> 1]);
          #pragma unroll
          for (int nw = 0; nw < NQ; ++nw) {
            const int r = r0 + 8 * nw + 2 * tig + (i & 1), j = j0 + (i >> 1) * 8;
            if (j >= d.tok_end || (r < p.GT && j > d.seq_len - p.T + r / p.G)) sv[mt][nw][i] = -INFINITY;
            else if (bad) sv[mt][nw][i] = __int_as_float(0x7fc00000);
            else if (WIDE) sv[mt][nw][i] *= qrow[24 * NQ + 8 * nw + 2 * tig + (i & 1)];
          }
        }
        #pragma unroll
        for (int k = 0; k < 2; ++k)  // P is 0: any scale of the window
          if (j0 + 8 * k >= d.tok_end || not_finite(vsc[mt][k])) vsc[mt][k] = __uint_as_float(slow);
      }
      asm volatile("" ::: "memory");  // a branch, not predicated instructions in every block
    };

    // The barrier of a block: its scores are masked and the references voted on; the copies that the next
    // block's scores and this block's product need have landed.
    auto vote = [&](int kbase) {
      bool over = false;
      if (kbase + kI4Block > safe_end) mask_block(kbase);
      #pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        over |= __float_as_uint(vsc[mt][0]) - slow >= swin || __float_as_uint(vsc[mt][1]) - slow >= swin;
        #pragma unroll
        for (int nw = 0; nw < NQ; ++nw)
          over |= fmaxf(sv[mt][nw][0], sv[mt][nw][2]) > thr[nw][0] || fmaxf(sv[mt][nw][1], sv[mt][nw][3]) > thr[nw][1];
      }
      cp_async_wait<kI4Stages - 2>();
      return bar_or(over);
    };
    [[maybe_unused]] auto less_ref = [&](float x, int nw, int e) { return x - (ref[nw][e] == -INFINITY ? 0.f : ref[nw][e]); };
    // New references: the exact maxima of the rows; of X from the first block's scales, or row by row.
    auto new_references = [&](bool first) {
      #pragma unroll
      for (int mt = 0; mt < MT; ++mt)
        #pragma unroll
        for (int k = 0; k < 2; ++k)
          if (not_finite(vsc[mt][k])) {
            #pragma unroll
            for (int nw = 0; nw < NQ; ++nw) sv[mt][nw][2 * k] = sv[mt][nw][2 * k + 1] = __int_as_float(0x7fc00000);
            vsc[mt][k] = __uint_as_float(slow);
          }
      #pragma unroll
      for (int nw = 0; nw < NQ; ++nw)
        #pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(sv[0][nw][e], sv[0][nw][e + 2]);
          #pragma unroll
          for (int mt = 1; mt < MT; ++mt) mx = fmaxf(mx, fmaxf(sv[mt][nw][e], sv[mt][nw][e + 2]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          if (gid == 0) xmax[w * 8 * NQ + 8 * nw + 2 * tig + e] = mx;
        }
      // exponents of the V scales: 0 (a key that no row sees) does not count; a negative scale, which no append
      // writes, is below them all
      int e_hi = 0, e_lo = 255;
      #pragma unroll
      for (int mt = 0; mt < MT; ++mt)
        #pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int e = __float_as_int(vsc[mt][k]) >> 23;
          if ((e & 0xff) != 0) {
            e_hi = max(e_hi, e);
            e_lo = min(e_lo, e);
          }
        }
      e_hi = __reduce_max_sync(0xffffffffu, e_hi);
      e_lo = __reduce_min_sync(0xffffffffu, e_lo);
      if (lane == 0) {
        xexp[w] = e_hi;
        xexp[W + w] = e_lo;
      }
      __syncthreads();
      #pragma unroll
      for (int i = 0; i < W; ++i) {
        e_hi = max(e_hi, xexp[i]);
        e_lo = min(e_lo, xexp[W + i]);
      }
      [[maybe_unused]] const bool was_wide = wide;
      if (first) {
        eref = min(max(e_hi + kI4Room, kI4Least), 254);
        slow = (uint32_t)max(eref - kI4Window, 0) << 23;
        swin = ((uint32_t)(eref + 1) << 23) - slow;
      }
      bool far = e_lo < (int)(slow >> 23) || e_hi > eref;
      [[maybe_unused]] float rold[NQ][2];
      if constexpr (WIDE) {
        #pragma unroll
        for (int nw = 0; nw < NQ; ++nw)
          #pragma unroll
          for (int e = 0; e < 2; ++e) {
            rold[nw][e] = ref[nw][e];
            #pragma unroll
            for (int i = 0; i < W; ++i) ref[nw][e] = fmaxf(ref[nw][e], xmax[i * 8 * NQ + 8 * nw + 2 * tig + e]);
            far |= ref[nw][e] != -INFINITY && fabsf(ref[nw][e] * fcol[nw][e]) >= kI4Far;
          }
        if (!wide && __any_sync(0xffffffffu, far)) {  // the same in every warp
          wide = true;
          swin = 0;  // every vote asks for new references
        }
      } else {
        if (far) *redo = 1;
      }
      [[maybe_unused]] float mx2[NQ][2];  // largest X of the rows, as an exponent
      if (WIDE && wide) {
        #pragma unroll
        for (int nw = 0; nw < NQ; ++nw)
          #pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = -INFINITY;
            #pragma unroll
            for (int mt = 0; mt < MT; ++mt)
              #pragma unroll
              for (int k = 0; k < 2; ++k)
                mx = fmaxf(mx, fmaf(less_ref(sv[mt][nw][2 * k + e], nw, e), fcol[nw][e], (float)(__float_as_int(vsc[mt][k]) >> 23 & 0xff)));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            if (gid == 0) xtop[(8 * nw + 2 * tig + e) * W + w] = mx;
          }
        __syncthreads();
        #pragma unroll
        for (int nw = 0; nw < NQ; ++nw)
          #pragma unroll
          for (int e = 0; e < 2; ++e) {
            mx2[nw][e] = -INFINITY;
            #pragma unroll
            for (int i = 0; i < W; ++i) mx2[nw][e] = fmaxf(mx2[nw][e], xtop[(8 * nw + 2 * tig + e) * W + i]);
          }
      }
      #pragma unroll
      for (int nw = 0; nw < NQ; ++nw)
        #pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int col = 8 * nw + 2 * tig + e;
          float mx = xmax[col];
          #pragma unroll
          for (int i = 1; i < W; ++i) mx = fmaxf(mx, xmax[i * 8 * NQ + col]);
          const float mold = thr[nw][e] == -INFINITY ? -INFINITY : -nmu[nw][e];
          const float mnew = fmaxf(mold, mx * fcol[nw][e]);  // the factor is positive
          const float mu = mnew == -INFINITY ? 0.f : mnew;
          float down = mold - mu;
          if (WIDE && wide && mold != -INFINITY)
            down = was_wide ? (rold[nw][e] - ref[nw][e]) * fcol[nw][e] : -fmaf(ref[nw][e], fcol[nw][e], -mold);
          const float alpha = fast_exp2(down);
          float a = alpha;
          if (WIDE && wide) {
            const int eold = was_wide ? xrow[col] : eref;
            const float top = fmaxf(down + (float)eold, mx2[nw][e]);  // exponent of the largest X so far
            const int enew = top > (float)kI4Least ? (int)ceilf(fminf(top, 254.f)) : kI4Least;
            a = fast_exp2(down + (float)(eold - enew));
            __syncwarp();  // all lanes have the old one
            if (gid == 0) xrow[col] = enew;
          }
          if (!WIDE && mnew != -INFINITY && fabsf(mnew) >= kI4Far) *redo = 1;
          nmu[nw][e] = -mu;
          thr[nw][e] = mnew == -INFINITY ? -INFINITY : (mnew + (float)kI4Tau) * qrow[16 * NQ + col];
          lrow[nw][e] *= alpha;
          zrow[nw][e] *= a;
          #pragma unroll
          for (int jj = 0; jj < 2; ++jj) {
            o[nw][jj][e] *= a;
            o[nw][jj][e + 2] *= a;
          }
        }
      if constexpr (WIDE) __syncwarp();
    };
    // X of this warp's keys, to buffer xs
    auto weights = [&](int xs) {
      const float pf = __int_as_float((2 * 127 + kI4XExp - eref) << 23);  // 2^kI4XExp / 2^(eref - 127); eref <= 254
      #pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const float sc[2] = {vsc[mt][0] * pf, vsc[mt][1] * pf};
        #pragma unroll
        for (int nw = 0; nw < NQ; ++nw) {
          float pv[4];
          uint32_t x[2];
          #pragma unroll
          for (int k = 0; k < 2; ++k) {
            float* v = sv[mt][nw] + 2 * k;
            float t0, t1;
            ffma2(t0, t1, v[0], v[1], fcol[nw][0], fcol[nw][1], nmu[nw][0], nmu[nw][1]);
            pv[2 * k] = fast_exp2(t0);
            pv[2 * k + 1] = fast_exp2(t1);
            fadd2(lrow[nw][0], lrow[nw][1], lrow[nw][0], lrow[nw][1], pv[2 * k], pv[2 * k + 1]);
            x[k] = pack_f16(pv[2 * k] * sc[k], pv[2 * k + 1] * sc[k]);
            const float2 xf = f16x2_to_float2(x[k]);  // as the product sees them
            zrow[nw][0] = fmaf(xf.x, vz[mt][k], zrow[nw][0]);
            zrow[nw][1] = fmaf(xf.y, vz[mt][k], zrow[nw][1]);
          }
          stsm_x2_t((smb + xs * C::XBUF + nw * 1024 + x_wr) ^ (mt * 32), x[0], x[1]);
        }
      }
    };

    // ... in a wide tile: X = 2^(S - m + exponents) times the scale's significand, so that neither factor alone leaves
    // fp32's range
    [[maybe_unused]] auto weights_wide = [&](int xs) {
      #pragma unroll
      for (int mt = 0; mt < MT; ++mt)
        #pragma unroll
        for (int nw = 0; nw < NQ; ++nw) {
          float x[4];
          #pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t sb = __float_as_uint(vsc[mt][i >> 1]);
            const int ev = max((int)(sb >> 23 & 0xff), 1);
            const float sig = (sb & 0x7f800000u) == 0 ? vsc[mt][i >> 1] * 0x1p126f : __uint_as_float((sb & 0x807fffffu) | 0x3f800000u);
            const float t = less_ref(sv[mt][nw][i], nw, i & 1) * fcol[nw][i & 1];
            lrow[nw][i & 1] += fast_exp2(t);
            x[i] = fast_exp2(t + (float)(ev - xrow[8 * nw + 2 * tig + (i & 1)] + kI4XExp)) * sig;
          }
          const uint32_t x0 = pack_f16(x[0], x[1]), x1 = pack_f16(x[2], x[3]);
          const float2 f0 = f16x2_to_float2(x0), f1 = f16x2_to_float2(x1);
          zrow[nw][0] += f0.x * vz[mt][0] + f1.x * vz[mt][1];
          zrow[nw][1] += f0.y * vz[mt][0] + f1.y * vz[mt][1];
          stsm_x2_t((smb + xs * C::XBUF + nw * 1024 + x_wr) ^ (mt * 32), x0, x1);
        }
    };

    const int nblk = uniform(n_blocks(d));
    int kbase = d.tok_begin;
    scores(g % kI4Stages);
    bool over = vote(kbase);
    // Between two barriers: the product of the block before, the weights of this one and the scores of the next, which
    // do not depend on one another.
    #pragma unroll 1
    for (int blk = 0; blk < nblk - 1; ++blk, ++g) {
      copy_step(g % kI4Stages, true);
      if (over || blk == 0) {
        if (blk > 0) product((g - 1) % kI4Stages, (blk - 1) & 1);
        new_references(blk == 0);
      } else {
        product((g - 1) % kI4Stages, (blk - 1) & 1);
      }
      if (WIDE && wide) weights_wide(blk & 1);
      else weights(blk & 1);
      scores((g + 1) % kI4Stages);
      kbase += kI4Block;
      over = vote(kbase);
    }
    copy_step(g % kI4Stages, true);
    if (nblk > 1) product((g - 1) % kI4Stages, nblk & 1);
    if (over || nblk == 1) new_references(nblk == 1);
    if (WIDE && wide) weights_wide((nblk - 1) & 1);
    else weights((nblk - 1) & 1);
    ++g;
    // ---- sums over the keys: of a warp's lanes, then of the warps
    #pragma unroll
    for (int nw = 0; nw < NQ; ++nw)
      #pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = lrow[nw][e], z = zrow[nw][e];
        #pragma unroll
        for (int i = 4; i < 32; i <<= 1) {
          l += __shfl_xor_sync(0xffffffffu, l, i);
          z += __shfl_xor_sync(0xffffffffu, z, i);
        }
        if (gid == 0) {
          xsum[(8 * nw + 2 * tig + e) * W + w] = l;
          xsum[(8 * NQ + 8 * nw + 2 * tig + e) * W + w] = z;
        }
      }
    cp_async_wait<kI4Stages - 2>();  // V of the last block
    __syncthreads();
    product((g - 1) % kI4Stages, (nblk - 1) & 1);

    if (unit + 1 <= f_unit) load_q(queue[(unit + 1) % kI4Queue]);  // beside the epilogue
    // ---- epilogue: normalise, store. O is in units of 2^(eref - 127 - kI4XExp): codes and X exactly so
    #pragma unroll
    for (int nw = 0; nw < NQ; ++nw)
      #pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = 0.f, z = 0.f;
        const float* xs = xsum + (8 * nw + 2 * tig + e) * W;
        #pragma unroll
        for (int i = 0; i < W; ++i) {
          l += xs[i];
          z += xs[8 * NQ * W + i];
        }
        if (o_rows[nw][e] < 0) continue;
        const float unref = __int_as_float(((WIDE && wide ? xrow[8 * nw + 2 * tig + e] : eref) - kI4XExp) << 23);
        const float inv = l == 0.f ? 0.f : unref / l;
        const float lse_v = l == 0.f ? -INFINITY : (__log2f(l) - nmu[nw][e]) * LN2;
        const float v[4] = {fmaf(o[nw][0][e], 16777216.f, -z) * inv, fmaf(o[nw][0][e + 2], 1048576.f, -z) * inv,
                            fmaf(o[nw][1][e], 16777216.f, -z) * inv, fmaf(o[nw][1][e + 2], 1048576.f, -z) * inv};
        if (d.slot < 0) {
          const int64_t row = first_row(d) + o_rows[nw][e];
          *reinterpret_cast<uint2*>(p.out_bf16 + row * D + 32 * w + 4 * gid) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
          if (w == 0 && gid == 0) p.lse[row] = lse_v;
        } else {
          const int64_t row = (int64_t)d.slot * p.GT + r0 + 8 * nw + 2 * tig + e;
          *reinterpret_cast<float4*>(p.part_o + row * D + 32 * w + 4 * gid) = make_float4(v[0], v[1], v[2], v[3]);
          if (w == 0 && gid == 0) p.part_lse[row] = lse_v;
        }
      }
  }
  cp_async_wait<0>();  // copies past the last block
  __syncthreads();
  return *redo != 0;
}

template <int D, int NQ>
__device__ __noinline__ void i4_wide_pass(const SplitInt4Params& p) {
  __syncthreads();  // the first pass is done with the shared memory
  i4_pass<D, NQ, true>(p);
}

// OVER: out lies over q. The first pass writes out, so the second one goes alone. (A kernel of its own: the same as a
// branch here costs the ordinary case 0.6 us.)
template <int D, int NQ, int CPS, bool OVER>
__global__ void __launch_bounds__(I4Cfg<D, NQ>::THREADS, CPS)
split_int4_kernel(const __grid_constant__ SplitInt4Params p) {
  // Everything below reads or writes what earlier kernels of the stream may still be working on: the
  // plan, the pages (a plan serves every layer of a step, so the kernel before this one can be the
  // append), the combine counters.
  griddep_wait();
  griddep_launch_dependents();  // the combine kernel may be scheduled; it waits for this grid itself
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < (int64_t)p.B * p.T * p.Hq;
       i += (int64_t)gridDim.x * blockDim.x)
    p.row_cnt[i] = 0;
  if constexpr (OVER) {
    i4_pass<D, NQ, true>(p);
  } else {
    if (i4_pass<D, NQ, false>(p)) i4_wide_pass<D, NQ>(p);
  }
}

// ------------------------------------------------------------------ host side
template <int D, int NQ, int CPS>
static cudaError_t launch_i4(const SplitInt4Params& p, int sms, cudaStream_t st) {
  using C = I4Cfg<D, NQ>;
  static_assert(CPS * (C::ALLOC + 1024) <= 228 * 1024, "the CTAs fit an SM's shared memory");
  const auto fn = p.over_q ? split_int4_kernel<D, NQ, CPS, true> : split_int4_kernel<D, NQ, CPS, false>;
  if (!ensure_smem_attr((const void*)fn, C::ALLOC)) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  const int groups = (p.GT + 8 * NQ - 1) / (8 * NQ);
  const int n = sms * CPS / groups;  // bins at a time
  cfg.gridDim = dim3((p.n_bins < n ? p.n_bins : n) * groups);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::ALLOC;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // launched while the previous kernel drains
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, p);
}

template <int D>
static cudaError_t launch_i4_gt(const SplitInt4Params& p, int sms, cudaStream_t st) {
  constexpr int CPS = D == 64 ? 8 : 4;
  return p.GT <= 8 ? launch_i4<D, 1, CPS>(p, sms, st) : launch_i4<D, 2, CPS>(p, sms, st);
}

bool split_int4_supported(int D, int GT) { return GT >= 1 && GT <= kMaxGT && (D == 64 || D == 128); }

cudaError_t launch_split_int4(const SplitInt4Params& p, int D, int device, cudaStream_t st) {
  if (!split_int4_supported(D, p.GT)) return cudaErrorInvalidValue;
  const int sms = default_bins(device) / split_ctas_per_sm();
  if (sms <= 0) return cudaErrorUnknown;
  return D == 128 ? launch_i4_gt<128>(p, sms, st) : launch_i4_gt<64>(p, sms, st);
}

}  // namespace decattn
