// kvq_paged_prompt.cuh — attention over the E4M3 pages for many query rows per
// kv head (prompts, chunks of prompts): tcgen05 with accumulators in tensor
// memory.
//
// The mathematics is kvq_paged_decode.cuh's: s = kappa * sk * (q . a) +
// log2(sv), w = 2^(s - m + 7), out = sum w c / sum (w / sv).  Keys, values and
// weights enter the tensor cores as fp16: codes exactly, fp16 queries exactly,
// bf16 rows through a power of two (elements below 2^-22 of their row's largest
// lose bits, an error below 2^-40 of it), weights rounded: half a step, 2^-11,
// of a token's weight * scale down to 2^-21 of the row's largest, and at most
// 2^-32 of that largest below (see kLazy).
//
// A CTA owns 256 query rows of one kv head (two tiles of 128; row r is new
// token r / R, head r % R of the group, so grouped heads share every key
// tile) and walks tiles of 128 tokens:
//   loader     (1 warp)   pages and scales, TMA of raw key / value tiles
//   converters (4 warps)  raw codes -> fp16 tiles in shared memory, 128-byte
//                         swizzle; the same layout serves keys (K-major
//                         operand) and values (N-major operand)
//   issuer     (1 warp)   S_w = Q_w K^T, O_w += P_w V   (w = 0, 1)
//   softmax    (2 x 4 warps) a thread owns a row: maximum, weights, P into
//                         tensor memory over S, rescaling of O when its
//                         maximum moved by more than kLazy
// Tensor memory: S0, S1 (128 columns each), O0, O1 (D columns each); P_w lies
// over S_w.  The issuer alternates the two row tiles, so one tile's softmax
// runs beside the other's products.
//
// Bound: the chain of a row tile.  A key tile costs 4 products of 128 x 128 x
// 128 (512 cycles each, the tensor pipe's 2048), but a row tile's softmax
// (about 1900 cycles) and the hand-overs to it and back lie between its scores
// and its output product, and only one other row tile's products fit beside
// them: about 3300 cycles a key tile, the tensor pipe 59 % active.  Measured: 2048
// new tokens behind 32768 (32 heads, D = 128) 943 us, 1.20 PFLOP/s, 62 % of the
// measured bf16 rate (two rounds of CTAs over 152 SMs: 84 % of a full one);
// without the softmax 805 us, without the conversion 885 us, without either
// 756 us.  Three prompts of up to 4001 tokens (40 heads) 254 us, where the
// causal half and 9 us a CTA of start and end weigh more.  Lanes that wait by a
// vote, so that the compiler knows a warp as converged, took 956 -> 943 and
// 262 -> 254 us.
// Measured and not kept, beside 957 and 265 us without the vote: two CTAs sharing
// each key tile (cta_group::2, half of the conversion each): 939 and 296 us; every
// CTA an equal share of the tiles, items joined from shares: 958 us, and prompts
// need a cost for each item; two threads a row: 1053 and 280 us; S read from
// tensor memory once, into 128 registers: 1037 and 261 us.
// Weights as fp16: against 64 bits the chunk's outputs are 2.8e-4 off (relative
// 2-norm; with fp32 weights 2.1e-4, the output's own rounding), bf16 prompts'
// 1.6e-3 with either.  A second half of a weight would need 128 more columns of
// tensor memory, which is full, and half as many products again.
#pragma once

#include <type_traits>

#include "kvq_paged.cuh"

namespace kvq {

struct PagedPromptParams {
  PagedAttnParams a;
  int items_max;  // row-tile pairs of all requests, at most
};

__host__ __device__ constexpr int round_up128(int x) { return (x + 127) / 128 * 128; }

template <int D>
struct PromptCfg {
  static constexpr int N = 128;                   // tokens of a tile
  static constexpr int ROWS = 256;                // query rows of a CTA
  static constexpr int NRAW = 2;                  // raw tiles in flight
  static constexpr int NT = 4;                    // fp16 tiles
  static constexpr int RAW = N * D;               // bytes of a raw tile
  static constexpr int TILE = N * D * 2;          // bytes of an fp16 tile
  static constexpr int QT = 128 * D * 2;          // bytes of a query tile
  static constexpr int REC = 8;                   // granule records of a tile
  static constexpr int NREC = 8;                  // tiles of the record ring
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_T = OFF_Q + 2 * QT;
  static constexpr int OFF_RAW = OFF_T + NT * TILE;
  static constexpr int OFF_REC = OFF_RAW + NRAW * RAW;
  static constexpr int OFF_BAR = OFF_REC + NREC * REC * 16;
  static constexpr int NBAR = 2 * NRAW + 2 * NT + NREC + 2 + 2 + 2 + 2 + 1;
  static constexpr int OFF_MISC = round_up128(OFF_BAR + NBAR * 8);
  static constexpr int SMEM = OFF_MISC + 128 + 1024;  // 1024 for the base's alignment
  static constexpr int THREADS = 512;
  // Registers of a thread: 128 at launch, then by role (two softmax groups,
  // the converters, the rest); the sum stays the launch's 512 * 128.
  static constexpr int R_SOFTMAX = 176, R_CONVERT = 96, R_REST = 64;
  static_assert(256 * R_SOFTMAX + 128 * R_CONVERT + 128 * R_REST == 512 * 128, "register split");
  static constexpr uint32_t S_COL = 0, O_COL = 256, P_OFF = 64;  // P: upper half of S
};

// ---- tcgen05 -------------------------------------------------------------

// Shared-memory operand descriptor.  High word: stride byte offset in 16-byte
// units, version 1, 128-byte swizzle; low word: start address and leading byte
// offset in 16-byte units.  Operands of one tile differ in the low word alone.
__host__ __device__ constexpr uint32_t umma_desc_hi(uint32_t sbo) {
  return (sbo >> 4) | (1u << 14) | (2u << 29);
}
__device__ __forceinline__ uint32_t umma_desc_lo(uint32_t addr, uint32_t lbo) {
  return ((addr >> 4) & 0x3fffu) | ((lbo >> 4) << 16);
}

// Instruction descriptor: fp32 accumulator, fp16 operands, M = 128.
__host__ __device__ constexpr uint32_t umma_idesc(int n, bool b_n_major) {
  return (1u << 4) | (b_n_major ? 1u << 16 : 0u) | (static_cast<uint32_t>(n / 8) << 17) |
         (static_cast<uint32_t>(128 / 16) << 24);
}

// The products are issued by one lane (`one`) of a warp that runs converged, so
// the operands' words stay warp-uniform values.
__device__ __forceinline__ void umma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi,
                                        uint32_t idesc, uint32_t accumulate, uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "setp.ne.b32 q, %6, 0;\n\tmov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate), "r"(one)
      : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t hi,
                                        uint32_t idesc, uint32_t accumulate, uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "setp.ne.b32 q, %6, 0;\n\tmov.b64 b, {%2, %3};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate), "r"(one)
      : "memory");
}
// Arrives on `bar` when the products issued so far are complete.
__device__ __forceinline__ void umma_commit(uint64_t* bar, uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_addr(bar)),
      "r"(one)
      : "memory");
}
__device__ __forceinline__ void tmem_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// This warp's 32 lanes, 32 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(addr)
      : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
        "l"(reinterpret_cast<unsigned long long&>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return d;
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Two weights as fp16, finite whatever their scores (NaN stays NaN).
__device__ __forceinline__ uint32_t weight_bits(float lo, float hi) {
  uint32_t x;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(x) : "f"(hi), "f"(lo));
  return x;
}

// Rounds of a wait between two roles of the CTA (each may suspend for a
// hardware-chosen time; a legitimate wait is microseconds).
constexpr uint32_t kRoleWait = 1u << 20;
// The reference maximum m is raised only when a score exceeds it by this much
// (log2), so most tiles skip the rescaling of O.  Weights are 2^(s - reference(m)),
// at most 2^(kLazy + kWeightLog2) = 2^15, which uses fp16's range.  A huge score's
// maximum and exponent are rounded apart, so there fp16's range is left to that.
constexpr float kLazy = 8.0f;
constexpr float kWeightLog2 = 7.0f, kWeightInv = 0x1p-7f;
__device__ __forceinline__ float reference(float m) {
  return fabsf(m) < 0x1p18f ? m - kWeightLog2 : m == -INFINITY ? 0.f : m;
}

// The work of a CTA: rows [row0, row0 + 256) of request b, kv head h.
struct PromptItem {
  int b, h, row0, rows;  // rows: the request's
  int q0, seq, n;
  int lo, hi;            // tokens [lo, hi) that any row of the CTA sees
  int t0, nt;            // first tile's first token, tiles
};

template <int D, bool BF16>
__global__ void __launch_bounds__(PromptCfg<D>::THREADS, 1)
    paged_prompt_kernel(const __grid_constant__ PagedPromptParams pp,
                        const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap) {
  using C = PromptCfg<D>;
  constexpr int N = C::N, NRAW = C::NRAW, NT = C::NT;
  const PagedAttnParams& p = pp.a;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - smem_addr(smem_raw));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* raw_full = bars;
  uint64_t* raw_empty = raw_full + NRAW;
  uint64_t* t_full = raw_empty + NRAW;
  uint64_t* t_empty = t_full + NT;
  uint64_t* rec_full = t_empty + NT;
  uint64_t* s_full = rec_full + C::NREC;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_done = p_full + 2;
  uint64_t* q_full = o_done + 2;
  uint64_t* drain = q_full + 2;
  float4* recs = reinterpret_cast<float4*>(smem + C::OFF_REC);
  int* whole = reinterpret_cast<int*>(smem + C::OFF_MISC + 64);  // [NREC] every granule is there
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC + 4);
  PromptItem* found = reinterpret_cast<PromptItem*>(smem + C::OFF_MISC + 16);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < NRAW; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 4);
    }
    for (int i = 0; i < NT; ++i) {
      mbar_init(&t_full[i], 4);
      mbar_init(&t_empty[i], 1);
    }
    for (int i = 0; i < C::NREC; ++i) mbar_init(&rec_full[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_done[i], 1);
      mbar_init(&q_full[i], 4);
    }
    mbar_init(drain, 1);
    fence_barrier_init();
    *abort_flag = 0;
    found->b = -1;
  }
  grid_dep_wait();

  // ---- which item: prefix sum of the requests' row-tile pairs ----------------
  {
    int* sums = reinterpret_cast<int*>(smem + C::OFF_T);  // before any tile is there
    const int H = p.H;
    const int item = blockIdx.x / H, h = blockIdx.x - item * H;
    auto pairs_of = [&](int b, PagedReq* r) {
      int bad;
      *r = paged_req(p, b, &bad);
      if (bad && blockIdx.x == 0) set_err(p.err, KVQ_PAGED_ERR_LENGTH);
      const int rows = r->n * p.R;
      if (rows < p.row_min || rows > p.row_max) return 0;
      return (rows + C::ROWS - 1) / C::ROWS;
    };
    const int per = (p.batch + C::THREADS - 1) / C::THREADS;
    const int b0 = min(tid * per, p.batch), b1 = min(b0 + per, p.batch);
    int mine = 0;
    PagedReq r;
    for (int b = b0; b < b1; ++b) mine = add_counts(mine, pairs_of(b, &r));
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl = add_counts(incl, x);
    }
    if (lane == 31) sums[warp] = incl;
    int at = __shfl_up_sync(0xffffffffu, incl, 1);
    if (lane == 0) at = 0;
    __syncthreads();
    for (int w = 0; w < warp; ++w) at = add_counts(at, sums[w]);
    if (item >= at && item < add_counts(at, mine)) {
      for (int b = b0; b < b1; ++b) {
        const int c = pairs_of(b, &r);
        if (item < add_counts(at, c)) {
          PromptItem it;
          it.b = b;
          it.h = h;
          // the last rows see the most tokens: they start first
          it.row0 = (c - 1 - (item - at)) * C::ROWS;
          it.rows = r.n * p.R;
          it.q0 = r.q0;
          it.seq = r.seq;
          it.n = r.n;
          const int last = min(it.row0 + C::ROWS, it.rows) - 1;
          it.hi = max(0, r.seq - r.n + row_token(p, last) + 1);
          it.lo = p.window == 0 ? 0 : max(0, r.seq - r.n + row_token(p, it.row0) + 1 - p.window);
          it.t0 = it.lo / N * N;
          it.nt = it.hi > it.t0 ? (it.hi - it.t0 + N - 1) / N : 0;
          *found = it;
          break;
        }
        at = add_counts(at, c);
      }
    }
  }
  __syncthreads();
  grid_dep_launch();
  const PromptItem it = *found;
  if (it.b < 0) return;
  const int nt = it.nt;
  if (nt == 0) {
    // no token is seen: zero rows
    for (int e = tid; e < C::ROWS * (D / 8); e += C::THREADS) {
      const int row = it.row0 + e / (D / 8);
      if (row >= it.rows) break;
      const int j = row_token(p, row);
      reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) +
                               static_cast<long long>(it.q0 + j) * p.out_stride +
                               (static_cast<long long>(it.h) * p.R + (row - j * p.R)) * D)[e % (D / 8)] =
          make_uint4(0, 0, 0, 0);
    }
    return;
  }
  if (warp == 13) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_addr(tmem_slot))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int halves = it.rows - it.row0 > 128 ? 2 : 1;

  // Bounded wait of a whole warp; false when it ran out or another role gave up.
  // Lanes see the barrier and the flag at different times: they decide together,
  // so that the warp stays converged for what it does next.  (A phase that one
  // lane has seen lasts until all have: the warp's own arrival ends the next.)
  const uint32_t rounds = min(p.wait_limit, kRoleWait);
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    for (uint32_t i = 0; i < rounds; ++i) {
      if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity & 1))) return true;
      if (__any_sync(0xffffffffu, *abort_flag)) return false;
    }
    *abort_flag = 1;
    set_err(p.err, KVQ_PAGED_ERR_WAIT);
    return false;
  };

  if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::R_REST));
    if (warp == 12) {
      // ================================================================ loader
      const int box = p.box_rows, nbox = N / box;
      const uint32_t box_bytes = static_cast<uint32_t>(box) * D;
      int raw = 0;  // raw tiles requested so far
      int pend = 0;
      // lane l holds granule l % 8 of tile l / 8 of a batch of four tiles
      auto granule_page = [&](int i) {
        const int tile = i + lane / 8;
        const int tok = it.t0 + tile * N + lane % 8 * 16;
        const int bx = tok & ~(box - 1), rep = max(bx, it.lo);
        if (tile >= nt || rep >= it.hi || bx + box <= it.lo) return -1;
        const int page = p.table[static_cast<size_t>(it.b) * p.max_pages + (rep >> p.lg_ps)];
        if (page >= 0 && page < p.n_pages) return page;
        set_err(p.err, KVQ_PAGED_ERR_BAD_PAGE);
        return -1;
      };
      int page = -1, next = granule_page(0);
      bool ok = true;
      for (int i = 0; i < nt && ok; ++i) {
        if (i % 4 == 0) {
          page = next;
          next = granule_page(i + 4);
        }
        // the tile's records
        if (lane / 8 == i % 4) {
          const int tok = it.t0 + i * N + lane % 8 * 16;
          float ks = 0.f, vs = 1.f;
          if (page >= 0) {
            const size_t at = static_cast<size_t>(page) * p.H + it.h;
            ks = p.k_scale[at];
            vs = p.v_scale[at];
          }
          const bool seen = page >= 0 && tok < it.hi && tok + 16 > it.lo;
          recs[i % C::NREC * C::REC + lane % 8] =
              make_float4(ks, lg2(vs), kWeightInv / vs, seen ? 1.f : 0.f);
          const uint32_t m = 0xffu << (lane & 24);
          const uint32_t all = __ballot_sync(m, seen);
          if (lane % 8 == 0) whole[i % C::NREC] = all == m;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&rec_full[i % C::NREC]);
        // lane l < nbox copies box l of the tile
        const int src = (i % 4) * 8 + (lane < nbox ? lane : 0) * (box / 16);
        const int pg = __shfl_sync(0xffffffffu, page, src);
        const bool mine = lane < nbox && pg >= 0;
        const int count = __popc(__ballot_sync(0xffffffffu, mine));
        const int tok = it.t0 + i * N + lane * box;
        const int row = mine ? ((pg * p.H + it.h) << p.lg_ps) + (tok & ((1 << p.lg_ps) - 1)) : 0;
#pragma unroll
        for (int side = 0; side < 2; ++side, ++raw) {
          const int s = raw % NRAW;
          if (raw >= NRAW && !wait(&raw_empty[s], raw / NRAW - 1)) {
            ok = false;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(&raw_full[s], count * box_bytes);
          __syncwarp();
          if (mine)
            tma_load_2d(smem + C::OFF_RAW + s * C::RAW + lane * box_bytes, side ? &vmap : &kmap, 0,
                        row, &raw_full[s]);
          pend = raw + 1;
        }
      }
      // no copy may be in flight when the CTA leaves: the last NRAW of them
      for (int r = max(0, pend - NRAW); r < pend; ++r)
        mbar_wait_bounded(&raw_full[r % NRAW], (r / NRAW) & 1, kRoleWait);
    } else if (warp == 13) {
      // ================================================================ issuer
      constexpr uint32_t id_s = umma_idesc(N, false), id_o = umma_idesc(D, true);
      constexpr uint32_t hi = umma_desc_hi(1024);
      const uint32_t one = lane == 0;
      const uint32_t q_lo = umma_desc_lo(base + C::OFF_Q, 16);
      const uint32_t k_lo = umma_desc_lo(base + C::OFF_T, 16);
      const uint32_t v_lo = umma_desc_lo(base + C::OFF_T, N * 128);
      auto scores = [&](int w, int i) {
        const uint32_t q = q_lo + w * (C::QT >> 4), k = k_lo + (2 * i) % NT * (C::TILE >> 4);
        const uint32_t d = tmem + C::S_COL + w * 128;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = ((ks >> 2) * (128 * 128) + (ks & 3) * 32) >> 4;
          umma_ss(d, q + off, k + off, hi, id_s, ks > 0, one);
        }
        umma_commit(&s_full[w], one);
      };
      auto outputs = [&](int w, int i) {
        const uint32_t v = v_lo + (2 * i + 1) % NT * (C::TILE >> 4);
        const uint32_t d = tmem + C::O_COL + w * D, a = tmem + C::S_COL + w * 128 + C::P_OFF;
#pragma unroll
        for (int ks = 0; ks < N / 16; ++ks)
          umma_ts(d, a + ks * 8, v + ks * (2048 >> 4), hi, id_o, i > 0 || ks > 0, one);
        umma_commit(&o_done[w], one);
      };
      auto tile_ready = [&](int x) { return wait(&t_full[x % NT], x / NT); };
      bool ok = tile_ready(0);
      for (int w = 0; w < halves && ok; ++w) {
        ok = wait(&q_full[w], 0);
        if (!ok) break;
        tmem_fence_after();
        scores(w, 0);
      }
      if (ok) umma_commit(&t_empty[0], one);
      for (int i = 0; i < nt && ok; ++i) {
        ok = tile_ready(2 * i + 1) && (i + 1 >= nt || tile_ready(2 * i + 2));
        for (int w = 0; w < halves && ok; ++w) {
          ok = wait(&p_full[w], i);
          if (!ok) break;
          tmem_fence_after();
          outputs(w, i);
          if (i + 1 < nt) scores(w, i + 1);
        }
        if (!ok) break;
        umma_commit(&t_empty[(2 * i + 1) % NT], one);
        if (i + 1 < nt) umma_commit(&t_empty[(2 * i + 2) % NT], one);
      }
      // no product and no arrival may be in flight when the CTA leaves
      umma_commit(drain, one);
      mbar_wait_bounded(drain, 0, kRoleWait);
    }
  } else if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::R_CONVERT));
    // ============================================================ converters
    const int ct = tid - 256;  // 0 .. 127
    constexpr int CH = D / 16;             // 16-byte chunks of a raw row
    constexpr int PASS = N * CH / 128;     // chunks a thread converts
    for (int x = 0; x < 2 * nt; ++x) {     // K0, V0, K1, V1, ...
      const int i = x >> 1, s = x % NRAW, d = x % NT;
      if (!wait(&raw_full[s], x / NRAW)) break;
      if (x >= NT && !wait(&t_empty[d], x / NT - 1)) break;
      const uint8_t* src = smem + C::OFF_RAW + s * C::RAW;
      uint8_t* dst = smem + C::OFF_T + d * C::TILE;
      const int tok = it.t0 + i * N;
      // rows of no page or no token may hold anything: they become zeros
      const bool edge = tok < it.lo || tok + N > it.hi || !whole[i % C::NREC];
#pragma unroll 4
      for (int k = 0; k < PASS; ++k) {
        int row, j;
        if constexpr (D == 128) {
          // eight lanes read two half rows and write two half rows, all on
          // different banks
          const int u = k * 16 + (ct >> 3);  // (row pair, half) of the tile
          const int pair = u >> 1, flip = u & 1;
          row = pair * 2 + ((ct >> 2) & 1);
          j = (ct & 3) + 4 * (((ct >> 2) & 1) ^ flip);
        } else {
          row = k * 32 + (ct >> 2);
          j = ct & 3;
        }
        const int sw = D == 128 ? (j ^ (row & 7)) : (j ^ ((row >> 1) & 3));
        uint4 v = *reinterpret_cast<const uint4*>(src + row * D + (sw << 4));
        if (edge) {
          const int tk = tok + row;
          if (tk < it.lo || tk >= it.hi || recs[i % C::NREC * C::REC + (row >> 4)].w == 0.f)
            v = make_uint4(0, 0, 0, 0);
        }
        uint4 lo, hi;
        e4m3x4_to_half2x2(v.x, lo.x, lo.y);
        e4m3x4_to_half2x2(v.y, lo.z, lo.w);
        e4m3x4_to_half2x2(v.z, hi.x, hi.y);
        e4m3x4_to_half2x2(v.w, hi.z, hi.w);
        uint8_t* o = dst + (j >> 2) * (N * 128) + row * 128;
        const int c0 = (j & 3) * 2;
        *reinterpret_cast<uint4*>(o + ((c0 ^ (row & 7)) << 4)) = lo;
        *reinterpret_cast<uint4*>(o + (((c0 + 1) ^ (row & 7)) << 4)) = hi;
      }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&t_full[d]);
        mbar_arrive(&raw_empty[s]);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::R_SOFTMAX));
    if ((warp >> 2) < halves) {
      // =============================================================== softmax
      const int w = warp >> 2;
      const int lrow = (warp & 3) * 32 + lane;
      const int row = it.row0 + w * 128 + lrow;
      const int tokj = row_token(p, min(row, it.rows - 1));
      const int pos = it.seq - it.n + tokj;
      const int first = p.window == 0 ? 0 : max(0, pos - p.window + 1);
      const uint32_t s_at = tmem + C::S_COL + w * 128 + (static_cast<uint32_t>((warp & 3) * 32) << 16);
      const uint32_t o_at = tmem + C::O_COL + w * D + (static_cast<uint32_t>((warp & 3) * 32) << 16);
      float cq = fabsf(p.qscale);  // the sign goes into the queries
      {
        // This warp's 32 query rows into their operand tile: a row is D / 8
        // lanes wide, so a copy moves whole rows, and all copies are on their
        // way at once.  (Loops that run once an item stay rolled: their code is
        // fetched as it runs, and fetching costs more than looping.)
        constexpr int LPR = D / 8, RPL = 32 / LPR;  // lanes of a row, rows of a copy
        const int sub = lane / LPR, vec = lane % LPR;
        const uint32_t tile = base + C::OFF_Q + w * C::QT;
#pragma unroll 1
        for (int i = 0; i < 32 / RPL; ++i) {
          const int tr = (warp & 3) * 32 + i * RPL + sub;
          const int gr = min(it.row0 + w * 128 + tr, it.rows - 1), j = row_token(p, gr);
          const void* src = reinterpret_cast<const uint4*>(
                                static_cast<const uint16_t*>(p.q) +
                                static_cast<long long>(it.q0 + j) * p.q_stride +
                                (static_cast<long long>(it.h) * p.R + (gr - j * p.R)) * D) + vec;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                           tile + (vec >> 3) * (128 * 128) + tr * 128 + (((vec & 7) ^ (tr & 7)) << 4)),
                       "l"(src)
                       : "memory");
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
        if (BF16 || p.qscale < 0.f) {
          // a thread's own row: as fp16, with the sign of the softmax scale
          uint8_t* own = smem + C::OFF_Q + w * C::QT + lrow * 128;
          float up = 1.f;
          if constexpr (BF16) {
            // the row times a power of two: its largest element to [2^14, 2^15)
            uint32_t mg = 0;
#pragma unroll 2
            for (int i = 0; i < D / 8; ++i) {
              const uint4 v = *reinterpret_cast<const uint4*>(
                  own + (i >> 3) * (128 * 128) + (((i & 7) ^ (lrow & 7)) << 4));
              mg = __vmaxu2(mg, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                         __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
            }
            const int e = max(static_cast<int>(max(mg & 0xffffu, mg >> 16) >> 7) - 127, -100);
            up = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
            cq *= __uint_as_float(static_cast<uint32_t>(127 - 14 + e) << 23);
          }
          if (p.qscale < 0.f) up = -up;
#pragma unroll 2
          for (int i = 0; i < D / 8; ++i) {
            uint4* at = reinterpret_cast<uint4*>(own + (i >> 3) * (128 * 128) +
                                                 (((i & 7) ^ (lrow & 7)) << 4));
            uint4 v = *at;
            auto cv = [&](uint32_t x) {
              float2 f;
              if constexpr (BF16) {
                f = make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
              } else {
                f = __half22float2(*reinterpret_cast<const __half2*>(&x));
              }
              return half2_bits(f.x * up, f.y * up);
            };
            v = make_uint4(cv(v.x), cv(v.y), cv(v.z), cv(v.w));
            *at = v;
          }
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[w]);
      }
      float m = -INFINITY, l = 0.f;
      bool ok = true;
      // tokens every row of this half sees
      const int r0 = it.row0 + w * 128, r1 = min(r0 + 128, it.rows) - 1;
      const int all_hi = it.seq - it.n + row_token(p, r0) + 1;
      const int all_lo = p.window == 0 ? 0 : max(0, it.seq - it.n + row_token(p, r1) + 1 - p.window);
      for (int i = 0; i < nt; ++i) {
        ok = wait(&rec_full[i % C::NREC], i / C::NREC) && wait(&s_full[w], i);
        if (!ok) break;
        tmem_fence_after();
        const int tok = it.t0 + i * N;
        const float4* rec = recs + i % C::NREC * C::REC;
        const bool edge = tok < all_lo || tok + N > all_hi || !whole[i % C::NREC];
        auto tile = [&](auto masked) {
          constexpr bool MASK = decltype(masked)::value;
          // Chunks of 32 columns, the next one loading while one is worked on:
          // first the maximum of chunks 0 .. 3, then the weights of 3 .. 0, so
          // the last chunk stays in registers and P (over the upper half of S)
          // overwrites only columns that are done with.
          uint32_t r[2][32];
          auto hide = [&](uint32_t (&x)[32], int c) {
            if constexpr (MASK) {
              // bit k: token tok + 32 c + k is seen
              const int up = pos - (tok + 32 * c), dn = first - (tok + 32 * c);
              uint32_t see = up >= 31 ? 0xffffffffu : up < 0 ? 0u : (2u << up) - 1;
              see &= dn <= 0 ? 0xffffffffu : dn > 31 ? 0u : 0xffffffffu << dn;
              if (rec[2 * c].w == 0.f) see &= 0xffff0000u;
              if (rec[2 * c + 1].w == 0.f) see &= 0x0000ffffu;
#pragma unroll
              for (int k = 0; k < 32; ++k)  // (the exponential of -inf is the weight 0)
                x[k] = (see >> k) & 1 ? x[k] : 0xff800000u;
            }
          };
          float mx = -INFINITY;
          tmem_ld32(s_at, r[0]);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            tmem_wait_ld();
            if (c < 3) tmem_ld32(s_at + 32 * (c + 1), r[(c + 1) & 1]);
            uint32_t(&x)[32] = r[c & 1];
            hide(x, c);
            // the raw maximum of each granule, then its scales
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              const float4 rc = rec[2 * c + g];
              float gm = -INFINITY;
#pragma unroll
              for (int k = 0; k < 16; ++k) gm = fmaxf(gm, __uint_as_float(x[16 * g + k]));
              // (never 0: -inf times it stays -inf)
              const float f = fmaxf(rc.x * cq, 1.17549435e-38f);
              mx = fmaxf(mx, fmaf(gm, f, rc.y));
            }
          }
          const float mn = mx > m + kLazy || m == -INFINITY ? mx : m;
          const float mb = reference(mn);
          const bool move = mn != m && m != -INFINITY;  // O holds sums at the old reference
          const float al = move ? ex2(reference(m) - mb) : 1.f;
          m = mn;
          l *= al;
          if (__any_sync(0xffffffffu, move)) {
            if (!wait(&o_done[w], i - 1)) return false;
            tmem_fence_after();
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {  // (few registers: S waits in 128)
              uint32_t o[16];
              tmem_ld16(o_at + 16 * c, o);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * al);
              tmem_st16(o_at + 16 * c, o);
            }
          }
#pragma unroll
          for (int c = 3; c >= 0; --c) {
            uint32_t h[16];
            uint32_t(&x)[32] = r[c & 1];
            if (c < 3) {
              tmem_wait_ld();
              hide(x, c);
            }
            if (c > 0) tmem_ld32(s_at + 32 * (c - 1), r[(c - 1) & 1]);
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              const float4 rc = rec[2 * c + g];
              const float f = fmaxf(rc.x * cq, 1.17549435e-38f), y = rc.y - mb;
              const float2 f2 = make_float2(f, f), y2 = make_float2(y, y);
              float2 sum = make_float2(0.f, 0.f);
#pragma unroll
              for (int k = 0; k < 16; k += 2) {
                const float2 z = fma2(make_float2(__uint_as_float(x[16 * g + k]),
                                                  __uint_as_float(x[16 * g + k + 1])), f2, y2);
                const float2 w = make_float2(ex2(z.x), ex2(z.y));
                sum = add2(sum, w);
                h[8 * g + k / 2] = weight_bits(w.x, w.y);
              }
              l = fmaf(sum.x + sum.y, rc.z, l);
            }
            tmem_st16(s_at + C::P_OFF + 16 * c, h);
          }
          tmem_wait_st();
          return true;
        };
        // (two bodies: one with the masks' branches in it measured 12 % slower)
        ok = edge ? tile(std::true_type{}) : tile(std::false_type{});
        if (!ok) break;
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[w]);
      }
      if (ok && wait(&o_done[w], nt - 1)) {
        tmem_fence_after();
        const float inv = l > 0.f ? kWeightInv / l : (l == 0.f ? 0.f : l);
        // Through the query tile (its products are complete), so that whole rows
        // are written: this warp's rows, chunks swizzled as the queries were.
        uint8_t* tile = smem + C::OFF_Q + w * C::QT;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t r[32], o[16];
          tmem_ld32(o_at + 32 * c, r);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float x = __uint_as_float(r[2 * k]) * inv, y = __uint_as_float(r[2 * k + 1]) * inv;
            if constexpr (BF16) {
              const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
              o[k] = *reinterpret_cast<const uint32_t*>(&b);
            } else {
              o[k] = half2_bits(x, y);
            }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int ch = 4 * c + k;
            *reinterpret_cast<uint4*>(tile + (ch >> 3) * (128 * 128) + lrow * 128 +
                                      (((ch & 7) ^ (lrow & 7)) << 4)) =
                make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          }
        }
        __syncwarp();
        constexpr int LPR = D / 8, RPL = 32 / LPR;
        const int sub = lane / LPR, vec = lane % LPR;
#pragma unroll 2
        for (int i = 0; i < 32 / RPL; ++i) {
          const int tr = (warp & 3) * 32 + i * RPL + sub;
          const int gr = it.row0 + w * 128 + tr, j = row_token(p, gr);
          const uint4 v = *reinterpret_cast<const uint4*>(tile + (vec >> 3) * (128 * 128) + tr * 128 +
                                                          (((vec & 7) ^ (tr & 7)) << 4));
          if (gr < it.rows)
            *(reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) +
                                       static_cast<long long>(it.q0 + j) * p.out_stride +
                                       (static_cast<long long>(it.h) * p.R + (gr - j * p.R)) * D) +
              vec) = v;
        }
        tmem_fence_before();
      }
    }
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  if (warp == 13) {
    tmem_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

template <int D, bool BF16>
cudaError_t launch_paged_prompt_t(const PagedPromptParams& p, const CUtensorMap& km,
                                  const CUtensorMap& vm, cudaStream_t st) {
  using C = PromptCfg<D>;
  auto fn = paged_prompt_kernel<D, BF16>;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(fn), C::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.items_max) * p.a.H);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, p, km, vm);
}

}  // namespace kvq
