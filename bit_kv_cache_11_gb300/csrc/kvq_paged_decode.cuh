// kvq_paged_decode.cuh — attention over the E4M3 pages for few query rows per
// kv head (kvq_paged_attention): a split of the token axis over warps.
//
// Mathematics.  With key codes a_t, value codes c_t and the page scales sk,
// sv of token t, in log2 units (kappa = softmax scale * log2 e):
//   s_t = kappa * sk_t * (q . a_t) + log2(sv_t)
//   m   = max s_t,  w_t = 2^(s_t - m + 15) <= 2^15
//   out = (sum_t w_t c_t) / (sum_t w_t / sv_t)
// The value scale rides in the exponent, so it costs one FMA a score and the
// codes themselves are the matrix operands: E4M3 converts to fp16 exactly.
// Weights, sums and outputs accumulate in fp32; the fp16 rounding of the w_t
// that multiply the codes is the only one besides the output's: half a step,
// 2^-11, of a token's weight * scale down to 2^-29 of the row's largest, and
// 2^-40 of that largest below (the factor 2^15 uses fp16's whole range, and
// 1 / sv carries 2^-15 so that the sum below stays as it is).  A second fp16
// half for the rest of a weight would double the value products; outputs are
// 16 bits, and their own rounding is as large: against 64 bits fp16 outputs are
// 2.2 .. 2.4e-4 off (relative 2-norm; fp32 weights 1.9 .. 2.2e-4), bf16 1.7e-3 with either.
//
// Split.  Every warp streams a contiguous, equal range of units of UT = 32
// (D = 128) or 64 (D = 64) tokens: 4 KB of key and 4 KB of value codes that
// TMA copies into one of its NS stages, with the 128- or 64-byte swizzle that
// makes the fragment reads free of bank conflicts.  A unit that belongs to
// several pages is several boxes.  A warp's last item stays in shared memory
// and the CTA joins its warps' shares; an item that crosses CTAs is joined by
// the CTA that arrives last, in CTA order, so results do not depend on timing.
//
// Bound: HBM while it streams (131072 tokens of 8 kv heads, 268 MB: the loops
// read 7.4 TB/s), latency around that: 4 us from the start of a launch to the
// first data (lengths, table, page, copy, one after the other) and 3 .. 6 us of
// joins.  Measured (us, and the share of the measured copy rate): 131072 tokens
// 49.7 (80 %), 8 x 4113 tokens of 32 heads 52.2 (76 %), 64 ragged requests of up to
// 2048 tokens 43.3 (57 %), five drafted tokens with a window 29.  Eight warps of
// three 8 KB stages were 3 % faster than twelve of two.  Code that runs once a
// launch is fetched as it runs: the joins are small loops, and one body of the
// unit serves edges too (together with the joins' loads in flight that took 15 %
// off the smallest call, now 8.6 us in a graph).
//
// Tensor-core operands (mma.sync m16n8k16, fp16 in, fp32 out).  Scores:
// A = 16 tokens x 16 channels of codes, B = 8 query rows.  Lane (g, t) reads
// 16-byte chunks of tokens g and g + 8; a 4-byte word gives the four
// channels of one k-step, and the query registers hold the same channels, so
// no data moves between lanes.  Values: A = 16 channels x 16 tokens; a byte
// permute pairs the codes of two tokens.  The scores' C fragment becomes the
// weights' B fragment by an 8x8 transpose (movmatrix).
//
// 4-bit pages (Q4).  A value is fp16(code * step + minimum), which one operation on
// two codes and one on the pair's steps and minima give (values4); these fp16
// numbers are the operands, and weights have no page scale in them.  ldmatrix hands
// a lane its key words as they lie (channels 8 t .. of a group, whose steps the
// token's 16 bytes of metadata hold) and, transposed, the codes of two tokens of
// four value channels in the halves of a word, so that no byte moves between
// lanes.  A unit is 5 KB; twelve warps of three stages (NT = 1) or eight of four.
// Bound: the chain from a shared-memory read over conversion and products to the
// softmax, which twelve warps of 168 registers do not hide: 456 instructions for 16
// tokens of a head (E4M3: 312), 2.07 of four issued a cycle, no pipe above 40 %.
// 131072 tokens of 8 heads, 168 MB, 52 us (47 % of the measured copy rate; 36 without
// the arithmetic, 42 without the values' conversion), no less than over E4M3 pages, 64
// ragged requests 38 us, one of 257 tokens 7.6.  Measured and not kept: eight
// warps 59 us, sixteen 52 (spills); the metadata by bulk copies 1 % slower; scores
// from the codes themselves (a product for each group, times the step) 50.2 us, but
// for keys that are not rounded to fp16, as a value's definition is: fp16 outputs
// 4.8e-4 off 64 bits instead of 2.3e-4 (fp32 weights 2.1e-4).
#pragma once

#include "kvq_decode_mma.cuh"
#include "kvq_paged4.cuh"

namespace kvq {

__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ float fast_log2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// 16 bytes into shared memory, and the arrival of the thread's copies so far.
__device__ __forceinline__ void async_copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void async_copies_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// Four 8 x 8 matrices of 16-bit units: lane (g, t) gets units 2t, 2t + 1 of row g, or
// (trans) unit g of rows 2t and 2t + 1.  Lane l names row l % 8 of matrix l / 8.
__device__ __forceinline__ void ldmatrix4(uint32_t a, uint32_t (&x)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
               : "r"(a));
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t a, uint32_t (&x)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
               : "r"(a));
}

// A token's {step, minimum} pairs of the 4-bit pages.
template <int D>
struct Meta4 {
  uint32_t m[D / 32];
  __device__ __forceinline__ void load(uint32_t a) {
    if constexpr (D == 128) {
      const uint4 v = lds128(a);
      m[0] = v.x;
      m[1] = v.y;
      m[2] = v.z;
      m[3] = v.w;
    } else {
      const uint2 v = lds64(a);
      m[0] = v.x;
      m[1] = v.y;
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) m[i] = 0;
  }
};

// Weights as fp16; one that the rounding of huge scores (over 2^22) lifts above
// fp16's largest number stays finite.
__device__ __forceinline__ uint32_t pack_weights(float lo, float hi) {
  uint32_t x;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(x) : "f"(hi), "f"(lo));
  return x;
}
constexpr float kWeightLog2 = 15.f, kWeightInv = 0x1p-15f;  // weights are 2^15 times

// What a row's sum of codes is multiplied by, from its sum of weights.
__device__ __forceinline__ float row_factor(float l) {
  return l > 0.f ? kWeightInv / l : (l == 0.f ? 0.f : l);
}

// A truth value that is known at compile time.
template <bool V>
struct Known {
  __device__ __forceinline__ operator bool() const { return V; }
};

// No page is needed (a table entry is never this: ids are below 2^31 - 1).
constexpr int kNoPage = 0x7fffffff;

template <int D, int NT, bool Q4>
struct PagedCfg {
  static constexpr int NW = paged_warps(NT, Q4);
  static constexpr int UT = paged_unit_tokens(D);  // tokens of a unit
  static constexpr int GR = UT / 16;               // 16-token granules of a unit
  static constexpr int NS = Q4 && NW == 8 ? 4 : 3;  // stages of a warp
  static constexpr int RG = 8 * NT;                // query rows of a group
  static constexpr int STAGE = Q4 ? 5120 : 8192;
  // places in a stage: keys, values, and the 4-bit pages' metadata
  static constexpr int OFF_V = Q4 ? 2048 : 4096, OFF_KM = 4096, OFF_VM = 4608;
  static constexpr int PART = RG * (D + 2);        // floats of a partial: O, then m, l
  static constexpr int RING = 64;                  // granule records of a warp
  static constexpr int OFF_BAR = NW * NS * STAGE;
  static constexpr int OFF_RING = OFF_BAR + round_up(NW * NS * 8, 128);
  static constexpr int OFF_SEG = OFF_RING + NW * RING * 16;
  static constexpr int OFF_ITEM = OFF_SEG + 1024;
  static constexpr int OFF_CUM = OFF_ITEM + NW * 4 * 48;
  static constexpr int smem(int batch) { return OFF_CUM + 4 * (batch + 1); }
  static_assert(PART * 4 <= NS * STAGE, "a warp's partial fits in its stages");
};

// An item's place: request, kv head, row group, and its units.
struct PagedItem {
  int b, h, grp;
  int u0, nu;      // first global unit, units
  int tok0;        // first token of unit 0 of the item
  int q0, rows;    // first row of q, query rows of the group
  int seq;
  int n;           // new tokens of the request
};

// A warp's part of an item, for the join.
struct PagedSeg {
  int u0, u1;      // the item's global units (u0 < 0: no segment)
  int h, grp, q0, rows;
};

template <int D, int NT, bool BF16, bool Q4>
__global__ void __launch_bounds__(PagedCfg<D, NT, Q4>::NW * 32, 1)
    paged_decode_kernel(const __grid_constant__ PagedAttnParams p,
                        const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap) {
  using C = PagedCfg<D, NT, Q4>;
  constexpr int NW = C::NW, UT = C::UT, GR = C::GR, NS = C::NS, RG = C::RG, PART = C::PART;
  constexpr int KC = D / 64;   // 16-byte chunks of a key row a lane reads
  constexpr int KS = D / 16;   // k-steps of the scores
  constexpr int MT = D / 16;   // m-tiles of the values
  extern __shared__ __align__(1024) uint8_t smem_paged[];
  uint8_t* const smem = smem_paged;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  uint8_t* stages = smem + warp * NS * C::STAGE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR) + warp * NS;
  float4* ring = reinterpret_cast<float4*>(smem + C::OFF_RING) + warp * C::RING;
  PagedSeg* segs = reinterpret_cast<PagedSeg*>(smem + C::OFF_SEG);  // [NW][2]
  PagedItem* items = reinterpret_cast<PagedItem*>(smem + C::OFF_ITEM) + warp * 4;
  int* flags = reinterpret_cast<int*>(smem + C::OFF_SEG + NW * 2 * sizeof(PagedSeg));
  int* cum = reinterpret_cast<int*>(smem + C::OFF_CUM);
  if (lane == 0) {
    for (int s = 0; s < NS; ++s) mbar_init(&bars[s], Q4 ? 33 : 1);
    fence_barrier_init();
    segs[2 * warp].u0 = segs[2 * warp + 1].u0 = -1;
    if (warp == 0) {
      tensormap_prefetch(&kmap);
      tensormap_prefetch(&vmap);
    }
  }
  grid_dep_wait();

  // ---- units of every request: prefix sum over the batch -------------------
  auto groups_of = [&](const PagedReq& r) { return (r.n * p.R + RG - 1) / RG; };
  auto units_of = [&](const PagedReq& r) {
    const int nu = (r.seq + UT - 1) / UT - first_seen(p, r) / UT;
    return nu > 1 ? nu : 1;  // an empty request still has its zero rows written
  };
  auto load_req = [&](int b, int* bad) {
    PagedReq r = paged_req(p, b, bad);
    const int rows = r.n * p.R;
    if (rows < p.row_min || rows > p.row_max) r.n = 0;
    return r;
  };
  {
    const int per = (p.batch + NW * 32 - 1) / (NW * 32);
    const int b0 = min(tid * per, p.batch), b1 = min(b0 + per, p.batch);
    int mine = 0;
    bool any_bad = false;
    auto cost = [&](int b) {
      int bad;
      const PagedReq r = load_req(b, &bad);
      any_bad |= bad != 0;
      return r.n > 0 ? p.H * groups_of(r) * units_of(r) : 0;
    };
    for (int b = b0; b < b1; ++b) mine = add_counts(mine, cost(b));
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl = add_counts(incl, x);
    }
    if (lane == 31) flags[warp] = incl;
    int at = __shfl_up_sync(0xffffffffu, incl, 1);  // the lanes' before
    if (lane == 0) at = 0;
    __syncthreads();
    for (int w = 0; w < warp; ++w) at = add_counts(at, flags[w]);
    for (int b = b0; b < b1; ++b) {
      cum[b] = at;
      at = add_counts(at, per == 1 ? mine : cost(b));
    }
    if (b1 == p.batch && b0 < b1) cum[p.batch] = at;
    if (any_bad && blockIdx.x == 0) set_err(p.err, KVQ_PAGED_ERR_LENGTH);
    __syncthreads();
  }
  grid_dep_launch();
  const int U = cum[p.batch];
  if (U == 0) return;
  if (U == kCountMax) {  // (the host refuses calls whose own rows could come to this)
    if (blockIdx.x == 0 && tid == 0) set_err(p.err, KVQ_PAGED_ERR_LENGTH);
    return;
  }
  // warps in use: at least one unit each, packed into the first CTAs
  const int W = min(p.n_warps, U);
  const int gw = blockIdx.x * NW + warp;
  auto first_of = [&](int w) { return static_cast<int>(static_cast<long long>(w) * U / W); };
  if (static_cast<int>(blockIdx.x) * NW >= W) return;
  const int ua = gw < W ? first_of(gw) : U, ub = gw < W ? first_of(gw + 1) : U;

  auto find_item = [&](int u, PagedItem& it) {
    int lo = 0, hi = p.batch;  // the last request with cum[b] <= u
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cum[mid] <= u) lo = mid;
      else hi = mid;
    }
    int bad;
    const PagedReq r = load_req(lo, &bad);
    const int G = groups_of(r), nu = units_of(r);
    const int i = (u - cum[lo]) / nu;
    it.b = lo;
    it.h = i / G;
    it.grp = i - it.h * G;
    it.u0 = cum[lo] + i * nu;
    it.nu = nu;
    it.tok0 = first_seen(p, r) / UT * UT;
    it.q0 = r.q0;
    it.rows = min(RG, r.n * p.R - it.grp * RG);
    it.seq = r.seq;
    it.n = r.n;
  };
  // Tokens [lo, hi) that any row of the group sees.
  auto seen_lo = [&](const PagedItem& it) {
    if (p.window == 0) return 0;
    const int lo = it.seq - it.n + row_token(p, it.grp * RG) + 1 - p.window;
    return lo > 0 ? lo : 0;
  };
  auto seen_hi = [&](const PagedItem& it) {
    return max(0, it.seq - it.n + row_token(p, it.grp * RG + it.rows - 1) + 1);
  };

  // ---- the load cursor, NS units ahead -------------------------------------
  PagedItem li = {};
  int lu = ua, lend = ua;      // next unit to load, end of its item
  int gbase = 0, grec = 0;     // granule records: read so far of this batch, ring position
  int llo = 0, lhi = 0;
  // The lanes hold 32 granules at a time: their pages, and in the ring their
  // scales.  The next 32 pages are requested as the current ones start, the
  // next scales half way, so neither wait stops the stream.
  int my_page = -1;
  int nx_page = -1;
  float nx_ks = 0.f, nx_vs = 1.f;  // (4-bit pages have none)
  // Page of the lane's granule when the batch starts at unit u (-1: none).
  auto granule_page = [&](int u) {
    const int tok = li.tok0 + (u - li.u0) * UT + lane * 16;
    // the granule's box, named by its first token that a row may see
    const int box = tok & ~(p.box_rows - 1);
    const int rep = max(box, llo);
    // (granules beyond this warp's range or the item are never used)
    if (rep < lhi && box + p.box_rows > llo && u + lane / GR < min(lend, ub))
      return p.table[static_cast<size_t>(li.b) * p.max_pages + (rep >> p.lg_ps)];
    return kNoPage;
  };
  auto check_page = [&](int page) {
    if (page == kNoPage) return -1;
    if (page >= 0 && page < p.n_pages) return page;
    set_err(p.err, KVQ_PAGED_ERR_BAD_PAGE);
    return -1;
  };
  auto granule_scales = [&](int page, float* ks, float* vs) {
    if (Q4 || page < 0) return;
    const size_t at = static_cast<size_t>(page) * p.H + li.h;
    *ks = p.k_scale[at];
    *vs = p.v_scale[at];
  };
  int n_items = 0;  // items entered by the load cursor
  // The lane's record of the batch that started at unit u0b, ring place rec0.
  auto put_record = [&](int u0b, int rec0, float ks, float vs) {
    const int tok = li.tok0 + (u0b - li.u0) * UT + lane * 16;
    const bool seen = my_page >= 0 && tok < lhi && tok + 16 > llo;
    ring[(rec0 + lane) & (C::RING - 1)] =
        Q4 ? make_float4(1.f, 0.f, kWeightInv, seen ? 1.f : 0.f)
           : make_float4(ks, fast_log2(vs), kWeightInv / vs, seen ? 1.f : 0.f);
  };
  const int nbox = UT / p.box_rows;  // boxes of a side
  // lane i < nbox copies key box i, lane nbox + i value box i; every lane copies 16
  // bytes of the 4-bit pages' metadata a side
  const bool key = lane < nbox;
  const int bx = key ? lane : lane - nbox;
  constexpr int ROW = Q4 ? D / 2 : D;  // bytes of a row of codes
  const uint32_t box_bytes = static_cast<uint32_t>(p.box_rows) * ROW;
  const int box_g = bx * (p.box_rows / 16) & (GR - 1);  // first granule of the lane's box
  auto issue = [&](int s) {
    const int u_first = lu, rec_first = grec;
    const bool fresh = lu == lend;
    float ks = 0.f, vs = 1.f;
    if (fresh) {
      find_item(lu, li);
      lend = li.u0 + li.nu;
      llo = seen_lo(li);
      lhi = seen_hi(li);
      if (lane == 0) items[n_items & 3] = li;
      ++n_items;
      my_page = check_page(granule_page(lu));
      granule_scales(my_page, &ks, &vs);  // on their way while the copies start
      gbase = 0;
    } else if (gbase == 32) {
      my_page = nx_page;
      put_record(lu, grec, nx_ks, nx_vs);
      gbase = 0;
    } else if (gbase == 16) {
      nx_page = check_page(nx_page);
      nx_ks = 0.f;
      nx_vs = 1.f;
      granule_scales(nx_page, &nx_ks, &nx_vs);
    }
    const int page = __shfl_sync(0xffffffffu, my_page, gbase + box_g);
    const bool mine = lane < 2 * nbox && page >= 0;
    const int n = __popc(__ballot_sync(0xffffffffu, mine));
    if (lane == 0) mbar_arrive_expect_tx(&bars[s], n * box_bytes);
    __syncwarp();
    const int tok0 = li.tok0 + (lu - li.u0) * UT;
    auto row_of = [&](int pg, int tok) { return ((pg * p.H + li.h) << p.lg_ps) + (tok & ((1 << p.lg_ps) - 1)); };
    uint8_t* st = stages + s * C::STAGE;
    if (mine)
      tma_load_2d(st + (key ? 0 : C::OFF_V) + bx * box_bytes, key ? &kmap : &vmap, 0,
                  row_of(page, tok0 + bx * p.box_rows), &bars[s]);
    if constexpr (Q4) {
      const int tok = lane * (128 / D);  // the lane's token of the unit
      const int pg = __shfl_sync(0xffffffffu, my_page, gbase + tok / 16);
      if (pg >= 0) {
        const size_t at = static_cast<size_t>(row_of(pg, tok0 + tok)) * (D / kGroup4);
        async_copy16(st + C::OFF_KM + lane * 16, p.meta[0] + at);
        async_copy16(st + C::OFF_VM + lane * 16, p.meta[1] + at);
      }
      async_copies_arrive(&bars[s]);
    }
    if (fresh) put_record(u_first, rec_first, ks, vs);
    if (gbase == 0) nx_page = granule_page(lu + 32 / GR);
    gbase += GR;
    grec += GR;
    ++lu;
    __syncwarp();
  };
#pragma unroll
  for (int s = 0; s < NS; ++s)
    if (lu < ub) issue(s);

  // ---- compute ---------------------------------------------------------------
  uint32_t qf[NT][KS][2];
  float acc[MT][NT][4];
  float m[NT][2], l[NT][2], cq[NT][2];
  PagedItem it = {};
  int iend = ua;               // end of the current item
  int lo = 0, hi = 0, full_lo = 0, full_hi = 0;
  int crec = 0;                // ring position of the unit's first granule
  bool failed = false;

  int k_items = 0;  // items entered here
  auto enter = [&]() {
    it = items[k_items & 3];
    ++k_items;
    iend = it.u0 + it.nu;
    lo = seen_lo(it);
    hi = seen_hi(it);
    // tokens [full_lo, full_hi) are seen by every row of the group
    full_hi = it.seq - it.n + row_token(p, it.grp * RG) + 1;
    full_lo = p.window == 0 ? 0 : hi - p.window;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = nt * 8 + g;  // this lane's query row
      float c = p.qscale;
      uint32_t w[KS * 2];
#pragma unroll
      for (int i = 0; i < KS * 2; ++i) w[i] = 0;
      if (r < it.rows) {
        const int row = it.grp * RG + r;
        const int j = row_token(p, row);
        const uint4* src = reinterpret_cast<const uint4*>(
            static_cast<const uint16_t*>(p.q) + static_cast<long long>(it.q0 + j) * p.q_stride +
            (static_cast<long long>(it.h) * p.R + (row - j * p.R)) * D + t * (Q4 ? 8 : D / 4));
#pragma unroll
        for (int i = 0; i < KS / 2; ++i) {
          const uint4 v = src[Q4 ? 4 * i : i];
          w[4 * i] = v.x;
          w[4 * i + 1] = v.y;
          w[4 * i + 2] = v.z;
          w[4 * i + 3] = v.w;
        }
      }
      if constexpr (BF16) {
        // The row times a power of two as fp16: its largest element comes to
        // [2^14, 2^15), so elements down to 2^-22 of it keep all their bits
        // and the rest an absolute error below 2^-40 of it.
        uint32_t mg = 0;
#pragma unroll
        for (int i = 0; i < KS * 2; ++i) mg = __vmaxu2(mg, w[i] & 0x7fff7fffu);
        uint32_t mx = max(mg & 0xffffu, mg >> 16);
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int e = max(static_cast<int>(mx >> 7) - 127, -100);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
        c *= __uint_as_float(static_cast<uint32_t>(127 - 14 + e) << 23);
#pragma unroll
        for (int i = 0; i < KS * 2; ++i)
          w[i] = pack_half2(__uint_as_float(w[i] << 16) * up,
                            __uint_as_float(w[i] & 0xffff0000u) * up);
      }
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        qf[nt][i][0] = w[2 * i];
        qf[nt][i][1] = w[2 * i + 1];
      }
      // columns 2t, 2t + 1 of the score fragment are rows of other lanes
      cq[nt][0] = __shfl_sync(0xffffffffu, c, 8 * t);
      cq[nt][1] = __shfl_sync(0xffffffffu, c, 8 * t + 4);
#pragma unroll
      for (int c2 = 0; c2 < 2; ++c2) {
        m[nt][c2] = -INFINITY;
        l[nt][c2] = 0.f;
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[mt][nt][i] = 0.f;
    }
  };

  // This lane's places in a stage: its key chunks of token g (token g + 8 is
  // 8 rows on, under the same swizzle), its value chunk of tokens 2t, 2t + 1.
  uint32_t koff[KC], voff[2];
#pragma unroll
  for (int c = 0; c < KC; ++c)
    koff[c] = D == 128 ? g * 128 + (((2 * t + c) ^ g) << 4) : g * 64 + ((t ^ (g >> 1)) << 4);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    voff[i] = C::OFF_V + (D == 128 ? (2 * t + i) * 128 + ((g ^ (2 * t + i)) << 4)
                               : (2 * t + i) * 64 + (((g >> 1) ^ t) << 4) + 8 * (g & 1));
  // 4-bit pages: the lane's row of a matrix pair that ldmatrix reads, tokens 0 .. 15
  // of group 0 and 1 (the next two groups are 32 bytes on, under the swizzle).
  uint32_t moff = 0;
  if constexpr (Q4) {
    const int row = (lane & 7) + (lane & 8), chunk = lane >> 4;
    moff = D == 128 ? row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4) : row * 32 + ((chunk ^ ((row >> 2) & 1)) << 4);
  }
  const uint32_t stages_s = smem_addr(stages);

  // One unit from stage memory.  edge: some of its tokens are hidden from some
  // rows (or not there at all).
  float4 rec[GR];  // the unit's granule records
  auto compute = [&](uint32_t st, int tok, auto at_edge) {
    const bool edge = at_edge;
    uint32_t pw[GR][NT][2];
    float s[GR][NT][4];
#pragma unroll
    for (int mt = 0; mt < GR; ++mt) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[mt][nt][i] = 0.f;
      if constexpr (Q4) {
        // words of channels 32 w + 8 t .. of tokens g and g + 8, and the tokens'
        // steps and minima
        const uint32_t meta = st + C::OFF_KM + (mt * 16 + g) * (D / 8);
        Meta4<D> ma, mb;
        ma.load(meta);
        mb.load(meta + D);
#pragma unroll
        for (int w = 0; w < D / 32; w += 2) {
          uint32_t x[4];
          ldmatrix4((st + mt * 8 * D + moff) ^ (16 * w), x);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t a[4], b[4];
            values4(x[2 * i], as_word(__low2half2(as_half2(ma.m[w + i]))), as_word(__high2half2(as_half2(ma.m[w + i]))), a);
            values4(x[2 * i + 1], as_word(__low2half2(as_half2(mb.m[w + i]))), as_word(__high2half2(as_half2(mb.m[w + i]))), b);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const int ks = 2 * (w + i);
              mma_16816(s[mt][nt], a[0], b[0], a[1], b[1], qf[nt][ks][0], qf[nt][ks][1]);
              mma_16816(s[mt][nt], a[2], b[2], a[3], b[3], qf[nt][ks + 1][0], qf[nt][ks + 1][1]);
            }
          }
        }
      } else {
#pragma unroll
        for (int c = 0; c < KC; ++c) {
          const uint4 a = lds128(st + koff[c] + mt * 16 * D);
          const uint4 b = lds128(st + koff[c] + (mt * 16 + 8) * D);
          const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_half2x2(aw[w], a0, a2);
            e4m3x4_to_half2x2(bw[w], a1, a3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_16816(s[mt][nt], a0, a1, a2, a3, qf[nt][4 * c + w][0], qf[nt][4 * c + w][1]);
          }
        }
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int mt = 0; mt < GR; ++mt) {
        const float f0 = Q4 ? cq[nt][0] : rec[mt].x * cq[nt][0], f1 = Q4 ? cq[nt][1] : rec[mt].x * cq[nt][1];
        const float lv = Q4 ? 0.f : rec[mt].y;
        float* x = s[mt][nt];
        x[0] = fmaf(x[0], f0, lv);
        x[1] = fmaf(x[1], f1, lv);
        x[2] = fmaf(x[2], f0, lv);
        x[3] = fmaf(x[3], f1, lv);
        if (edge) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int row = it.grp * RG + nt * 8 + 2 * t + c;
            const int pos = it.seq - it.n + row_token(p, row);
            const int first = p.window == 0 ? 0 : pos - p.window + 1;
            const int ta = tok + mt * 16 + g, tb = ta + 8;
            const bool there = rec[mt].w != 0.f;
            if (!there || ta > pos || ta < first) x[c] = -INFINITY;
            if (!there || tb > pos || tb < first) x[2 + c] = -INFINITY;
          }
        }
        mx[0] = fmaxf(mx[0], fmaxf(x[0], x[2]));
        mx[1] = fmaxf(mx[1], fmaxf(x[1], x[3]));
      }
      float al[2], mb[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], 4));
        mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], 8));
        mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], 16));
        const float mn = fmaxf(m[nt][c], mx[c]);
        mb[c] = mn == -INFINITY ? 0.f : mn;
        al[c] = fast_exp2(m[nt][c] - mb[c]);
        m[nt][c] = mn;
        l[nt][c] *= al[c];
        mb[c] -= kWeightLog2;
      }
#pragma unroll
      for (int mt = 0; mt < GR; ++mt) {
        float* x = s[mt][nt];
        x[0] = fast_exp2(x[0] - mb[0]);
        x[1] = fast_exp2(x[1] - mb[1]);
        x[2] = fast_exp2(x[2] - mb[0]);
        x[3] = fast_exp2(x[3] - mb[1]);
        const float wi = Q4 ? kWeightInv : rec[mt].z;
        l[nt][0] = fmaf(x[0] + x[2], wi, l[nt][0]);
        l[nt][1] = fmaf(x[1] + x[3], wi, l[nt][1]);
        pw[mt][nt][0] = movmatrix(pack_weights(x[0], x[1]));
        pw[mt][nt][1] = movmatrix(pack_weights(x[2], x[3]));
      }
      if (__any_sync(0xffffffffu, al[0] != 1.f || al[1] != 1.f)) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          acc[mt][nt][0] *= al[0];
          acc[mt][nt][1] *= al[1];
          acc[mt][nt][2] *= al[0];
          acc[mt][nt][3] *= al[1];
        }
      }
    }
#pragma unroll
    for (int mt = 0; mt < GR; ++mt) {
      if constexpr (Q4) {
        // Transposed matrices: channels 32 w + 4 g .. + 3 of tokens 2t and 2t + 1
        // (2t + 8 and 2t + 9) in the halves of a word.
        Meta4<D> mv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tr = mt * 16 + 2 * t + (i & 1) + 8 * (i >> 1);
          mv[i].load(st + C::OFF_VM + tr * (D / 8));
          // (what lies in hidden rows may be NaN, which a weight of 0 would not cancel)
          if (edge && (tok + tr < lo || tok + tr >= hi || rec[mt].w == 0.f)) mv[i].clear();
        }
#pragma unroll
        for (int w = 0; w < D / 32; w += 2) {
          uint32_t x[4];
          ldmatrix4_trans((st + C::OFF_V + mt * 8 * D + moff) ^ (16 * w), x);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t a[4], b[4];
            values4(x[2 * i], pair_lo(mv[0].m[w + i], mv[1].m[w + i]), pair_hi(mv[0].m[w + i], mv[1].m[w + i]), a);
            values4(x[2 * i + 1], pair_lo(mv[2].m[w + i], mv[3].m[w + i]), pair_hi(mv[2].m[w + i], mv[3].m[w + i]), b);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_16816(acc[2 * (w + i)][nt], a[0], a[1], b[0], b[1], pw[mt][nt][0], pw[mt][nt][1]);
              mma_16816(acc[2 * (w + i) + 1][nt], a[2], a[3], b[2], b[3], pw[mt][nt][0], pw[mt][nt][1]);
            }
          }
        }
      } else {
        // value rows of tokens 2t, 2t + 1, 2t + 8, 2t + 9 of the granule:
        // channels [D/8 * g, D/8 * (g + 1))
        constexpr int VW = D / 32;  // words of a lane's row
        uint32_t v[4][VW];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t at = st + voff[i & 1] + (mt * 16 + 8 * (i >> 1)) * D;
          if constexpr (D == 128) {
            const uint4 x = lds128(at);
            v[i][0] = x.x;
            v[i][1] = x.y;
            v[i][2] = x.z;
            v[i][3] = x.w;
          } else {
            const uint2 x = lds64(at);
            v[i][0] = x.x;
            v[i][1] = x.y;
          }
          if (edge) {
            // what lies in hidden rows may decode to NaN, which a weight of 0
            // would not cancel
            const int tk = tok + mt * 16 + 2 * t + (i & 1) + 8 * (i >> 1);
            if (tk < lo || tk >= hi || rec[mt].w == 0.f) {
#pragma unroll
              for (int w = 0; w < VW; ++w) v[i][w] = 0;
            }
          }
        }
#pragma unroll
        for (int w = 0; w < VW; ++w) {
          const uint32_t x0 = __byte_perm(v[0][w], v[1][w], 0x5140), x1 = __byte_perm(v[0][w], v[1][w], 0x7362);
          const uint32_t y0 = __byte_perm(v[2][w], v[3][w], 0x5140), y1 = __byte_perm(v[2][w], v[3][w], 0x7362);
          uint32_t a0, a1, a2, a3, b0, b1, b2, b3;
          e4m3x4_to_half2x2(x0, a0, a1);
          e4m3x4_to_half2x2(y0, a2, a3);
          e4m3x4_to_half2x2(x1, b0, b1);
          e4m3x4_to_half2x2(y1, b2, b3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_16816(acc[2 * w][nt], a0, a1, a2, a3, pw[mt][nt][0], pw[mt][nt][1]);
            mma_16816(acc[2 * w + 1][nt], b0, b1, b2, b3, pw[mt][nt][0], pw[mt][nt][1]);
          }
        }
      }
    }
  };

  // The first of this lane's channels in m-tile mt.
  auto channel = [&](int mt) { return Q4 ? mt / 2 * 32 + 4 * g + 2 * (mt & 1) : g * (D / 8) + 2 * mt; };
  // Leaves the current item after unit u - 1: a finished output, or a partial.
  auto leave = [&](bool last) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], 4);
        l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], 8);
        l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], 16);
      }
    const bool whole = it.u0 >= ua && iend <= ub;
    if (whole) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int r = nt * 8 + 2 * t + c;
          if (r >= it.rows) continue;
          const int row = it.grp * RG + r, j = row_token(p, row);
          const float inv = row_factor(l[nt][c]);
          uint32_t w[D / 16];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const float x = acc[mt][nt][c] * inv, y = acc[mt][nt][2 + c] * inv;
            if constexpr (BF16) {
              const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
              w[mt] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
              w[mt] = pack_half2(x, y);
            }
          }
          uint16_t* head = static_cast<uint16_t*>(p.out) + static_cast<long long>(it.q0 + j) * p.out_stride +
                           (static_cast<long long>(it.h) * p.R + (row - j * p.R)) * D;
          if constexpr (Q4) {
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
              *reinterpret_cast<uint2*>(head + channel(2 * i)) = make_uint2(w[2 * i], w[2 * i + 1]);
          } else {
            uint4* dst = reinterpret_cast<uint4*>(head + channel(0));
#pragma unroll
            for (int i = 0; i < D / 64; ++i)
              dst[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
          }
        }
      return;
    }
    float* dst = last ? reinterpret_cast<float*>(stages)
                      : p.warp_part + static_cast<size_t>(gw) * PART;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = nt * 8 + 2 * t + c;
#pragma unroll
        for (int mt = 0; mt < MT; mt += 2) {
          *reinterpret_cast<float4*>(dst + r * D + channel(mt)) =
              make_float4(acc[mt][nt][c], acc[mt][nt][2 + c], acc[mt + 1][nt][c], acc[mt + 1][nt][2 + c]);
        }
        if (g == 0) {
          dst[RG * D + 2 * r] = m[nt][c];
          dst[RG * D + 2 * r + 1] = l[nt][c];
        }
      }
    if (lane == 0) {
      PagedSeg& sg = segs[2 * warp + (last ? 1 : 0)];
      sg.u0 = it.u0;
      sg.u1 = iend;
      sg.h = it.h;
      sg.grp = it.grp;
      sg.q0 = it.q0;
      sg.rows = it.rows;
    }
  };

  int st = 0;
  uint32_t phase = 0;
  for (int u = ua; u < ub; ++u) {
    if (u == iend) {
      if (u > ua) leave(false);
      if (failed) {
        find_item(u, li);
        if (lane == 0) items[k_items & 3] = li;
        __syncwarp();
      }
      enter();
    }
    // (decided for the whole warp: its lanes stay together)
    if (!failed && !__all_sync(0xffffffffu, mbar_wait_bounded(&bars[st], phase, min(p.wait_limit, kWaitLimit)))) {
      // A copy did not arrive in time: record it and let the warp's copies land
      // (bounded).  The warp goes on without data from item to item, so that the
      // shares that it owes are there, every CTA of a shared item draws its
      // ticket and the tickets return to zero.
      failed = true;
      set_err(p.err, KVQ_PAGED_ERR_WAIT);
      for (int k = u; k < lu; ++k) {
        mbar_wait_bounded(&bars[st], phase);
        if (++st == NS) {
          st = 0;
          phase ^= 1;
        }
      }
      __syncwarp();
    }
    if (failed) {
      u = min(iend, ub) - 1;
      continue;
    }
    const int tok = it.tok0 + (u - it.u0) * UT;
    if (tok < hi && tok + UT > lo) {
      const uint32_t sp = stages_s + st * C::STAGE;
      bool there = true;
#pragma unroll
      for (int i = 0; i < GR; ++i) {
        rec[i] = ring[(crec + i) & (C::RING - 1)];
        there &= rec[i].w != 0.f;
      }
      const bool edge = !there || tok < full_lo || tok + UT > full_hi;
      if constexpr (Q4) {
        if (edge) compute(sp, tok, Known<true>{});
        else compute(sp, tok, Known<false>{});
      } else {
        compute(sp, tok, edge);
      }
    }
    crec += GR;
    __syncwarp();
    if (lu < ub) issue(st);
    if (++st == NS) {
      st = 0;
      phase ^= 1;
    }
  }
  if (ua < ub) leave(true);

  // ---- the CTA's join ---------------------------------------------------------
  // Every warp lists the segments (two a warp: the partial it left on its way,
  // in global memory, and its last one, in its stages) and their groups, runs
  // of segments of one item; then each takes (group, row) tasks in turn.
  __syncthreads();
  const int cu0 = first_of(min(static_cast<int>(blockIdx.x) * NW, W));
  const int cu1 = first_of(min((static_cast<int>(blockIdx.x) + 1) * NW, W));
  const int cta = blockIdx.x;
  PagedSeg sg = {-1, -1, 0, 0, 0, 0};
  if (lane < 2 * NW) sg = segs[lane];
  const uint32_t valid = __ballot_sync(0xffffffffu, sg.u0 >= 0);
  const uint32_t below = valid & ((1u << lane) - 1);
  const int before = __shfl_sync(0xffffffffu, sg.u0, below ? 31 - __clz(below) : 0);
  const uint32_t leaders = __ballot_sync(0xffffffffu, sg.u0 >= 0 && (!below || before != sg.u0));
  const int n_groups = __popc(leaders);
  const float* mine = lane & 1 ? reinterpret_cast<const float*>(smem + (lane >> 1) * NS * C::STAGE)
                               : p.warp_part + static_cast<size_t>(cta * NW + (lane >> 1)) * PART;
  constexpr int VL = D / 4;     // lanes that hold a row as float4
  const int ch = lane % VL * 4;
  const bool writes = lane < VL;

  // Row r of a finished item.
  auto finish = [&](int h, int grp, int q0, int r, float L, float4 o) {
    const int row = grp * RG + r, j = row_token(p, row);
    const float inv = row_factor(L);
    uint2 w;
    if constexpr (BF16) {
      const __nv_bfloat162 a = __floats2bfloat162_rn(o.x * inv, o.y * inv);
      const __nv_bfloat162 b = __floats2bfloat162_rn(o.z * inv, o.w * inv);
      w = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    } else {
      w = make_uint2(pack_half2(o.x * inv, o.y * inv), pack_half2(o.z * inv, o.w * inv));
    }
    if (writes)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) +
                                static_cast<long long>(q0 + j) * p.out_stride +
                                (static_cast<long long>(h) * p.R + (row - j * p.R)) * D + ch) = w;
  };

  uint32_t open = 0;  // leaders of groups that other CTAs share
  for (int k = 0, task = 0; k < n_groups; ++k) {
    uint32_t rest = leaders;
    for (int i = 0; i < k; ++i) rest &= rest - 1;
    const int lead = __ffs(rest) - 1;
    rest &= rest - 1;
    const uint32_t upto = rest ? (1u << (__ffs(rest) - 1)) - 1 : 0xffffffffu;
    const uint32_t members = valid & upto & ~((1u << lead) - 1);
    const int u0 = __shfl_sync(0xffffffffu, sg.u0, lead), u1 = __shfl_sync(0xffffffffu, sg.u1, lead);
    const int h = __shfl_sync(0xffffffffu, sg.h, lead), grp = __shfl_sync(0xffffffffu, sg.grp, lead);
    const int q0 = __shfl_sync(0xffffffffu, sg.q0, lead), rows = __shfl_sync(0xffffffffu, sg.rows, lead);
    const bool starts = u0 >= cu0, whole = starts && u1 <= cu1;
    if (!whole) open |= 1u << lead;
    float* slot = p.cta_part + static_cast<size_t>(2 * cta + (starts ? 1 : 0)) * PART;
    auto put = [&](int r, float M, float L, float4 o) {
      if (whole) {
        finish(h, grp, q0, r, L, o);
      } else {
        if (writes) *reinterpret_cast<float4*>(slot + r * D + ch) = o;
        if (lane == 0) *reinterpret_cast<float2*>(slot + RG * D + 2 * r) = make_float2(M, L);
      }
    };
    if (__popc(members) <= 2) {
      // One or two members (many short items): one warp joins the group's
      // rows, all their loads on their way at once.  Lane 16 i + r weighs row
      // r of member i.
      if (task++ % NW != warp) continue;
      const int ma = lead, mb_ = 31 - __clz(members);
      const bool two = mb_ != ma;
      const float* pa = reinterpret_cast<const float*>(
          __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), ma));
      const float* pb = reinterpret_cast<const float*>(
          __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), mb_));
      float2 ml = make_float2(-INFINITY, 0.f);
      const int rr = lane & 15;
      if (rr < RG && (lane < 16 || two))
        ml = *reinterpret_cast<const float2*>((lane < 16 ? pa : pb) + RG * D + 2 * rr);
      const float M = fmaxf(ml.x, __shfl_xor_sync(0xffffffffu, ml.x, 16));
      const float w = lane < 16 || two ? fast_exp2(ml.x - (M == -INFINITY ? 0.f : M)) : 0.f;
      float L = ml.y * w;
      L += __shfl_xor_sync(0xffffffffu, L, 16);
      float4 a[4], b[4], na[4], nb[4];
      auto fetch = [&](int r0, float4(&xa)[4], float4(&xb)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          xa[i] = *reinterpret_cast<const float4*>(pa + (r0 + i) * D + ch);
          xb[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (two) xb[i] = *reinterpret_cast<const float4*>(pb + (r0 + i) * D + ch);
        }
      };
      fetch(0, na, nb);
#pragma unroll 1
      for (int r0 = 0; r0 < rows; r0 += 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = na[i];
          b[i] = nb[i];
        }
        if (r0 + 4 < rows) fetch(r0 + 4, na, nb);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = r0 + i;
          const float wa = __shfl_sync(0xffffffffu, w, r), wb = __shfl_sync(0xffffffffu, w, 16 + r);
          const float Mr = __shfl_sync(0xffffffffu, M, r), Lr = __shfl_sync(0xffffffffu, L, r);
          if (r < rows)
            put(r, Mr, Lr, make_float4(fmaf(a[i].x, wa, b[i].x * wb), fmaf(a[i].y, wa, b[i].y * wb),
                                       fmaf(a[i].z, wa, b[i].z * wb), fmaf(a[i].w, wa, b[i].w * wb)));
        }
      }
      continue;
    }
    for (int r = 0; r < rows; ++r, ++task) {
      if (task % NW != warp) continue;
      const bool in = (members >> lane) & 1;
      float2 ml = make_float2(-INFINITY, 0.f);
      if (in) ml = *reinterpret_cast<const float2*>(mine + RG * D + 2 * r);
      float M = ml.x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      const float w = in ? fast_exp2(ml.x - (M == -INFINITY ? 0.f : M)) : 0.f;
      const float L = warp_sum(in ? ml.y * w : 0.f);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (uint32_t left = members; left;) {
        float4 x[4];
        float ws[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // up to four loads on their way
          const int src = left ? __ffs(left) - 1 : lead;
          const float* at = reinterpret_cast<const float*>(
              __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), src));
          ws[i] = __shfl_sync(0xffffffffu, w, src);
          x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (left) x[i] = *reinterpret_cast<const float4*>(at + r * D + ch);
          else ws[i] = 0.f;
          left &= left - 1;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          o.x = fmaf(x[i].x, ws[i], o.x);
          o.y = fmaf(x[i].y, ws[i], o.y);
          o.z = fmaf(x[i].z, ws[i], o.z);
          o.w = fmaf(x[i].w, ws[i], o.w);
        }
      }
      put(r, M, L, o);
    }
  }
  if (open) {
    // At most two groups of a CTA are shared, its first and its last.  The
    // CTAs of an item are those of its first to its last unit; the one that
    // draws the last ticket joins them, in their order.
    auto owner = [&](int u) {
      return static_cast<int>(((static_cast<long long>(u) + 1) * W - 1) / U) / NW;
    };
    __threadfence();
    __syncthreads();
    if (warp == 0 && ((open >> lane) & 1)) {
      const int ca = owner(sg.u0), cb = owner(sg.u1 - 1);
      const int seen = atomicAdd(&p.tickets[ca], 1);
      const bool all = seen == cb - ca;
      if (all) p.tickets[ca] = 0;  // nobody else comes: ready for the next launch
      flags[lane] = all;
    }
    __syncthreads();
    for (uint32_t todo = open; todo; todo &= todo - 1) {
      const int lead = __ffs(todo) - 1;
      if (!flags[lead]) continue;
      __threadfence();
      const int u0 = __shfl_sync(0xffffffffu, sg.u0, lead), u1 = __shfl_sync(0xffffffffu, sg.u1, lead);
      const int h = __shfl_sync(0xffffffffu, sg.h, lead), grp = __shfl_sync(0xffffffffu, sg.grp, lead);
      const int q0 = __shfl_sync(0xffffffffu, sg.q0, lead), rows = __shfl_sync(0xffffffffu, sg.rows, lead);
      const int ca = owner(u0), cb = owner(u1 - 1);
      auto part = [&](int c) {
        return p.cta_part + static_cast<size_t>(2 * c + (c == ca ? 1 : 0)) * PART;
      };
      if (cb == ca + 1) {
        // two shares (many items): all rows of a warp on their way at once
        const float *pa = part(ca), *pb = part(cb);
        constexpr int RW = (RG + NW - 1) / NW;  // rows of a warp
        float2 ma[RW], mb_[RW];
        float4 xa[RW], xb[RW];
#pragma unroll
        for (int i = 0; i < RW; ++i) {
          const int r = min(warp + i * NW, RG - 1);
          ma[i] = __ldcg(reinterpret_cast<const float2*>(pa + RG * D + 2 * r));
          mb_[i] = __ldcg(reinterpret_cast<const float2*>(pb + RG * D + 2 * r));
          xa[i] = __ldcg(reinterpret_cast<const float4*>(pa + r * D + ch));
          xb[i] = __ldcg(reinterpret_cast<const float4*>(pb + r * D + ch));
        }
#pragma unroll
        for (int i = 0; i < RW; ++i) {
          const int r = warp + i * NW;
          if (r >= rows) continue;  // (its floats were never written)
          const float M = fmaxf(ma[i].x, mb_[i].x), mz = M == -INFINITY ? 0.f : M;
          const float wa = fast_exp2(ma[i].x - mz), wb = fast_exp2(mb_[i].x - mz);
          finish(h, grp, q0, r, fmaf(ma[i].y, wa, mb_[i].y * wb),
                 make_float4(fmaf(xa[i].x, wa, xb[i].x * wb), fmaf(xa[i].y, wa, xb[i].y * wb),
                             fmaf(xa[i].z, wa, xb[i].z * wb), fmaf(xa[i].w, wa, xb[i].w * wb)));
        }
        continue;
      }
      for (int r = warp; r < rows; r += NW) {
        float M = -INFINITY;
        for (int c = ca + lane; c <= cb; c += 32) M = fmaxf(M, __ldcg(part(c) + RG * D + 2 * r));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        const float mb = M == -INFINITY ? 0.f : M;
        float L = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = ca; c <= cb; c += 8) {
          float4 x[8];
          float2 ml[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float* at = part(min(c + i, cb));
            ml[i] = __ldcg(reinterpret_cast<const float2*>(at + RG * D + 2 * r));
            x[i] = __ldcg(reinterpret_cast<const float4*>(at + r * D + ch));
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (c + i > cb) continue;
            const float w = fast_exp2(ml[i].x - mb);
            L = fmaf(ml[i].y, w, L);
            o.x = fmaf(x[i].x, w, o.x);
            o.y = fmaf(x[i].y, w, o.y);
            o.z = fmaf(x[i].z, w, o.z);
            o.w = fmaf(x[i].w, w, o.w);
          }
        }
        finish(h, grp, q0, r, L, o);
      }
    }
  }
}

template <int D, int NT, bool BF16, bool Q4>
cudaError_t launch_paged_decode_t(const PagedAttnParams& p, const CUtensorMap& km,
                                  const CUtensorMap& vm, cudaStream_t st) {
  using C = PagedCfg<D, NT, Q4>;
  auto fn = paged_decode_kernel<D, NT, BF16, Q4>;
  const int smem = C::smem(p.batch);
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(fn), C::smem(kPagedMaxBatch));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.n_warps / C::NW);
  cfg.blockDim = dim3(C::NW * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, p, km, vm);
}

}  // namespace kvq
