// kvq_paged_store.cu — new keys and values into the E4M3 pages
// (kvq_paged_store).
//
// For every page and kv head that receives rows, with amax over the new rows'
// finite elements:
//   e     = the least exponent in [-15, 40] with amax <= 448 * 2^e
//   scale = max(2^e, the page's scale when it holds older rows)
//   code  = E4M3(x / scale), nearest even, saturating (NaN: code 0)
// and when the scale grows, the older rows' codes c become E4M3(c * old /
// scale).  Scales are powers of two, so x / scale is exact in fp32 and every
// code is rounded once; E4M3 keeps the same relative precision at any power
// of two, which is why a finer scale would gain nothing above its subnormals.
//
// A run is a maximal sequence of tokens whose slots are consecutive rows of
// one page; its first token leads it and whoever finds a leader stores the
// whole run, so no two CTAs touch the same page and head.
//
// Bound: HBM for prompts (3 bytes a value: 2 read, 1 written), latency for
// single tokens.  Measured: 26298 tokens x 8 heads x 128, 162 MB, 28.8 us (83 %
// of the measured copy rate); 4861 tokens x 32 heads x 64 in 16-row pages, 60 MB,
// 14.3 us (62 %; the launch and the last CTAs take the rest); 256 single tokens
// 2.4 us.  One test per side for NaN instead of two selects a value, and fp16
// codes without a step through fp32, took 31 -> 29 and 16 -> 14.5 us.
#include "kvq_rotary.cuh"

namespace kvq {
namespace {

// Magnitude bits of two 16-bit floats: ordered as unsigned halves, NaN above
// infinity above the finite values.
__device__ __forceinline__ uint32_t mag2(uint32_t w) { return w & 0x7fff7fffu; }

template <bool BF16>
__device__ __forceinline__ uint32_t inf_bits() {
  return BF16 ? 0x7f80u : 0x7c00u;
}

template <bool BF16>
__device__ __forceinline__ float2 to_float2(uint32_t w) {
  if constexpr (BF16) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  } else {
    const __half2 h = *reinterpret_cast<const __half2*>(&w);
    return __half22float2(h);
  }
}

// Largest of a 16-byte vector's eight magnitudes, as bits.
__device__ __forceinline__ uint32_t vec_max(uint4 v, uint32_t m2) {
  m2 = __vmaxu2(m2, mag2(v.x));
  m2 = __vmaxu2(m2, mag2(v.y));
  m2 = __vmaxu2(m2, mag2(v.z));
  return __vmaxu2(m2, mag2(v.w));
}
// The same over the finite elements only.
template <bool BF16>
__device__ __forceinline__ uint32_t vec_max_finite(uint4 v, uint32_t m2) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t a = mag2(w[i]);
    if ((a & 0xffffu) >= inf_bits<BF16>()) a &= 0xffff0000u;
    if ((a >> 16) >= inf_bits<BF16>()) a &= 0xffffu;
    m2 = __vmaxu2(m2, a);
  }
  return m2;
}
__device__ __forceinline__ uint32_t fold2(uint32_t m2) { return max(m2 & 0xffffu, m2 >> 16); }

// The least exponent in range with |value| <= 448 * 2^e = 1.75 * 2^(e + 8).
__device__ __forceinline__ int exp_for(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, kPagedMinExp), kPagedMaxExp);
}
template <bool BF16>
__device__ __forceinline__ int exp_for_bits(uint32_t mag) {
  float a;
  if constexpr (BF16) a = __uint_as_float(mag << 16);
  else a = __half2float(__ushort_as_half(static_cast<unsigned short>(mag)));
  return exp_for(a);
}
// Exponent of a stored scale, rounded up to a power of two of the range;
// kPagedMinExp when it is no positive finite number (a page nothing was
// stored into).
__device__ __forceinline__ int exp_of_scale(float s) {
  if (!(s > 0.f) || !isfinite(s)) return kPagedMinExp;
  const uint32_t b = __float_as_uint(s);
  const int e = static_cast<int>(b >> 23) - 127 + ((b & 0x7fffffu) ? 1 : 0);
  return min(max(e, kPagedMinExp), kPagedMaxExp);
}
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

__device__ __forceinline__ uint32_t codes2(float2 x) {
  return __nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
}

// Two fp16 pairs -> four E4M3 codes, nearest even.
__device__ __forceinline__ uint32_t codes4(uint32_t lo, uint32_t hi) {
  uint32_t c;
  asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f16x2 l, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 h, %2;\n\tmov.b32 %0, {l, h};\n\t}"
      : "=r"(c)
      : "r"(lo), "r"(hi));
  return c;
}

// Eight values times `inv` = 2^-e as E4M3 codes.  `plain` (see plain_codes)
// values take the shorter way, others pass through fp32 with NaN replaced by 0
// (the conversion would keep it).
// fp16 stays fp16 on the shorter way: the product, at most 448, is exact where
// it is at least 2^-14, and below, where it may round, it stays below 2^-10,
// the tie between code 0 and E4M3's least value 2^-9.
template <bool BF16>
__device__ __forceinline__ uint2 codes8(uint4 v, float inv, bool plain) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if (!BF16 && plain) {
    const __half2 s = __float2half2_rn(inv);
    uint32_t x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __hmul2(*reinterpret_cast<const __half2*>(&w[i]), s);
      x[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint2(codes4(x[0], x[1]), codes4(x[2], x[3]));
  }
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 f = to_float2<BF16>(w[i]);
    f.x *= inv;
    f.y *= inv;
    if (!plain) {
      f.x = f.x == f.x ? f.x : 0.f;
      f.y = f.y == f.y ? f.y : 0.f;
    }
    c[i] = codes2(f);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// No NaN or infinity among the values; for fp16, 2^-e is a number of that type
// (a page's older rows can hold its exponent above fp16's own need of 8).
template <bool BF16>
__device__ __forceinline__ bool plain_codes(bool odd, int e) {
  return !odd && (BF16 || e <= 24);
}

// Eight E4M3 codes times `f` (a power of two <= 1), rounded again.
__device__ __forceinline__ uint2 rescale8(uint2 v, float f) {
  uint32_t w[4], c[4];
  e4m3x4_to_half2x2(v.x, w[0], w[1]);
  e4m3x4_to_half2x2(v.y, w[2], w[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    x.x *= f;
    x.y *= f;
    c[i] = codes2(x);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// True when token t leads a run: it has a slot, and the token before it is
// not the page's row before it.
__device__ __forceinline__ bool leads(const PagedStoreParams& p, int t, int slot, int prev) {
  return slot >= 0 && (t == 0 || prev != slot - 1 || (slot & ((1 << p.lg_ps) - 1)) == 0);
}

__device__ __forceinline__ const uint4* vec_ptr(const PagedStoreParams& p, int side, long long t,
                                                int h, int D, int vec) {
  return reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(side ? p.x[1] : p.x[0]) +
                                        t * (side ? p.stride[1] : p.stride[0]) + h * D) + vec;
}

// Vector `vec` of token t's key (side 0, turned by its angles when ROT) or value, 0
// for a lane that is not `live`; a row's vectors are in consecutive lanes.
template <int D, bool BF16, bool ROT>
__device__ __forceinline__ uint4 load_vec(const PagedStoreParams& p, int side, long long t, int h, int vec, int lane,
                                          bool live) {
  const uint4 v = live ? __ldg(vec_ptr(p, side, t, h, D, vec)) : make_uint4(0, 0, 0, 0);
  if constexpr (ROT) {
    const uint4 k = turn_chunk<BF16>(v, ChunkTurn(vec, lane, p.rot, p.interleaved),
                                     static_cast<const uint16_t*>(p.x[0]) + t * p.stride[0] + h * D, vec,
                                     p.angles + t * (p.rot >> 1), p.rot, p.interleaved, live && side == 0);
    if (side == 0) return k;
  }
  return v;
}

// ---- short runs: a warp stores a whole run of one head ------------------------
//
// Lanes [0, 16) serve K and [16, 32) V; a side's lanes hold a row as 16-byte
// vectors (D / 8 of them, 16 / (D / 8) rows at a time).  What does not depend on where
// the run ends is asked for first: one load gives its slot and the 31 behind it, and
// the scale is on its way before they are compared (1024 single tokens x 8 heads: 4.7
// -> 4.3 us, 5.0 -> 4.3 in pages of 16 x 64; the rows asked for as early: 10 % more for
// runs of five tokens).
template <int D, bool BF16, bool ROT>
__device__ __forceinline__ void store_run(const PagedStoreParams& p, int t, int h, int lane) {
  constexpr int VPR = D / 8, RPS = 16 / VPR;  // vectors of a row, rows a step
  const int left = p.n_tokens - t;
  const int mine = lane < left ? p.slots[t + lane] : -1;
  const int slot = __shfl_sync(0xffffffffu, mine, 0);
  const int page = slot >> p.lg_ps, row0 = slot & ((1 << p.lg_ps) - 1);
  if (page >= p.n_pages) {
    if (lane == 0) set_err(p.err, KVQ_PAGED_ERR_BAD_PAGE);
    return;
  }
  const int side = lane >> 4, l = lane & 15, sub = l / VPR, vec = l % VPR;
  float* scale = (side ? p.scale[1] : p.scale[0]) + static_cast<size_t>(page) * p.H + h;
  const float was = *scale;
  // rows of the run: until the page ends or the slots stop following (the first 32 are
  // at hand)
  const int most = min((1 << p.lg_ps) - row0, left);
  const uint32_t ends = __ballot_sync(0xffffffffu, lane >= most || mine != slot + lane);
  int n = ends ? __ffs(ends) - 1 : 32;
  while (!ends && n < most) {
    const int i = n + lane;
    const bool ok = i < most && p.slots[t + i] == slot + i;
    const uint32_t m = __ballot_sync(0xffffffffu, !ok);
    if (m) {
      n += __ffs(m) - 1;
      break;
    }
    n += 32;
  }
  auto load = [&](int i, bool live) { return load_vec<D, BF16, ROT>(p, side, t + i, h, vec, lane, live); };
  // a lane's rows begin at `sub`; lanes that turn keys make their rounds together
  const int lo = ROT ? 0 : sub, up = sub - lo;
  const uint4 first = load(sub, sub < n);
  uint32_t m2 = vec_max(first, 0);
  for (int i = lo + RPS; i < n; i += RPS) m2 = vec_max(load(i + up, i + up < n), m2);
  auto side_max = [](uint32_t x) {  // over the side's sixteen lanes
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
  };
  uint32_t mag = side_max(fold2(m2));
  const bool odd = mag >= inf_bits<BF16>();  // the side holds a NaN or an infinity
  if (__any_sync(0xffffffffu, odd)) {
    m2 = 0;
    for (int i = lo; i < n; i += RPS) m2 = vec_max_finite<BF16>(load(i + up, i + up < n), m2);
    mag = side_max(fold2(m2));
    if (odd && l == 0) set_err(p.err, KVQ_PAGED_ERR_NONFINITE);
  }
  int e = exp_for_bits<BF16>(mag);
  uint8_t* base = (side ? p.pages[1] : p.pages[0]) + ((static_cast<size_t>(page) * p.H + h) << p.lg_ps) * D + vec * 8;
  if (row0 > 0) {
    const int eo = exp_of_scale(was);
    e = max(e, eo);
    const float now = exp2i(e);
    if (was != now && was > 0.f) {
      const float f = was / now;
      for (int i = sub; i < row0; i += RPS) {
        uint2* c = reinterpret_cast<uint2*>(base + static_cast<size_t>(i) * D);
        *c = rescale8(*c, f);
      }
    }
  }
  const float inv = exp2i(-e);
  const bool plain = plain_codes<BF16>(odd, e);
  if (sub < n) *reinterpret_cast<uint2*>(base + static_cast<size_t>(row0 + sub) * D) = codes8<BF16>(first, inv, plain);
  for (int i = lo + RPS; i < n; i += RPS) {
    const uint2 c = codes8<BF16>(load(i + up, i + up < n), inv, plain);
    if (i + up < n) *reinterpret_cast<uint2*>(base + static_cast<size_t>(row0 + i + up) * D) = c;
  }
  if (l == 0) *scale = exp2i(e);
}

// ---- the kernel: a CTA looks at a chunk of tokens and one head ----------------
//
// It lists the chunk's leaders.  Where runs are short (more than an eighth of
// the tokens lead), each warp stores whole runs.  Where they are long, a team
// of TEAM = page_size * D / 32 threads stores a run: four 16-byte vectors of
// either side a thread cover a whole page, stay in registers between the maximum
// and the codes, and are all on their way at once; a CTA holds as many teams
// as fit 256 threads (512 for the largest page).
//
// Measured with either way alone (8 heads of 128, pages of 64, us): 256 single
// tokens 2.4 by warps and 12 by teams, 2048 single tokens 8.7 and 88; four
// prompts of 256 tokens 19 and 4.1, of 1024 tokens 18 and 4.3.
//
// A call of up to kShortChunks tokens x heads takes chunks of 8 tokens, so that
// its runs spread over the SMs; a larger one takes chunks of as many rows as its
// teams hold.  Measured (8 heads, short / whole chunks, us of a graph's call):
//   tokens x heads                       2048       4096       8192      16384
//   single tokens, 64 x 128          2.4/ 8.0   2.7/ 7.9   4.3/ 8.0   7.5/ 8.7
//   single tokens, 16 x 64           2.4/15.1   2.8/15.3   4.4/15.4   7.7/15.7
//   runs of 5, 64 x 128              3.2/ 4.3   4.0/ 4.4   6.0/ 4.5   9.2/ 5.5
//   runs of 5, 16 x 64               2.8/ 6.9   2.8/ 7.0   4.7/ 7.1   7.1/ 7.2
//   one prompt, 64 x 128             3.0/ 2.7   3.6/ 2.8   4.2/ 2.7   5.5/ 3.3
//   one prompt, 16 x 64              2.7/ 2.7   2.7/ 2.8   3.4/ 2.7   4.9/ 2.9
// The host does not know the runs: the turn lies where prompts lose by short
// chunks what single tokens gain.
//
// With keys that turn (ROT) the partner of a channel comes from the lane that
// holds it, and the angles from memory, 32 bytes a vector.  Measured (26298 tokens
// x 8 heads x 128, bf16, halves / interleaved): 27.6 us without turning, 44 / 41
// with it (120 channels of 128 turned, one by one: 63).  Warps that held one side each
// took 53 / 48: those of the values waited for those of the keys.  What is left of the
// difference are the angles' loads, one step after the other.  With 32 query heads in
// the same launch, their CTAs evenly among these, 106 / 111 us (floor 87) with three
// CTAs an SM (80 registers); with four (64) 43 / 39 and, with the queries, 114 / 103,
// with two (128) 54 / 50 and 129 / 139.
//
// One launch for a step's keys, values and queries saves single tokens a launch and
// gains little or loses on prompts, whose query CTAs have this kernel's registers.  Both
// sides (us in a graph; the append with its queries / alone, plus kvq_rotate alone):
//   64 tokens, 8 + 32 heads of 128                  halves   2.7/  4.9   interleaved   2.7/  4.4
//   256 tokens, 8 + 32 heads of 128                          3.9/  5.4                 3.1/  5.1
//   4861 tokens, 32 + 32 heads of 64, 16 turned             22.9/ 21.3                20.8/ 17.9
//   16000 tokens, 8 + 32 heads of 64                        33.1/ 32.5                34.6/ 30.6
//   16000 tokens, 8 + 32 heads of 128, 64 turned            66.1/ 66.0                64.0/ 63.6
//   26298 tokens, 8 + 32 heads of 128                      105.9/110.6               110.9/106.7
// A caller who has such prompts may call kvq_rotate for the queries: the bits are equal.
template <int TEAM>
__host__ __device__ constexpr int chunk_threads() {
  return TEAM == 512 ? 512 : 256;
}
constexpr int kSteps = 4;
constexpr int kShortChunks = 8192;

template <int D, bool BF16, bool ROT, int TEAM>
__global__ void __launch_bounds__(chunk_threads<TEAM>(), (ROT ? 768 : 1024) / chunk_threads<TEAM>())
    paged_store_kernel(const PagedStoreParams p) {
  constexpr int THREADS = chunk_threads<TEAM>(), TEAMS = THREADS / TEAM, WARPS = TEAM / 32;
  constexpr int VPR = D / 8, RPS = TEAM / VPR, CHUNK = RPS * kSteps * TEAMS;  // the most
  __shared__ int s_list[CHUNK];
  __shared__ int s_count;
  __shared__ uint32_t s_max[TEAMS][2][2][WARPS];  // [team][pass][side][warp]
  const int tid = threadIdx.x, lane = tid & 31;
  const int team = tid / TEAM, l = tid % TEAM;
  const int sub = l / VPR, vec = l % VPR;
  const int tb = blockIdx.x * p.chunk;
  int h = blockIdx.y;
  const int ps = 1 << p.lg_ps;
  if (tid == 0) s_count = 0;
  grid_dep_wait();
  grid_dep_launch();
  if constexpr (ROT) {
    // rows of CTAs for the heads lie evenly among those for the step's queries, so
    // that the ones' arithmetic runs beside the others' traffic
    h = blockIdx.y * p.H / gridDim.y;
    if (gridDim.y > p.H && (blockIdx.y + 1) * p.H / gridDim.y == h) {
      const long long t0 = (static_cast<long long>(blockIdx.y - h) * gridDim.x + blockIdx.x) * p.q.tokens;
      if (t0 < p.q.n_tokens) rotate_any<BF16, THREADS>(p.q, t0, tid);
      return;
    }
  }
  __syncthreads();
  if (tid < p.chunk) {
    const int t = tb + tid;
    if (t < p.n_tokens && leads(p, t, p.slots[t], t > 0 ? p.slots[t - 1] : -1))
      s_list[atomicAdd(&s_count, 1)] = t;
  }
  __syncthreads();
  const int count = s_count;
  if (count * 8 > p.chunk) {
    for (int i = tid >> 5; i < count; i += THREADS / 32) store_run<D, BF16, ROT>(p, s_list[i], h, lane);
    return;
  }
  auto team_sync = [&]() {
    if constexpr (WARPS > 1) asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(TEAM) : "memory");
    else __syncwarp();
  };
  // The largest values of either side over the team.
  auto team_max = [&](int pass, uint32_t (&x)[2]) {
#pragma unroll
    for (int side = 0; side < 2; ++side) x[side] = __reduce_max_sync(~0u, x[side]);
    if constexpr (WARPS > 1) {
      if (lane == 0) {
        s_max[team][pass][0][l >> 5] = x[0];
        s_max[team][pass][1][l >> 5] = x[1];
      }
      team_sync();
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        x[0] = max(x[0], s_max[team][pass][0][w]);
        x[1] = max(x[1], s_max[team][pass][1][w]);
      }
    }
  };
  for (int i_run = team; i_run < count; i_run += TEAMS) {
    const int t = s_list[i_run];
    const int slot = p.slots[t];
    const int page = slot >> p.lg_ps, row0 = slot & (ps - 1);
    if (page >= p.n_pages) {
      if (l == 0) set_err(p.err, KVQ_PAGED_ERR_BAD_PAGE);
      continue;
    }
    // rows that follow the leader: token t + i in row row0 + i of the page
    const int most = min(ps - row0, p.n_tokens - t);
    uint4 x[2][kSteps];
    uint32_t rows = 0;  // bit s: this thread holds vectors of step s
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int i = s * RPS + sub;
      if (i < most && (i == 0 || p.slots[t + i] == slot + i)) rows |= 1u << s;
    }
#pragma unroll
    for (int side = 0; side < 2; ++side) {
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        x[side][s] = make_uint4(0, 0, 0, 0);
        if ((rows >> s) & 1) x[side][s] = __ldg(vec_ptr(p, side, t + s * RPS + sub, h, D, vec));
      }
    }
    float was[2] = {0.f, 0.f};
    const size_t head = static_cast<size_t>(page) * p.H + h;
    if (row0 > 0) {
      was[0] = p.scale[0][head];
      was[1] = p.scale[1][head];
    }
    if constexpr (ROT) {
      const ChunkTurn ct(vec, lane, p.rot, p.interleaved);
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const long long tok = t + s * RPS + sub;
        x[0][s] = turn_chunk<BF16>(x[0][s], ct, static_cast<const uint16_t*>(p.x[0]) + tok * p.stride[0] + h * D, vec,
                                   p.angles + tok * (p.rot >> 1), p.rot, p.interleaved, (rows >> s) & 1);
      }
    }
    uint32_t mag[2];
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      uint32_t m2 = 0;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) m2 = vec_max(x[side][s], m2);
      mag[side] = fold2(m2);
    }
    team_max(0, mag);
    // a side holds a NaN or an infinity
    const bool odd[2] = {mag[0] >= inf_bits<BF16>(), mag[1] >= inf_bits<BF16>()};
    if (odd[0] || odd[1]) {
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        uint32_t m2 = 0;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) m2 = vec_max_finite<BF16>(x[side][s], m2);
        mag[side] = fold2(m2);
      }
      team_max(1, mag);
      if (l == 0) set_err(p.err, KVQ_PAGED_ERR_NONFINITE);
    }
    int e[2];
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      e[side] = exp_for_bits<BF16>(mag[side]);
      uint8_t* base = (side ? p.pages[1] : p.pages[0]) + (head << p.lg_ps) * D + vec * 8;
      if (row0 > 0) {
        e[side] = max(e[side], exp_of_scale(was[side]));
        const float now = exp2i(e[side]);
        if (was[side] != now && was[side] > 0.f) {
          const float f = was[side] / now;
          for (int i = sub; i < row0; i += RPS) {
            uint2* c = reinterpret_cast<uint2*>(base + static_cast<size_t>(i) * D);
            *c = rescale8(*c, f);
          }
        }
      }
      const float inv = exp2i(-e[side]);
      if (plain_codes<BF16>(odd[side], e[side])) {
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          if ((rows >> s) & 1)
            *reinterpret_cast<uint2*>(base + static_cast<size_t>(row0 + s * RPS + sub) * D) =
                codes8<BF16>(x[side][s], inv, true);
        }
      } else {
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          if ((rows >> s) & 1)
            *reinterpret_cast<uint2*>(base + static_cast<size_t>(row0 + s * RPS + sub) * D) =
                codes8<BF16>(x[side][s], inv, false);
        }
      }
    }
    team_sync();  // s_max and `was` are read
    if (l < 2) (l ? p.scale[1] : p.scale[0])[head] = exp2i(l ? e[1] : e[0]);
  }
}

template <int D, bool BF16, bool ROT, int TEAM>
cudaError_t launch_team(PagedStoreParams p, cudaStream_t st) {
  constexpr int THREADS = chunk_threads<TEAM>();
  const int most = kSteps * TEAM * 8 / D * (THREADS / TEAM);
  p.chunk = static_cast<long long>(p.n_tokens) * p.H <= kShortChunks ? 8 : most;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.n_tokens + p.chunk - 1) / p.chunk, p.H);
  if (ROT && p.q.n_heads > 0) {
    const long long ctas = rotate_ctas(&p.q, THREADS);
    cfg.gridDim.y += static_cast<unsigned>((ctas + cfg.gridDim.x - 1) / cfg.gridDim.x);
  }
  cfg.blockDim = dim3(THREADS);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_store_kernel<D, BF16, ROT, TEAM>, p);
}

template <int D, bool BF16, bool ROT>
cudaError_t launch(const PagedStoreParams& p, cudaStream_t st) {
  switch ((D << p.lg_ps) / (8 * kSteps)) {
    case 32:
      if constexpr (D == 64) return launch_team<D, BF16, ROT, 32>(p, st);
      break;
    case 64: return launch_team<D, BF16, ROT, 64>(p, st);
    case 128: return launch_team<D, BF16, ROT, 128>(p, st);
    case 256: return launch_team<D, BF16, ROT, 256>(p, st);
    case 512:
      if constexpr (D == 128) return launch_team<D, BF16, ROT, 512>(p, st);
      break;
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_paged_store(const PagedStoreParams& p, int D, int dtype, cudaStream_t st) {
  const bool bf = dtype == KVQ_DTYPE_BF16;
  const bool rot = p.rot > 0;
  if (D == 128) {
    if (rot) return bf ? launch<128, true, true>(p, st) : launch<128, false, true>(p, st);
    return bf ? launch<128, true, false>(p, st) : launch<128, false, false>(p, st);
  }
  if (D == 64) {
    if (rot) return bf ? launch<64, true, true>(p, st) : launch<64, false, true>(p, st);
    return bf ? launch<64, true, false>(p, st) : launch<64, false, false>(p, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace kvq
