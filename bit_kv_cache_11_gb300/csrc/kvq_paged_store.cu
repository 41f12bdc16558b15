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
// single tokens.  Measured: 26298 tokens x 8 heads x 128, 162 MB, 28.9 us (84 %
// of the measured copy rate); 4861 tokens x 32 heads x 64 in 16-row pages, 60 MB,
// 14.5 us (62 %; the launch and the last CTAs take the rest); 256 single tokens
// 2.5 us.  One test per side for NaN instead of two selects a value, and fp16
// codes without a step through fp32, took 31.0 -> 28.9 and 16.0 -> 14.5 us.
#include "kvq_paged.cuh"

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

// ---- short runs: a warp stores a whole run of one head ------------------------
//
// Lanes [0, 16) serve K and [16, 32) V; a side's lanes hold a row as 16-byte
// vectors (D / 8 of them, 16 / (D / 8) rows at a time).
template <int D, bool BF16>
__device__ __forceinline__ void store_run(const PagedStoreParams& p, int t, int h, int lane) {
  constexpr int VPR = D / 8, RPS = 16 / VPR;  // vectors of a row, rows a step
  const int slot = p.slots[t];
  const int page = slot >> p.lg_ps, row0 = slot & ((1 << p.lg_ps) - 1);
  if (page >= p.n_pages) {
    if (lane == 0) set_err(p.err, KVQ_PAGED_ERR_BAD_PAGE);
    return;
  }
  const int side = lane >> 4, l = lane & 15, sub = l / VPR, vec = l % VPR;
  // rows of the run: until the page ends or the slots stop following
  const int most = min((1 << p.lg_ps) - row0, p.n_tokens - t);
  int n = 1;
  while (n < most) {
    const int i = n + lane;
    const bool ok = i < most && p.slots[t + i] == slot + i;
    const uint32_t m = __ballot_sync(0xffffffffu, !ok);
    if (m) {
      n += __ffs(m) - 1;
      break;
    }
    n += 32;
  }
  float* scale = (side ? p.scale[1] : p.scale[0]) + static_cast<size_t>(page) * p.H + h;
  const float was = *scale;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const uint4 first = sub < n ? *vec_ptr(p, side, t + sub, h, D, vec) : zero;
  uint32_t m2 = vec_max(first, 0);
  for (int i = sub + RPS; i < n; i += RPS) m2 = vec_max(*vec_ptr(p, side, t + i, h, D, vec), m2);
  auto side_max = [](uint32_t x) {  // over the side's sixteen lanes
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
  };
  uint32_t mag = side_max(fold2(m2));
  const bool odd = mag >= inf_bits<BF16>();  // the side holds a NaN or an infinity
  if (__any_sync(0xffffffffu, odd)) {
    m2 = 0;
    for (int i = sub; i < n; i += RPS)
      m2 = vec_max_finite<BF16>(*vec_ptr(p, side, t + i, h, D, vec), m2);
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
  for (int i = sub + RPS; i < n; i += RPS)
    *reinterpret_cast<uint2*>(base + static_cast<size_t>(row0 + i) * D) =
        codes8<BF16>(*vec_ptr(p, side, t + i, h, D, vec), inv, plain);
  if (l == 0) *scale = exp2i(e);
}

// ---- the kernel: a CTA looks at a chunk of tokens and one head ----------------
//
// It lists the chunk's leaders.  Where runs are short (more than an eighth of
// the tokens lead), each warp stores whole runs.  Where they are long, a team
// of TEAM = page_size * D / 64 threads stores one side of a run: eight 16-byte
// vectors a thread cover a whole page, stay in registers between the maximum
// and the codes, and are all on their way at once; a CTA holds as many teams
// as fit 256 threads (512 for the largest page).
//
// Measured with either way alone (8 heads of 128, pages of 64, us): 256 single
// tokens 2.5 by warps and 75 by teams, 2048 single tokens 6.8 and 94; four
// prompts of 256 tokens 20 and 5.0, of 1024 tokens 29 and 7.6.
//
// A call of up to kShortChunks tokens x heads takes chunks of 8 tokens, so that
// its runs spread over the SMs; a larger one takes chunks of as many rows as its
// teams hold.  Measured (8 heads, short / whole chunks, us of a graph's call):
//   tokens x heads                       2048       4096       8192      16384
//   single tokens, 64 x 128          2.5/ 7.7   3.0/ 7.8   4.6/ 7.8   7.8/ 9.0
//   single tokens, 16 x 64           2.5/13.8   3.0/13.9   4.6/14.2   7.9/14.7
//   runs of 5, 64 x 128              3.2/ 4.5   3.9/ 4.6   6.0/ 4.6   9.5/ 5.4
//   runs of 5, 16 x 64               3.0/ 7.6   3.5/ 7.8   5.5/ 8.1   8.4/ 8.5
//   one prompt, 64 x 128             3.2/ 3.0   3.8/ 3.0   4.6/ 3.1   5.9/ 3.7
//   one prompt, 16 x 64              3.0/ 2.8   3.6/ 2.8   4.6/ 2.9   7.1/ 2.9
// The host does not know the runs: the turn lies where prompts lose by short
// chunks what single tokens gain.
template <int TEAM>
__host__ __device__ constexpr int chunk_threads() {
  return TEAM == 256 ? 512 : 256;
}
constexpr int kSteps = 8;
constexpr int kShortChunks = 8192;

template <int D, bool BF16, int TEAM>
__global__ void __launch_bounds__(chunk_threads<TEAM>(), 1024 / chunk_threads<TEAM>())
    paged_store_kernel(const PagedStoreParams p) {
  constexpr int THREADS = chunk_threads<TEAM>(), TEAMS = THREADS / (2 * TEAM);
  constexpr int VPR = D / 8, RPS = TEAM / VPR, CHUNK = TEAM * 64 / D * TEAMS;  // the most
  constexpr int WPT = TEAM > 32 ? TEAM / 32 : 1;  // warps of a team's side
  __shared__ int s_list[CHUNK];
  __shared__ int s_count;
  __shared__ uint32_t s_max[TEAMS][2][2][WPT];  // [team][pass][side][warp]
  const int tid = threadIdx.x, lane = tid & 31;
  const int side = tid / TEAM & 1, team = tid / (2 * TEAM), l = tid % TEAM;
  const int sub = l / VPR, vec = l % VPR;
  const int tb = blockIdx.x * p.chunk, h = blockIdx.y;
  const int ps = 1 << p.lg_ps;
  if (tid == 0) s_count = 0;
  grid_dep_wait();
  grid_dep_launch();
  __syncthreads();
  if (tid < p.chunk) {
    const int t = tb + tid;
    if (t < p.n_tokens && leads(p, t, p.slots[t], t > 0 ? p.slots[t - 1] : -1))
      s_list[atomicAdd(&s_count, 1)] = t;
  }
  __syncthreads();
  const int count = s_count;
  if (count * 8 > p.chunk) {
    for (int i = tid >> 5; i < count; i += THREADS / 32) store_run<D, BF16>(p, s_list[i], h, lane);
    return;
  }
  // Threads of a run's two sides wait for one another (whole warps when a
  // side is 16 or 32 threads).
  auto team_sync = [&]() {
    if constexpr (TEAM > 32)
      asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(2 * TEAM) : "memory");
    else __syncwarp();
  };
  // The side's largest value of x; *both: the larger one of the two sides.
  auto side_max = [&](int pass, uint32_t x, uint32_t* both) {
    if constexpr (TEAM > 32) {
      x = __reduce_max_sync(0xffffffffu, x);
      if (lane == 0) s_max[team][pass][side][l >> 5] = x;
      team_sync();
      uint32_t m[2] = {0, 0};
#pragma unroll
      for (int w = 0; w < WPT; ++w) {
        m[0] = max(m[0], s_max[team][pass][0][w]);
        m[1] = max(m[1], s_max[team][pass][1][w]);
      }
      *both = max(m[0], m[1]);
      return side ? m[1] : m[0];
    } else {
#pragma unroll
      for (int o = 1; o < TEAM; o <<= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
      *both = __reduce_max_sync(0xffffffffu, x);  // the warp's: it decides for its lanes
      return x;
    }
  };
  // (all lanes of a warp make the same number of rounds)
  const int rounds = TEAM >= 32 ? (count - team + TEAMS - 1) / TEAMS : (count + TEAMS - 1) / TEAMS;
  for (int k = 0; k < rounds; ++k) {
    const int i_run = k * TEAMS + team;
    const bool has = i_run < count;
    const int t = has ? s_list[i_run] : 0;
    const int slot = has ? p.slots[t] : 0;
    const int page = slot >> p.lg_ps, row0 = slot & (ps - 1);
    const bool good = has && page < p.n_pages;
    if (has && !good && l == 0 && side == 0) set_err(p.err, KVQ_PAGED_ERR_BAD_PAGE);
    // rows that follow the leader: token t + i in row row0 + i of the page
    const int most = good ? min(ps - row0, p.n_tokens - t) : 0;
    float* scale = (side ? p.scale[1] : p.scale[0]) + static_cast<size_t>(good ? page : 0) * p.H + h;
    uint4 x[kSteps];
    uint32_t rows = 0;  // bit s: this thread holds a vector of step s
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int i = s * RPS + sub;
      if (i < most && (i == 0 || p.slots[t + i] == slot + i)) rows |= 1u << s;
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      x[s] = make_uint4(0, 0, 0, 0);
      if ((rows >> s) & 1) x[s] = __ldg(vec_ptr(p, side, t + s * RPS + sub, h, D, vec));
    }
    const float was = good && row0 > 0 ? *scale : 0.f;
    uint32_t m2 = 0, both;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) m2 = vec_max(x[s], m2);
    uint32_t mag = side_max(0, fold2(m2), &both);
    const bool odd = mag >= inf_bits<BF16>();  // the side holds a NaN or an infinity
    if (both >= inf_bits<BF16>()) {
      m2 = 0;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) m2 = vec_max_finite<BF16>(x[s], m2);
      mag = side_max(1, fold2(m2), &both);
      if (odd && l == 0) set_err(p.err, KVQ_PAGED_ERR_NONFINITE);
    }
    int e = exp_for_bits<BF16>(mag);
    if (good) {
      uint8_t* base = (side ? p.pages[1] : p.pages[0]) +
                      ((static_cast<size_t>(page) * p.H + h) << p.lg_ps) * D + vec * 8;
      if (row0 > 0) {
        e = max(e, exp_of_scale(was));
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
      if (plain_codes<BF16>(odd, e)) {
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          if ((rows >> s) & 1)
            *reinterpret_cast<uint2*>(base + static_cast<size_t>(row0 + s * RPS + sub) * D) =
                codes8<BF16>(x[s], inv, true);
        }
      } else {
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          if ((rows >> s) & 1)
            *reinterpret_cast<uint2*>(base + static_cast<size_t>(row0 + s * RPS + sub) * D) =
                codes8<BF16>(x[s], inv, false);
        }
      }
    }
    team_sync();  // s_max and `was` are read
    if (good && l == 0) *scale = exp2i(e);
  }
}

template <int D, bool BF16, int TEAM>
cudaError_t launch_team(PagedStoreParams p, cudaStream_t st) {
  constexpr int THREADS = chunk_threads<TEAM>();
  const int most = TEAM * 64 / D * (THREADS / (2 * TEAM));
  p.chunk = static_cast<long long>(p.n_tokens) * p.H <= kShortChunks ? 8 : most;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.n_tokens + p.chunk - 1) / p.chunk, p.H);
  cfg.blockDim = dim3(THREADS);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_store_kernel<D, BF16, TEAM>, p);
}

template <int D, bool BF16>
cudaError_t launch(const PagedStoreParams& p, cudaStream_t st) {
  switch ((D << p.lg_ps) / 64) {
    case 16:
      if constexpr (D == 64) return launch_team<D, BF16, 16>(p, st);
      break;
    case 32: return launch_team<D, BF16, 32>(p, st);
    case 64: return launch_team<D, BF16, 64>(p, st);
    case 128: return launch_team<D, BF16, 128>(p, st);
    case 256:
      if constexpr (D == 128) return launch_team<D, BF16, 256>(p, st);
      break;
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_paged_store(const PagedStoreParams& p, int D, int dtype, cudaStream_t st) {
  const bool bf = dtype == KVQ_DTYPE_BF16;
  if (D == 128) return bf ? launch<128, true>(p, st) : launch<128, false>(p, st);
  if (D == 64) return bf ? launch<64, true>(p, st) : launch<64, false>(p, st);
  return cudaErrorInvalidValue;
}

}  // namespace kvq
