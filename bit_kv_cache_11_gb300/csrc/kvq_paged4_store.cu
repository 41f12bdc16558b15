// kvq_paged4_store.cu — new keys and values into the 4-bit pages, the keys (and
// the step's queries) turned on the way (kvq_paged4_append), and tokens read
// back (kvq_paged4_read).
//
// Per token, kv head and group of 32 channels, x fp16 within +-65408:
//   step = fp16((mx - mn) / 15),  code = rint((x - mn) / step) in [0, 15]
// A thread holds 16 channels, half a group: its neighbour's minimum and maximum
// complete the statistics, its codes are one 8-byte store.
//
// The divide is three packed operations on two quotients, exact for steps of 11
// bits, and the rounding one more; ties need no branch, which values of few bits
// would take often.
//
// Bound: arithmetic, about 300 instructions a thread (73 % of the issue slots; the
// L1 takes 73 % of its time with keys turned).  Measured (us; 26298 tokens x 8 heads
// x 128, bf16: 142 MB, floor 20.8): 35 without turning, 48 with halves, 42 with
// interleaved pairs, 27 to read back (78 % of the measured copy rate); 64 tokens 1.9
// and 2.5.  Partners by shuffles and half of the angles a lane 49; places worked out
// once a thread 55, the next item's loads ahead no better (both cost registers, 48 ->
// 64 and more, and with them threads); shuffles by the masks of the pairs, not of the
// warp, 2 us more.
#include <algorithm>

#include "kvq_paged4.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 256;

// A pair of 16-bit values as an fp16 pair within +-kMost4, NaN as 0.
template <bool BF16>
__device__ __forceinline__ uint32_t as_fp16(uint32_t w) {
  float2 f = pair_to_float2<BF16>(w);
  f.x = f.x == f.x ? fminf(fmaxf(f.x, -kMost4), kMost4) : 0.f;
  f.y = f.y == f.y ? fminf(fmaxf(f.y, -kMost4), kMost4) : 0.f;
  return as_word(__floats2half2_rn(f.x, f.y));
}

// range / 15 correctly rounded: with y = 1 / 15 rounded, q + (range - 15 q) y is
// (Markstein's theorem; range is 0 or at least 2^-24, so nothing underflows).
__device__ __forceinline__ float fifteenth(float range) {
  constexpr float y = 1.f / 15.f;
  const float q = range * y;
  return fmaf(fmaf(-15.f, q, range), y, q);
}
__device__ __forceinline__ float about_inverse(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float2 twice(float x) { return make_float2(x, x); }

// Smallest and largest of eight pairs; NaN where one of them is.
template <bool BF16>
__device__ __forceinline__ float2 bounds(const uint32_t (&w)[8]) {
  if constexpr (BF16) {
    auto b2 = [](uint32_t x) { return *reinterpret_cast<const __nv_bfloat162*>(&x); };
    __nv_bfloat162 lo = b2(w[0]), hi = lo;
#pragma unroll
    for (int j = 1; j < 8; ++j) {
      lo = __hmin2_nan(lo, b2(w[j]));
      hi = __hmax2_nan(hi, b2(w[j]));
    }
    return make_float2(__bfloat162float(__hmin_nan(__low2bfloat16(lo), __high2bfloat16(lo))),
                       __bfloat162float(__hmax_nan(__low2bfloat16(hi), __high2bfloat16(hi))));
  } else {
    __half2 lo = as_half2(w[0]), hi = lo;
#pragma unroll
    for (int j = 1; j < 8; ++j) {
      lo = __hmin2_nan(lo, as_half2(w[j]));
      hi = __hmax2_nan(hi, as_half2(w[j]));
    }
    return make_float2(__half2float(__hmin_nan(__low2half(lo), __high2half(lo))),
                       __half2float(__hmax_nan(__low2half(hi), __high2half(hi))));
  }
}

// Step and minimum of a group, of which the lane holds the 16 channels w (turned to
// fp16 here) and its neighbour the others; by whole warps.  *odd: one of the 16 is
// infinite or NaN.
template <bool BF16>
__device__ __forceinline__ __half2 group_of(uint32_t (&w)[8], bool* odd) {
  float2 b = bounds<BF16>(w);
  *odd = false;
  if (!(b.x >= -kMost4 && b.y <= kMost4)) {  // beyond the bounds, infinite or NaN
    *odd = !isfinite(b.x) || !isfinite(b.y);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = as_fp16<BF16>(w[j]);
    b = bounds<false>(w);
  } else if constexpr (BF16) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 f = pair_to_float2<true>(w[j]);
      w[j] = as_word(__floats2half2_rn(f.x, f.y));
    }
    // (rounding keeps the order)
    b = make_float2(__half2float(__float2half_rn(b.x)), __half2float(__float2half_rn(b.y)));
  }
  // (a minimum or a range of -0 is stored as 0)
  const float mn = fminf(b.x, __shfl_xor_sync(~0u, b.x, 1)) + 0.f;
  const float range = fmaxf(b.y, __shfl_xor_sync(~0u, b.y, 1)) - mn + 0.f;
  return __floats2half2_rn(fifteenth(range), mn);
}

// The two words of codes of 16 channels.
template <bool KEY>
__device__ __forceinline__ uint2 codes16(const uint32_t (&w)[8], __half2 meta) {
  const float step = __low2float(meta), mn = __high2float(meta);
  // The divide, correctly rounded: with an approximate reciprocal (2^-22), q + (d -
  // q step) inv errs by less than 2^-18 of its last place (the remainder is exact),
  // and a quotient by a step of 11 bits is no nearer than 2^-12 to the middle
  // between two fp32 numbers.  Then rint by the fp32 numbers around 1.5 * 2^23,
  // whose last bit is 1 and whose bits are this one's plus the code.  (A step that
  // is no normal fp16 number may be far too small: codes end at 15.)
  constexpr float kRint = 12582912.f;
  constexpr uint32_t kBits = 0x4b400000u, kAll = 0x11111111u;
  const float inv = step > 0.f ? about_inverse(step) : 0.f;
  uint32_t o[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint32_t word = 0u - kBits * kAll;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 d = add2(__half22float2(as_half2(w[4 * c + j])), twice(-mn));
      float2 q = fma2(d, twice(inv), twice(0.f));
      q = fma2(fma2(q, twice(-step), d), twice(inv), q);
      const float2 r = add2(q, twice(kRint));
      word += __float_as_uint(fminf(r.x, kRint + 15.f)) << (KEY ? 4 * j : 8 * j);
      word += __float_as_uint(fminf(r.y, kRint + 15.f)) << (KEY ? 4 * j + 16 : 8 * j + 4);
    }
    o[c] = word;
  }
  return make_uint2(o[0], o[1]);
}

// Channels c .. c + 7 of a key at `head`, in `own`, after the turn by angles a.
template <bool BF16>
__device__ __forceinline__ uint4 turned(uint4 own, const uint16_t* head, int c, const float2* a, int rot, int interleaved) {
  if (c >= rot) return own;
  const int half = rot >> 1;
  if (!rotate_aligned(rot, interleaved)) return turn_single<BF16>(own, head, c, a, rot, interleaved);
  if (interleaved) return turn_interleaved<BF16>(own, a + (c >> 1));
  const int oc = c < half ? c + half : c - half;
  const float sign = c < oc ? -1.f : 1.f;
  const uint4 other = __ldg(reinterpret_cast<const uint4*>(head + oc));
  a += min(c, oc);
  return make_uint4(turn_own<BF16>(own.x, other.x, angles2(a), sign), turn_own<BF16>(own.y, other.y, angles2(a + 2), sign),
                    turn_own<BF16>(own.z, other.z, angles2(a + 4), sign), turn_own<BF16>(own.w, other.w, angles2(a + 6), sign));
}

// Tokens [t0, t0 + g.tokens): a thread takes 16 channels, half a group.
template <int D, bool BF16>
__device__ __forceinline__ void append_tokens(const Paged4StoreParams& p, const Grid4& g, long long t0, int tid) {
  constexpr int TPR = D / 16;  // threads of a row
  const int n = static_cast<int>(min(static_cast<long long>(g.tokens), p.n_tokens - t0));
  const uint32_t total = static_cast<uint32_t>(n) * 2 * g.per.d;
  for (uint32_t i0 = tid; (i0 & ~31u) < total; i0 += kThreads) {
    const uint32_t i = min(i0, total - 1);  // (whole warps shuffle)
    const uint32_t st = i / g.per, r = i - st * g.per.d, t = st >> 1, side = st & 1;
    const uint32_t h = r / TPR, c = 16 * (r - h * TPR);
    const uint16_t* head = static_cast<const uint16_t*>(side ? p.x[1] : p.x[0]) +
                           (t0 + t) * (side ? p.stride[1] : p.stride[0]) + h * D;
    const int slot = p.slots[t0 + t];
    uint4 v[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) v[j] = __ldg(reinterpret_cast<const uint4*>(head + c + 8 * j));
    if (side == 0 && p.rot > 0) {
      const float2* a = p.angles + (t0 + t) * (p.rot >> 1);
#pragma unroll
      for (int j = 0; j < 2; ++j) v[j] = turned<BF16>(v[j], head, c + 8 * j, a, p.rot, p.interleaved);
    }
    uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
    bool odd;
    const __half2 meta = group_of<BF16>(w, &odd);
    const int page = slot >> p.lg_ps;
    if (slot < 0 || i0 >= total) continue;
    if (page >= p.n_pages) {
      if (r == 0) set_err(p.err, KVQ_PAGED_ERR_BAD_PAGE);
      continue;
    }
    const uint2 codes = side ? codes16<false>(w, meta) : codes16<true>(w, meta);
    if (odd) set_err(p.err, KVQ_PAGED_ERR_NONFINITE);
    const size_t at = (((static_cast<size_t>(page) * p.H + h) << p.lg_ps) + (slot & ((1 << p.lg_ps) - 1))) * (D / 2) + c / 2;
    *reinterpret_cast<uint2*>((side ? p.codes[1] : p.codes[0]) + at) = codes;
    if ((c & 16) == 0) (side ? p.meta[1] : p.meta[0])[at / 16] = as_word(meta);
  }
}

template <int D, bool BF16, RotateKind KIND>
__global__ void __launch_bounds__(kThreads) paged4_append_kernel(const Paged4StoreParams p, const Grid4 g) {
  grid_dep_wait();
  grid_dep_launch();
  // CTAs for keys and values lie evenly among those for the step's queries, so that
  // the ones' arithmetic runs beside the others' traffic.  Both sides (us in a graph;
  // with the queries / the append alone, plus kvq_rotate alone; halves, interleaved):
  //   64 tokens, 8 + 32 heads of 128                   2.4/  4.6    2.3/  4.0
  //   256 tokens, 8 + 32 heads of 128                  3.1/  4.7    2.6/  4.2
  //   4861 tokens, 32 + 32 heads of 64, 16 turned     25.0/ 22.5   18.7/ 19.2
  //   16000 tokens, 8 + 32 heads of 64                34.2/ 33.7   29.5/ 30.9
  //   16000 tokens, 8 + 32 heads of 128, 64 turned    69.9/ 67.2   54.9/ 64.2
  //   26298 tokens, 8 + 32 heads of 128              105.4/114.1   90.0/107.6
  const unsigned kv = static_cast<unsigned>(static_cast<unsigned long long>(blockIdx.x) * g.kv_ctas / gridDim.x);
  if ((static_cast<unsigned long long>(blockIdx.x) + 1) * g.kv_ctas / gridDim.x != kv) {
    append_tokens<D, BF16>(p, g, static_cast<long long>(kv) * g.tokens, threadIdx.x);
  } else {
    rotate_tokens<BF16, KIND, kThreads>(p.q, static_cast<long long>(blockIdx.x - kv) * p.q.tokens, threadIdx.x);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) paged4_read_kernel(const Paged4ReadParams p, const Grid4 g) {
  constexpr int VPR = D / 8, U = 4;
  grid_dep_wait();
  grid_dep_launch();
  const long long t0 = static_cast<long long>(blockIdx.x) * g.tokens;
  const int n = static_cast<int>(min(static_cast<long long>(g.tokens), p.n_tokens - t0));
  const uint32_t total = static_cast<uint32_t>(n) * 2 * g.per.d;
  for (uint32_t i0 = threadIdx.x; i0 < total; i0 += U * kThreads) {
    uint32_t word[U], meta[U];
    uint4* out[U];
    bool key[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const uint32_t i = i0 + k * kThreads;
      out[k] = nullptr;
      word[k] = meta[k] = 0;
      if (i >= total) continue;
      const uint32_t st = i / g.per, r = i - st * g.per.d, t = st >> 1, side = st & 1;
      uint16_t* to = side ? p.out[1] : p.out[0];
      if (to == nullptr) continue;
      const uint32_t h = r / VPR, vec = r - h * VPR;
      out[k] = reinterpret_cast<uint4*>(to + ((t0 + t) * p.H + h) * D) + vec;
      key[k] = side == 0;
      const int slot = p.slots[t0 + t];
      const int page = slot >> p.lg_ps;
      if (slot < 0) continue;
      if (page >= p.n_pages) {
        if (r == 0) set_err(p.err, KVQ_PAGED_ERR_BAD_PAGE);
        continue;
      }
      const size_t at = ((static_cast<size_t>(page) * p.H + h) << p.lg_ps) + (slot & ((1 << p.lg_ps) - 1));
      word[k] = __ldg(reinterpret_cast<const uint32_t*>((side ? p.codes[1] : p.codes[0]) + at * (D / 2)) + vec);
      meta[k] = __ldg((side ? p.meta[1] : p.meta[0]) + at * (D / kGroup4) + (vec >> 2));
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (out[k] == nullptr) continue;
      uint32_t o[4];
      values4(word[k], pair_lo(meta[k], meta[k]), pair_hi(meta[k], meta[k]), o);
      // a key's pairs are neighbours, a value's are channels j and j + 4
      *out[k] = key[k] ? make_uint4(o[0], o[1], o[2], o[3])
                       : make_uint4(pair_lo(o[0], o[1]), pair_lo(o[2], o[3]), pair_hi(o[0], o[1]), pair_hi(o[2], o[3]));
    }
  }
}

template <typename... K, typename... A>
cudaError_t launch(void (*fn)(K...), long long ctas, cudaStream_t st, A... args) {
  if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, args...);
}

template <int D, bool BF16>
cudaError_t append(Paged4StoreParams p, cudaStream_t st) {
  const Grid4 g = grid4(p.n_tokens, 2LL * p.H * (D / 16), 2, kThreads);
  const long long ctas = static_cast<long long>(g.kv_ctas) + (p.q.n_heads ? rotate_ctas(&p.q, kThreads) : 0);
  switch (p.q.n_heads ? rotate_kind(p.q.rot, p.q.interleaved) : kInterleaved) {
    case kInterleaved: return launch(paged4_append_kernel<D, BF16, kInterleaved>, ctas, st, p, g);
    case kHalves: return launch(paged4_append_kernel<D, BF16, kHalves>, ctas, st, p, g);
    default: return launch(paged4_append_kernel<D, BF16, kSingle>, ctas, st, p, g);
  }
}

}  // namespace

cudaError_t launch_paged4_append(const Paged4StoreParams& p, int D, int dtype, cudaStream_t st) {
  const bool bf = dtype == KVQ_DTYPE_BF16;
  if (D == 128) return bf ? append<128, true>(p, st) : append<128, false>(p, st);
  return bf ? append<64, true>(p, st) : append<64, false>(p, st);
}

cudaError_t launch_paged4_read(const Paged4ReadParams& p, int D, cudaStream_t st) {
  const Grid4 g = grid4(p.n_tokens, 2LL * p.H * (D / 8), 16, kThreads);
  return D == 128 ? launch(paged4_read_kernel<128>, g.kv_ctas, st, p, g)
                  : launch(paged4_read_kernel<64>, g.kv_ctas, st, p, g);
}

}  // namespace kvq
