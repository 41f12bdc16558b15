// kvq_paged4_store.cu — new keys and values into the 4-bit pages, the keys (and
// the step's queries) turned on the way (kvq_paged4_append), and tokens read
// back (kvq_paged4_read).
//
// Per token, kv head and group of 32 channels, x fp16 within +-65408:
//   step = fp16((mx - mn) / 15),  code = rint((x - mn) / step) in [0, 15]
// A thread holds eight channels (a word of codes), four threads a group, and
// several words' loads are on their way at once.
#include <algorithm>

#include "kvq_paged4.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 256;
constexpr int kWords = 2;  // of a thread at a time

// A pair of 16-bit values as an fp16 pair within +-kMost4, NaN as 0.
template <bool BF16>
__device__ __forceinline__ uint32_t as_fp16(uint32_t w) {
  float2 f = pair_to_float2<BF16>(w);
  f.x = f.x == f.x ? fminf(fmaxf(f.x, -kMost4), kMost4) : 0.f;
  f.y = f.y == f.y ? fminf(fmaxf(f.y, -kMost4), kMost4) : 0.f;
  return as_word(__floats2half2_rn(f.x, f.y));
}

// rint(d / step) where the quotient is rounded to fp32 before.
__device__ __forceinline__ uint32_t code_of(float d, float step) {
  return step > 0.f ? min(max(__float2int_rn(__fdiv_rn(d, step)), 0), 15) : 0;
}

// The word of codes and the {step, minimum} pair of eight channels v, whose group
// is the four lanes of a quad.  *odd: a value is infinite or NaN.
template <bool BF16, bool KEY>
__device__ __forceinline__ uint32_t quantize8(uint4 v, uint32_t quad, uint32_t* meta, bool* odd) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
  // largest magnitudes: beyond kMost4 (bf16: its largest number below) the
  // values need a look each
  uint32_t m2 = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) m2 = __vmaxu2(m2, w[j] & 0x7fff7fffu);
  const uint32_t mag = max(m2 & 0xffffu, m2 >> 16);
  *odd = mag >= (BF16 ? 0x7f80u : 0x7c00u);
  if (mag > (BF16 ? 0x477fu : 0x7bfcu)) {
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = as_fp16<BF16>(w[j]);
  } else if constexpr (BF16) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = pair_to_float2<true>(w[j]);
      w[j] = as_word(__floats2half2_rn(f.x, f.y));
    }
  }
  const __half2 lo2 = __hmin2(__hmin2(as_half2(w[0]), as_half2(w[1])), __hmin2(as_half2(w[2]), as_half2(w[3])));
  const __half2 hi2 = __hmax2(__hmax2(as_half2(w[0]), as_half2(w[1])), __hmax2(as_half2(w[2]), as_half2(w[3])));
  // (minimum, -maximum) in one word for the quad
  __half2 both = __halves2half2(__hmin(__low2half(lo2), __high2half(lo2)), __hneg(__hmax(__low2half(hi2), __high2half(hi2))));
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) both = __hmin2(both, as_half2(__shfl_xor_sync(quad, as_word(both), o)));
  // (a minimum or a range of -0 is stored as 0)
  const float mn = __low2float(both) + 0.f, range = -__high2float(both) - mn + 0.f;
  const __half sh = __float2half_rn(__fdiv_rn(range, 15.f));
  const float step = __half2float(sh);
  *meta = as_word(__halves2half2(sh, __float2half_rn(mn)));
  // rint by the fp32 numbers around 1.5 * 2^23, whose last bit is 1; a quotient
  // near a tie (the reciprocal errs by 2^-18 of a step at most) is divided out.
  constexpr float kRint = 12582912.f;
  const float inv = step > 0.f ? __frcp_rn(step) : 0.f;
  float d[8], tie = 0.f;
  uint32_t word = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 f = __half22float2(as_half2(w[j >> 1]));
    d[j] = (j & 1 ? f.y : f.x) - mn;
    const float r = fmaf(d[j], inv, kRint);
    tie = fmaxf(tie, fabsf(fmaf(d[j], inv, kRint - r)));
    const uint32_t c = __float_as_uint(fminf(r, kRint + 15.f)) & 15u;
    word |= c << (KEY ? 4 * (j >> 1) + 16 * (j & 1) : 4 * j);
  }
  if (tie > 0.5f - 0x1p-16f) {
    word = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) word |= code_of(d[j], step) << (KEY ? 4 * (j >> 1) + 16 * (j & 1) : 4 * j);
  }
  return word;
}

struct Grid4 {
  int tokens;         // of a CTA
  Divisor per;  // words of a token and side
  unsigned kv_ctas;
};

template <int D, bool BF16>
__device__ __forceinline__ void append_tokens(const Paged4StoreParams& p, const Grid4& g, long long t0, int tid) {
  constexpr int VPR = D / 8;
  const int n = static_cast<int>(min(static_cast<long long>(g.tokens), p.n_tokens - t0));
  const uint32_t per = 2 * g.per.d, total = static_cast<uint32_t>(n) * per;
  const uint32_t quad = 0xfu << (tid & 28);
  for (uint32_t i0 = 0; i0 < total; i0 += kWords * kThreads) {
    uint4 v[kWords];
    size_t at[kWords];  // row of the pool
    int vec[kWords];
    bool good[kWords], key[kWords];
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
      const uint32_t i = i0 + k * kThreads + tid;
      good[k] = false;
      if (i >= total) continue;  // (whole quads)
      const uint32_t st = i / g.per, r = i - st * g.per.d, t = st >> 1, side = st & 1;
      const uint32_t h = r / VPR;
      vec[k] = r - h * VPR;
      key[k] = side == 0;
      const int slot = p.slots[t0 + t];
      const int page = slot >> p.lg_ps;
      good[k] = slot >= 0 && page < p.n_pages;
      if (slot >= 0 && !good[k] && r == 0) set_err(p.err, KVQ_PAGED_ERR_BAD_PAGE);
      if (!good[k]) continue;
      at[k] = ((static_cast<size_t>(page) * p.H + h) << p.lg_ps) + (slot & ((1 << p.lg_ps) - 1));
      const uint16_t* head = static_cast<const uint16_t*>(side ? p.x[1] : p.x[0]) +
                             (t0 + t) * (side ? p.stride[1] : p.stride[0]) + h * D;
      v[k] = __ldg(reinterpret_cast<const uint4*>(head) + vec[k]);
      if (key[k] && p.rot > 0)
        v[k] = turned_chunk<BF16>(v[k], head, vec[k], p.angles + (t0 + t) * (p.rot >> 1), p.rot, p.interleaved);
    }
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
      if (!good[k]) continue;
      bool odd;
      uint32_t meta;
      const uint32_t word = key[k] ? quantize8<BF16, true>(v[k], quad, &meta, &odd)
                                   : quantize8<BF16, false>(v[k], quad, &meta, &odd);
      if (odd) set_err(p.err, KVQ_PAGED_ERR_NONFINITE);
      const int side = key[k] ? 0 : 1;
      *reinterpret_cast<uint32_t*>(p.codes[side] + at[k] * (D / 2) + vec[k] * 4) = word;
      if ((vec[k] & 3) == 0) p.meta[side][at[k] * (D / kGroup4) + (vec[k] >> 2)] = meta;
    }
  }
}

template <int D, bool BF16, RotateKind KIND>
__global__ void __launch_bounds__(kThreads) paged4_append_kernel(const Paged4StoreParams p, const Grid4 g) {
  grid_dep_wait();
  grid_dep_launch();
  if (blockIdx.x < g.kv_ctas) {
    append_tokens<D, BF16>(p, g, static_cast<long long>(blockIdx.x) * g.tokens, threadIdx.x);
  } else {
    rotate_tokens<BF16, KIND, kThreads>(p.q, static_cast<long long>(blockIdx.x - g.kv_ctas) * p.q.tokens, threadIdx.x);
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

// CTAs that take the tokens' words: a few rounds each, fewer while that leaves
// SMs idle.
Grid4 grid_of(int n_tokens, int H, int D, int rounds) {
  const long long per = 2LL * H * (D / 8), all = per * n_tokens;
  const long long want = std::min<long long>(static_cast<long long>(rounds) * kThreads, std::max<long long>(kThreads, all / (152 * 4)));
  Grid4 g = {};
  g.tokens = static_cast<int>(std::max<long long>(1, std::min<long long>(want / per, n_tokens)));
  g.per = divisor(static_cast<uint32_t>(per / 2), per * g.tokens);
  g.kv_ctas = static_cast<unsigned>((n_tokens + g.tokens - 1) / g.tokens);
  return g;
}

template <int D, bool BF16>
cudaError_t append(Paged4StoreParams p, cudaStream_t st) {
  const Grid4 g = grid_of(p.n_tokens, p.H, D, 4 * kWords);
  const long long ctas = g.kv_ctas + (p.q.n_heads ? rotate_ctas(&p.q, kThreads) : 0);
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
  const Grid4 g = grid_of(p.n_tokens, p.H, D, 16);
  return D == 128 ? launch(paged4_read_kernel<128>, g.kv_ctas, st, p, g)
                  : launch(paged4_read_kernel<64>, g.kv_ctas, st, p, g);
}

}  // namespace kvq
