// kvq_paged4_store.cu — new keys and values into the 4-bit pages, the keys (and
// the step's queries) turned on the way (kvq_paged4_append), and tokens read
// back (kvq_paged4_read).
//
// Per token, kv head and group of 32 channels, x fp16 within +-65408:
//   step = fp16((mx - mn) / 15),  code = rint((x - mn) / step) in [0, 15]
// A thread holds eight channels, four threads a group.
#include <algorithm>

#include "kvq_paged4.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 256;

// A pair of 16-bit values as fp16 pair within +-kMost4, NaN as 0; *odd when one
// of them is infinite or NaN.
template <bool BF16>
__device__ __forceinline__ uint32_t as_fp16(uint32_t w, bool* odd) {
  float2 f = pair_to_float2<BF16>(w);
  *odd |= !isfinite(f.x) || !isfinite(f.y);
  f.x = f.x == f.x ? fminf(fmaxf(f.x, -kMost4), kMost4) : 0.f;
  f.y = f.y == f.y ? fminf(fmaxf(f.y, -kMost4), kMost4) : 0.f;
  const __half2 h = __floats2half2_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// rint(d / step) where the quotient is rounded to fp32 before.
__device__ __forceinline__ int code_of(float d, float step) {
  return step > 0.f ? min(max(__float2int_rn(__fdiv_rn(d, step)), 0), 15) : 0;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads) paged4_append_kernel(const Paged4StoreParams p, long long kv_items,
                                                                 long long items) {
  constexpr int VPR = D / 8;
  grid_dep_wait();
  grid_dep_launch();
  const long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= items) return;
  if (i >= kv_items) {
    const long long k = i - kv_items;
    const long long per = static_cast<long long>(p.q.n_heads) * p.q.units;
    const long long t = k / per;
    const int r = static_cast<int>(k - t * per), h = r / p.q.units;
    rotate_unit<BF16>(p.q, t, h, r - h * p.q.units);
    return;
  }
  // (kv_items is a multiple of 32: a warp is all here)
  const long long per = 2LL * p.H * VPR;
  const long long t = i / per;
  const bool real = t < p.n_tokens;
  const int r = static_cast<int>(i - t * per);
  const int side = r >= p.H * VPR, rh = r - side * p.H * VPR, h = rh / VPR, vec = rh - h * VPR;
  const int slot = real ? p.slots[t] : -1;
  const int page = slot >> p.lg_ps, row = slot & ((1 << p.lg_ps) - 1);
  const bool good = slot >= 0 && page < p.n_pages;
  if (slot >= 0 && !good && r == 0) set_err(p.err, KVQ_PAGED_ERR_BAD_PAGE);
  uint4 v = make_uint4(0, 0, 0, 0);
  if (good) {
    const uint16_t* head = static_cast<const uint16_t*>(side ? p.x[1] : p.x[0]) +
                           t * (side ? p.stride[1] : p.stride[0]) + h * D;
    v = __ldg(reinterpret_cast<const uint4*>(head) + vec);
    if (side == 0 && p.rot > 0)
      v = turned_chunk<BF16>(v, head, vec, p.angles + t * (p.rot >> 1), p.rot, p.interleaved);
  }
  bool odd = false;
  const uint32_t w[4] = {as_fp16<BF16>(v.x, &odd), as_fp16<BF16>(v.y, &odd), as_fp16<BF16>(v.z, &odd),
                         as_fp16<BF16>(v.w, &odd)};
  if (odd) set_err(p.err, KVQ_PAGED_ERR_NONFINITE);
  float x[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = pair_to_float2<false>(w[j]);
    x[2 * j] = f.x;
    x[2 * j + 1] = f.y;
  }
  float mn = x[0], mx = x[0];
#pragma unroll
  for (int j = 1; j < 8; ++j) {
    mn = fminf(mn, x[j]);
    mx = fmaxf(mx, x[j]);
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  if (!good) return;
  mn += 0.f;  // (a minimum or a range of -0 is stored as 0)
  const __half sh = __float2half_rn(__fdiv_rn(mx - mn + 0.f, 15.f));
  const float step = __half2float(sh);
  uint32_t word = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t c = code_of(x[j] - mn, step);
    word |= c << (side ? 4 * j : 4 * (j >> 1) + 16 * (j & 1));
  }
  const size_t at = (((static_cast<size_t>(page) * p.H + h) << p.lg_ps) + row);
  *reinterpret_cast<uint32_t*>((side ? p.codes[1] : p.codes[0]) + at * (D / 2) + vec * 4) = word;
  if ((vec & 3) == 0) {
    const __half2 m = __halves2half2(sh, __float2half_rn(mn));
    (side ? p.meta[1] : p.meta[0])[at * (D / kGroup4) + (vec >> 2)] = *reinterpret_cast<const uint32_t*>(&m);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) paged4_read_kernel(const Paged4ReadParams p, long long items) {
  constexpr int VPR = D / 8;
  grid_dep_wait();
  grid_dep_launch();
  const long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= items) return;
  const long long per = 2LL * p.H * VPR;
  const long long t = i / per;
  const int r = static_cast<int>(i - t * per);
  const int side = r >= p.H * VPR, rh = r - side * p.H * VPR, h = rh / VPR, vec = rh - h * VPR;
  uint16_t* out = side ? p.out[1] : p.out[0];
  if (out == nullptr) return;
  const int slot = p.slots[t];
  const int page = slot >> p.lg_ps, row = slot & ((1 << p.lg_ps) - 1);
  uint32_t o[4] = {0, 0, 0, 0};
  if (slot >= 0 && page >= p.n_pages) {
    if (r == 0 || (p.out[0] == nullptr && rh == 0)) set_err(p.err, KVQ_PAGED_ERR_BAD_PAGE);
  } else if (slot >= 0) {
    const size_t at = (((static_cast<size_t>(page) * p.H + h) << p.lg_ps) + row);
    const uint32_t word = *reinterpret_cast<const uint32_t*>((side ? p.codes[1] : p.codes[0]) + at * (D / 2) + vec * 4);
    const uint32_t m = (side ? p.meta[1] : p.meta[0])[at * (D / kGroup4) + (vec >> 2)];
    const __half2 sm = *reinterpret_cast<const __half2*>(&m);
    const __half2 s2 = __low2half2(sm), m2 = __high2half2(sm);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // codes of channels 2j, 2j + 1 in the halves' low bits
      const uint32_t w = side ? (word >> (8 * j) & 0xfu) | (word >> (8 * j + 4) & 0xfu) << 16 : word >> (4 * j);
      const __half2 x = __hfma2(codes_to_half2(w), s2, m2);
      o[j] = *reinterpret_cast<const uint32_t*>(&x);
    }
  }
  *(reinterpret_cast<uint4*>(out + (static_cast<size_t>(t) * p.H + h) * D) + vec) = make_uint4(o[0], o[1], o[2], o[3]);
}

template <typename... K, typename... A>
cudaError_t launch(void (*fn)(K...), long long items, cudaStream_t st, A... args) {
  if (items > static_cast<long long>(kThreads) * 0x7fffffff) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((items + kThreads - 1) / kThreads));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, args...);
}

}  // namespace

cudaError_t launch_paged4_append(const Paged4StoreParams& p, int D, int dtype, cudaStream_t st) {
  const long long kv = (static_cast<long long>(p.n_tokens) * 2 * p.H * (D / 8) + 31) / 32 * 32;
  const long long items = kv + static_cast<long long>(p.n_tokens) * p.q.n_heads * p.q.units;
  const bool bf = dtype == KVQ_DTYPE_BF16;
  if (D == 128)
    return bf ? launch(paged4_append_kernel<128, true>, items, st, p, kv, items)
              : launch(paged4_append_kernel<128, false>, items, st, p, kv, items);
  return bf ? launch(paged4_append_kernel<64, true>, items, st, p, kv, items)
            : launch(paged4_append_kernel<64, false>, items, st, p, kv, items);
}

cudaError_t launch_paged4_read(const Paged4ReadParams& p, int D, cudaStream_t st) {
  const long long items = static_cast<long long>(p.n_tokens) * 2 * p.H * (D / 8);
  return D == 128 ? launch(paged4_read_kernel<128>, items, st, p, items)
                  : launch(paged4_read_kernel<64>, items, st, p, items);
}

}  // namespace kvq
