// kvq_rotary.cu — rotary positions: frequencies (host), a step's angles, and
// heads turned by them (include/kvq.h).
//
//   a' = a cos - b sin,  b' = b cos + a sin,  angle = position * f_i
//
// Cosines and sines are computed once a step and not once a head or layer: 64
// pairs are 512 bytes a token, 1/24 of what its 8 + 8 + 32 heads of 128 read, and
// fifty instructions a pair would come to each of those heads.
// Bound: HBM for prompts, a launch for decodes.  Measured: 16003 tokens x 40
// heads of 128 (half of each turned, interleaved, 328 MB) 49.4 us, 98 % of the
// measured copy rate; 26298 tokens x 32 heads (halves, 443 MB) 66 us, 99 %; 64
// tokens x 32 heads 2.1 us in a graph.  Pairs that do not lie in aligned chunks are
// turned channel by channel, two bytes a load: 16003 tokens x 40 heads of 96, 24 of
// them turned, 188 us (32 of them, aligned halves, 41); 26298 x 32 heads of 128, 120
// turned, 211; 64 tokens x 32 heads 4.7.
#include <algorithm>
#include <cmath>

#include "kvq_rotary.cuh"

namespace kvq {
void count_launches(uint64_t n);

namespace {

constexpr int kThreads = 256;

// ---- angles ---------------------------------------------------------------------
//
// position * turn modulo 2^64 is the exact part of a turn; the nearest quarter
// comes off the top of its upper 32 bits, the rest (at most an eighth of a turn)
// becomes an angle within pi / 4, whose Taylor series to x^9 and x^10 leave 2^-29
// and 2^-33.
__device__ __forceinline__ float2 unit_of(int pos, uint2 turn) {  // turn: low, high word
  const uint32_t n = static_cast<uint32_t>(pos);
  uint32_t phase = __umulhi(n, turn.x) + n * turn.y;
  if (pos < 0) phase -= turn.x;  // n is 2^32 above the position
  const uint32_t quarter = (phase + (1u << 29)) >> 30;
  // what the quarter leaves, as a signed fraction of it
  const float x = static_cast<float>(static_cast<int32_t>(phase << 2)) * 3.65729521e-10f;  // 2 pi / 2^34
  const float y = x * x;
  const float s = fmaf(fmaf(fmaf(fmaf(2.7557319e-6f, y, -1.9841270e-4f), y, 8.3333333e-3f), y, -0.16666667f) * y, x, x);
  const float c = fmaf(fmaf(fmaf(fmaf(fmaf(-2.7557319e-7f, y, 2.4801587e-5f), y, -1.3888889e-3f), y, 4.1666667e-2f), y,
                            -0.5f), y, 1.0f);
  const float a = quarter & 1 ? s : c, b = quarter & 1 ? c : s;
  return make_float2(quarter == 1 || quarter == 2 ? -a : a, quarter & 2 ? -b : b);
}

// Bound: 131072 positions of 64 pairs write 67 MB (10 us) and take fifty
// instructions a pair, 10 us at full issue (71 % of the slots are used, by 3.4 rounds of
// CTAs); 14.7 us, 69 % of the measured copy rate (16.3 with the
// phase as one 64-bit product, 38.6 with a pair a thread and its place by 64-bit
// division).  64 positions: 1.3 us in a graph.
//
// A thread takes V neighbouring pairs of a token and every gridDim.x * rows-th
// token, so that the frequencies are read once.
template <int V>
__global__ void __launch_bounds__(kThreads) rotary_angles_kernel(const AnglesParams p) {
  const uint32_t row = threadIdx.x / p.lanes, k = (threadIdx.x - row * p.lanes.d) * V;
  const uint32_t rows = kThreads / p.lanes;
  grid_dep_wait();
  grid_dep_launch();
  if (row >= rows) return;
  uint2 turn[V];
#pragma unroll
  for (int i = 0; i < V; ++i) turn[i] = reinterpret_cast<const uint2*>(p.turns)[k + i];
  const long long step = static_cast<long long>(gridDim.x) * rows;
#pragma unroll 4
  for (long long t = static_cast<long long>(blockIdx.x) * rows + row; t < p.n_tokens; t += step) {
    const int pos = p.positions[t];
    float2 u[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      u[i] = unit_of(pos, turn[i]);
      u[i].x *= p.magnitude;
      u[i].y *= p.magnitude;
    }
    float2* out = p.angles + t * p.half + k;
    if constexpr (V == 2) *reinterpret_cast<float4*>(out) = make_float4(u[0].x, u[0].y, u[1].x, u[1].y);
    else *out = u[0];
  }
}

// ---- rotate ---------------------------------------------------------------------

template <bool BF16, RotateKind KIND>
__global__ void __launch_bounds__(kThreads) rotate_kernel(const RotateParams p) {
  grid_dep_wait();
  grid_dep_launch();
  rotate_tokens<BF16, KIND, kThreads>(p, static_cast<long long>(blockIdx.x) * p.tokens, threadIdx.x);
}

template <typename P>
cudaError_t launch(void (*fn)(P), const P& p, long long ctas, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, p);
}

template <bool BF16>
cudaError_t launch_kind(RotateParams p, cudaStream_t st) {
  const long long ctas = rotate_ctas(&p, kThreads);
  switch (rotate_kind(p.rot, p.interleaved)) {
    case kInterleaved: return launch(rotate_kernel<BF16, kInterleaved>, p, ctas, st);
    case kHalves: return launch(rotate_kernel<BF16, kHalves>, p, ctas, st);
    default: return launch(rotate_kernel<BF16, kSingle>, p, ctas, st);
  }
}

bool dev_ptr(const void* p, uintptr_t a) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace

kvq_status check_rotary(const kvq_rotary* r, int head_dim, int n_tokens) {
  if (r == nullptr || r->rotary_dim < 2 || r->rotary_dim % 2 != 0 || r->rotary_dim > head_dim ||
      (r->interleaved != 0 && r->interleaved != 1))
    return KVQ_ERR_INVALID_ARG;
  return n_tokens == 0 || dev_ptr(r->angles, 16) ? KVQ_OK : KVQ_ERR_INVALID_ARG;
}

kvq_status rotate_params(RotateParams* p, const kvq_rotary* rotary, const void* x, int dtype, long long x_stride,
                         void* out, long long out_stride, int n_tokens, int n_heads, int head_dim) {
  if (head_dim < 1 || (dtype != KVQ_DTYPE_FP16 && dtype != KVQ_DTYPE_BF16)) return KVQ_ERR_INVALID_ARG;
  const kvq_status s = check_rotary(rotary, head_dim, n_tokens);
  if (s != KVQ_OK) return s;
  if (head_dim % 8 != 0 || head_dim > 256) return KVQ_ERR_UNSUPPORTED;
  const long long least = static_cast<long long>(n_heads) * head_dim;
  if (n_tokens > 0 && (!dev_ptr(x, 16) || !dev_ptr(out, 16) || x_stride < least || out_stride < least ||
                       x_stride % 8 != 0 || out_stride % 8 != 0 || (x == out && x_stride != out_stride)))
    return KVQ_ERR_INVALID_ARG;
  p->x = static_cast<const uint16_t*>(x);
  p->out = static_cast<uint16_t*>(out);
  p->x_stride = x_stride;
  p->out_stride = out_stride;
  p->angles = reinterpret_cast<const float2*>(rotary->angles);
  p->n_tokens = n_tokens;
  p->n_heads = n_heads;
  p->D = head_dim;
  p->rot = rotary->rotary_dim;
  p->interleaved = rotary->interleaved;
  p->units.d = rotate_units(head_dim, rotary->rotary_dim, rotary->interleaved);
  if (static_cast<long long>(n_heads) * head_dim > 1 << 28) return KVQ_ERR_UNSUPPORTED;  // 32-bit places in a token
  return KVQ_OK;
}

cudaError_t launch_rotary_angles(AnglesParams p, cudaStream_t st) {
  const int v = p.half % 2 == 0 ? 2 : 1, lanes = p.half / v;  // (at most 128 pairs: 256 threads hold a token)
  p.lanes = divisor(lanes, kThreads + 1);
  const int rows = kThreads / lanes;
  const long long ctas = angles_ctas(p.n_tokens, rows);
  return v == 2 ? launch(rotary_angles_kernel<2>, p, ctas, st) : launch(rotary_angles_kernel<1>, p, ctas, st);
}

cudaError_t launch_rotate(const RotateParams& p, int dtype, cudaStream_t st) {
  return dtype == KVQ_DTYPE_BF16 ? launch_kind<true>(p, st) : launch_kind<false>(p, st);
}

}  // namespace kvq

using namespace kvq;

extern "C" {

kvq_status kvq_rotary_turns(int64_t* turns, int rotary_dim, double base, double factor,
                            double original_len, double low, double high) {
  if (turns == nullptr || rotary_dim < 2 || rotary_dim % 2 != 0 || !std::isfinite(base) || base <= 1.0 ||
      !std::isfinite(factor) || factor < 1.0 || !std::isfinite(original_len) || original_len < 0.0)
    return KVQ_ERR_INVALID_ARG;
  if (original_len > 0.0 && (!std::isfinite(low) || !std::isfinite(high) || low < 0.0 || high <= low))
    return KVQ_ERR_INVALID_ARG;
  if (rotary_dim > 256) return KVQ_ERR_UNSUPPORTED;
  constexpr double two_pi = 6.283185307179586476925;
  for (int i = 0; i < rotary_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rotary_dim);
    double keep = 0.0;
    if (original_len > 0.0) keep = std::min(1.0, std::max(0.0, (original_len * f / two_pi - low) / (high - low)));
    f = f * keep + f / factor * (1.0 - keep);
    turns[i] = static_cast<int64_t>(std::llrint(f / two_pi * 0x1p64));  // f <= 1: below 2^62
  }
  return KVQ_OK;
}

kvq_status kvq_rotary_angles(const int* positions, int n_tokens, const int64_t* turns,
                             int rotary_dim, float magnitude, float* angles, void* stream) {
  if (n_tokens < 0 || rotary_dim < 2 || rotary_dim % 2 != 0 || !std::isfinite(magnitude)) return KVQ_ERR_INVALID_ARG;
  if (rotary_dim > 256) return KVQ_ERR_UNSUPPORTED;
  if (n_tokens == 0) return KVQ_OK;
  if (!dev_ptr(positions, 4) || !dev_ptr(turns, 8) || !dev_ptr(angles, 16)) return KVQ_ERR_INVALID_ARG;
  AnglesParams p;
  p.positions = positions;
  p.turns = turns;
  p.angles = reinterpret_cast<float2*>(angles);
  p.n_tokens = n_tokens;
  p.half = rotary_dim / 2;
  p.magnitude = magnitude;
  if (launch_rotary_angles(p, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
    cudaGetLastError();
    return KVQ_ERR_CUDA;
  }
  count_launches(1);
  return KVQ_OK;
}

kvq_status kvq_rotate(const kvq_rotary* rotary, const void* x, int dtype, long long x_stride,
                      void* out, long long out_stride, int n_tokens, int n_heads, int head_dim,
                      void* stream) {
  if (n_tokens < 0 || n_heads < 1) return KVQ_ERR_INVALID_ARG;
  RotateParams p;
  const kvq_status s = rotate_params(&p, rotary, x, dtype, x_stride, out, out_stride, n_tokens, n_heads, head_dim);
  if (s != KVQ_OK || n_tokens == 0) return s;
  if (launch_rotate(p, dtype, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
    cudaGetLastError();
    return KVQ_ERR_CUDA;
  }
  count_launches(1);
  return KVQ_OK;
}

}  // extern "C"
