// kvq_paged4_attention.cu — attention over the 4-bit pages, the plain way: a CTA
// takes one query row, its warps take tokens in turn, and their running maxima,
// sums and outputs are joined at the end.
#include "kvq_paged4.cuh"

namespace kvq {
namespace {

constexpr int kWarps = 4;

template <int D, bool BF16>
__global__ void __launch_bounds__(kWarps * 32) paged4_attention_kernel(const PagedAttnParams p) {
  constexpr int CH = D / 32;  // channels of a lane
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][D];
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x, hq = blockIdx.y, h = hq / p.R;
  // the request of the row
  int b = -1;
  PagedReq r = {};
  for (int i = 0; i < p.batch; ++i) {
    int bad;
    const PagedReq x = paged_req(p, i, &bad);
    if (bad && row == 0 && hq == 0 && threadIdx.x == 0) set_err(p.err, KVQ_PAGED_ERR_LENGTH);
    if (x.n > 0 && row >= x.q0 && row < x.q0 + x.n) {
      b = i;
      r = x;
    }
  }
  if (b < 0) return;
  const int pos = r.seq - r.n + row - r.q0;
  const int first = p.window ? max(0, pos - p.window + 1) : 0;
  const uint16_t* q = static_cast<const uint16_t*>(p.q) + row * p.q_stride + static_cast<long long>(hq) * D;
  // lane's channels: two bytes of codes; in keys the four even (or odd) channels of a word
  float x[CH];
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    const int n = lane * CH + j, c = n / 8 * 8 + n % 4 * 2 + n % 8 / 4;
    x[j] = one_to_float<BF16>(q[c]) * p.qscale;
  }
  float m = -INFINITY, l = 0.f, o[CH] = {};
  for (int t = first + warp; t <= pos; t += kWarps) {
    const int page = p.table[static_cast<size_t>(b) * p.max_pages + (t >> p.lg_ps)];
    if (page < 0 || page >= p.n_pages) {
      if (lane == 0) set_err(p.err, KVQ_PAGED_ERR_BAD_PAGE);
      continue;
    }
    const size_t at = ((static_cast<size_t>(page) * p.H + h) << p.lg_ps) + (t & ((1 << p.lg_ps) - 1));
    float side[2][CH];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint32_t meta = p.meta[s][at * (D / kGroup4) + lane * CH / kGroup4];
      const __half2 sm = *reinterpret_cast<const __half2*>(&meta);
      uint32_t w = CH == 4 ? *reinterpret_cast<const uint16_t*>(p.codes[s] + at * (D / 2) + lane * 2)
                           : p.codes[s][at * (D / 2) + lane];
#pragma unroll
      for (int j = 0; j < CH; ++j, w >>= 4)
        side[s][j] = __half2float(__low2half(__hfma2(codes_to_half2(w), __low2half2(sm), __high2half2(sm))));
    }
    float z = 0.f;
#pragma unroll
    for (int j = 0; j < CH; ++j) z = fmaf(x[j], side[0][j], z);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
    const float mn = fmaxf(m, z), mb = mn == -INFINITY ? 0.f : mn;
    const float al = exp2f(m - mb), w = exp2f(z - mb);
    m = mn;
    l = fmaf(l, al, w);
#pragma unroll
    for (int j = 0; j < CH; ++j) o[j] = fmaf(o[j], al, w * side[1][j]);
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int j = 0; j < CH; ++j) s_o[warp][lane * CH + j] = o[j];
  __syncthreads();
  float M = -INFINITY;
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w]);
  const float mb = M == -INFINITY ? 0.f : M;
  float L = 0.f;
  for (int w = 0; w < kWarps; ++w) L += s_l[w] * exp2f(s_m[w] - mb);
  uint16_t* out = static_cast<uint16_t*>(p.out) + row * p.out_stride + static_cast<long long>(hq) * D;
  for (int c = threadIdx.x; c < D; c += kWarps * 32) {
    float v = 0.f;
    for (int w = 0; w < kWarps; ++w) v += s_o[w][c] * exp2f(s_m[w] - mb);
    out[c] = float_to_one<BF16>(L > 0.f ? v / L : L == 0.f ? 0.f : L);
  }
}

}  // namespace

cudaError_t launch_paged4_attention(const PagedAttnParams& p, int D, bool bf16, cudaStream_t st) {
  const dim3 grid(p.n_tokens, p.H * p.R), block(kWarps * 32);
  if (D == 128) {
    if (bf16) paged4_attention_kernel<128, true><<<grid, block, 0, st>>>(p);
    else paged4_attention_kernel<128, false><<<grid, block, 0, st>>>(p);
  } else {
    if (bf16) paged4_attention_kernel<64, true><<<grid, block, 0, st>>>(p);
    else paged4_attention_kernel<64, false><<<grid, block, 0, st>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace kvq
