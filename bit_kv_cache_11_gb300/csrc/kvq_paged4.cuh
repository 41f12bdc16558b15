// kvq_paged4.cuh — the paged 4-bit cache (include/kvq.h, "Paged 4-bit cache"):
// launch parameter blocks and the codes' arithmetic.  Internal to csrc/.
#pragma once

#include "kvq_rotary.cuh"

namespace kvq {

constexpr int kGroup4 = 32;            // channels of a group
constexpr float kMost4 = 65408.f;      // largest magnitude that is stored

struct Paged4StoreParams {
  uint8_t* codes[2];  // K, V: [n_pages][H][ps][D / 2]
  uint32_t* meta[2];  // [n_pages][H][ps][D / 32] {step, minimum} fp16 pairs
  const void* x[2];   // k, v: token t, head h at t * stride + h * D
  long long stride[2];
  const int* slots;
  int n_tokens;
  int n_pages, H, lg_ps;
  int* err;
  const float2* angles;  // keys turn when rot > 0
  int rot, interleaved;
  RotateParams q;        // the step's queries; n_heads 0: none
};

struct Paged4ReadParams {
  const uint8_t* codes[2];
  const uint32_t* meta[2];
  uint16_t* out[2];  // fp16 [n_tokens][H][D]; may be null
  const int* slots;
  int n_tokens;
  int n_pages, H, lg_ps;
  int* err;
};

// CTAs of `threads` for `per` threads' work a token of both sides: `rounds` of it
// each, fewer while that leaves SMs idle.
struct Grid4 {
  int tokens;   // of a CTA
  Divisor per;  // threads of a token and side
  unsigned kv_ctas;
};
inline Grid4 grid4(int n_tokens, long long per, int rounds, int threads) {
  const long long all = per * n_tokens;
  const long long want = std::min<long long>(static_cast<long long>(rounds) * threads, std::max<long long>(threads, all / (152 * 4)));
  Grid4 g = {};
  g.tokens = static_cast<int>(std::max<long long>(1, std::min<long long>(want / per, n_tokens)));
  g.per = divisor(static_cast<uint32_t>(per / 2), per * g.tokens);
  g.kv_ctas = static_cast<unsigned>(ctas_of(n_tokens, g.tokens));
  return g;
}

__device__ __forceinline__ uint32_t pair_lo(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x5410); }
__device__ __forceinline__ uint32_t pair_hi(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7632); }
__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }
__device__ __forceinline__ uint32_t as_word(__half2 x) { return *reinterpret_cast<const uint32_t*>(&x); }

// (x & mask) | bits in one operation.
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(y) : "r"(x), "r"(mask), "r"(bits));
  return y;
}

// The four code pairs of a word, (bits 4j .., bits 4j + 16 ..), j = 0 .. 3, as values
// code * step + least, rounded once.  A code in the mantissa of 1024 is 1024 + code,
// four bits higher 1024 + 16 code: one operation on the pair gives the code
// itself, exactly.
__device__ __forceinline__ void values4(uint32_t w, uint32_t step, uint32_t least, uint32_t (&v)[4]) {
  const __half2 minus = __float2half2_rn(-1024.f), sixteenth = __float2half2_rn(0.0625f), less = __float2half2_rn(-64.f);
#pragma unroll
  for (int j = 0; j < 4; j += 2, w >>= 8) {
    const uint32_t lo = and_or(w, 0x000f000fu, 0x64006400u), hi = and_or(w, 0x00f000f0u, 0x64006400u);
    v[j] = as_word(__hfma2(__hadd2(as_half2(lo), minus), as_half2(step), as_half2(least)));
    v[j + 1] = as_word(__hfma2(__hfma2(as_half2(hi), sixteenth, less), as_half2(step), as_half2(least)));
  }
}

cudaError_t launch_paged4_append(const Paged4StoreParams& p, int D, int dtype, cudaStream_t st);
cudaError_t launch_paged4_read(const Paged4ReadParams& p, int D, cudaStream_t st);

}  // namespace kvq
