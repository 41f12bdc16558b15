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

// Two codes in the low four bits of a word's halves as fp16.
__device__ __forceinline__ __half2 codes_to_half2(uint32_t w) {
  const uint32_t x = (w & 0x000f000fu) | 0x64006400u;  // 1024 + code
  return __hsub2(*reinterpret_cast<const __half2*>(&x), __float2half2_rn(1024.f));
}

cudaError_t launch_paged4_append(const Paged4StoreParams& p, int D, int dtype, cudaStream_t st);
cudaError_t launch_paged4_attention(const PagedAttnParams& p, int D, bool bf16, cudaStream_t st);
cudaError_t launch_paged4_read(const Paged4ReadParams& p, int D, cudaStream_t st);

}  // namespace kvq
