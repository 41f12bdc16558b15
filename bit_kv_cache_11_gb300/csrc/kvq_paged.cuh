// kvq_paged.cuh — launch parameter blocks and device helpers of the paged
// 8-bit cache (include/kvq.h, "Paged 8-bit cache").  Internal to csrc/.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvq.h"
#include "kvq_device.cuh"

namespace kvq {

// Exponents of the smallest and the largest page scale.  2^-15 times E4M3's
// smallest step 2^-9 is fp16's smallest number, so fp16 inputs lose nothing
// to the floor; the ceiling keeps every weight p * scale of the attention
// inside fp32 (include/kvq.h).
constexpr int kPagedMinExp = -15;
constexpr int kPagedMaxExp = 40;

struct PagedPlanParams {
  const int* ctx_len;
  const int* new_len;
  int batch;
  int* table;
  int max_pages;
  const int* free_pages;
  int free_cap;
  const int* n_free;
  int lg_ps;
  int n_tokens;
  int* cu_new;
  int* seq_len;
  int* slots;
  int* positions;  // may be null
  int* n_left;
  int* err;
};

// Most tokens of a store into E4M3 pages: its CTAs look at up to 512 tokens from a
// 32-bit one on.
constexpr int kPagedMaxStore = 0x7fffffff - 512;

// Attention over the pages.  Work is a flat sequence of units: request b's
// query rows (row r = new token r / R, query head r % R of the kv head's
// group) form groups of RG rows, and item (b, kv head, group) owns nu_b
// units of UT consecutive tokens.  Warps take equal contiguous unit ranges.
struct PagedAttnParams {
  const void* q;
  void* out;
  long long q_stride, out_stride;
  const int* table;
  int max_pages;
  const int* cu_new;
  const int* seq_len;
  int batch, n_tokens, max_new;
  int H, R, lg_ps, n_pages, box_rows;
  uint32_t r_magic;  // ceil(2^32 / R): row / R by one high product (R > 1)
  const float* k_scale;
  const float* v_scale;
  const uint32_t* meta[2];  // the 4-bit pages' metadata, whose calls have no scales
  float qscale;  // softmax scale * log2(e)
  int window;    // 0: none
  // rows (new tokens * R) of the requests this launch serves: those with
  // row_min <= rows <= row_max
  int row_min, row_max;
  int n_warps;
  int* tickets;   // [CTAs], zero between launches
  float* warp_part;  // [n_warps][RG * (D + 2)]
  float* cta_part;   // [2 * CTAs][RG * (D + 2)]
  uint32_t wait_limit;  // try_wait rounds of a main-loop wait, when below the kernel's own limit
  int* err;
};

__device__ __forceinline__ void set_err(int* err, int bit) {
  if (err != nullptr) atomicOr(err, bit);
}

__device__ __forceinline__ void grid_dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dep_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Four E4M3 codes -> exact fp16 pairs: bytes 0 and 1, bytes 2 and 3.
__device__ __forceinline__ void e4m3x4_to_half2x2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
        "l"(reinterpret_cast<unsigned long long&>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return d;
}

// Tiled copy of one box of a 2-D tensor map into shared memory.
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int x, int y,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4}], [%2];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(x), "r"(y)
      : "memory");
}

// Brings a tensor map of the kernel's parameters into the descriptor cache.
__device__ __forceinline__ void tensormap_prefetch(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// row / R for row < 2^28: row * ceil(2^32 / R) overshoots row / R * 2^32 by less
// than row * (R - 1) / R < 2^32 / R.
__device__ __forceinline__ int row_token(const PagedAttnParams& p, int row) {
  return p.R == 1 ? row : static_cast<int>(__umulhi(static_cast<uint32_t>(row), p.r_magic));
}

// Sum of two counts, at most 2^31 - 1.  Offsets that decrease let requests share
// rows, and their counts' sum pass any bound on the call's rows.
constexpr int kCountMax = 0x7fffffff;
__device__ __forceinline__ int add_counts(int a, int b) {
  return static_cast<int>(min(static_cast<uint32_t>(a) + static_cast<uint32_t>(b),
                              static_cast<uint32_t>(kCountMax)));
}

// Lengths of request b as the attention uses them: new tokens, first new
// token's row of q, all tokens.  Values that break the contract of
// include/kvq.h serve nothing (n = 0) and set the error word.
struct PagedReq {
  int n, q0, seq;
};

__device__ __forceinline__ PagedReq paged_req(const PagedAttnParams& p, int b, int* bad) {
  PagedReq r;
  const int c0 = p.cu_new[b], c1 = p.cu_new[b + 1];
  r.seq = p.seq_len[b];
  r.q0 = c0;
  r.n = c1 - c0;
  *bad = 0;
  if (c0 < 0 || c1 < c0 || c1 > p.n_tokens || r.n > p.max_new || r.seq < 0 ||
      r.seq > (static_cast<long long>(p.max_pages) << p.lg_ps)) {
    *bad = 1;
    r.n = 0;
    r.seq = 0;
  }
  return r;
}

// First token any row of the request may see.
__device__ __forceinline__ int first_seen(const PagedAttnParams& p, const PagedReq& r) {
  if (p.window == 0) return 0;
  const int lo = r.seq - r.n + 1 - p.window;
  return lo > 0 ? lo : 0;
}

cudaError_t launch_paged_plan(const PagedPlanParams& p, cudaStream_t st);
cudaError_t paged_decode_d64(const PagedAttnParams& p, const CUtensorMap& km, const CUtensorMap& vm,
                             bool bf16, int nt, cudaStream_t st);
cudaError_t paged_decode_d128(const PagedAttnParams& p, const CUtensorMap& km,
                              const CUtensorMap& vm, bool bf16, int nt, cudaStream_t st);
cudaError_t launch_paged_prompt(const PagedAttnParams& a, int items_max, const CUtensorMap& km,
                                const CUtensorMap& vm, int D, bool bf16, cudaStream_t st);
// The same over 4-bit pages.
cudaError_t paged4_decode_d64(const PagedAttnParams& p, const CUtensorMap& km, const CUtensorMap& vm,
                              bool bf16, int nt, cudaStream_t st);
cudaError_t paged4_decode_d128(const PagedAttnParams& p, const CUtensorMap& km,
                               const CUtensorMap& vm, bool bf16, int nt, cudaStream_t st);
cudaError_t launch_paged4_prompt(const PagedAttnParams& a, int items_max, const CUtensorMap& km,
                                 const CUtensorMap& vm, int D, bool bf16, cudaStream_t st);
// Lets kernel `fn` use `bytes` of dynamic shared memory on the current device
// (set once per kernel and device).
cudaError_t allow_smem(const void* fn, int bytes);
// Warps per CTA of the decode kernel, its most CTAs (one per SM of a GB300) and
// the tokens of a unit.
// (4-bit stages are smaller, and their arithmetic wants more warps)
constexpr int paged_warps(int nt, bool four) { return four && nt == 1 ? 12 : 8; }
constexpr int kPagedMaxCtas = 152;
// A request with at most this many query rows per kv head (new tokens * R) is
// served by the decode kernel, which splits its tokens over all SMs and reads
// them once per 16 rows; one with more rows by the prompt kernel, which reads
// them once per 256 rows but gives each of the call's batch * H (request,
// head) items at most one SM.  Measured (us, decode / prompt kernel; R = 4):
//   8 items of 32768 tokens, D = 128: 32 rows 43 / 409, 128 rows 110 / 410
//                            D = 64:  32 rows 31 / 348, 128 rows 69 / 349
//   128 items of 4000 tokens, D = 128: 32 rows 67 / 64, 64 rows 116 / 65
//                             D = 64:  32 rows 45 / 53, 64 rows 74 / 53
//   512 items of 1000 tokens, D = 128: 64 rows 116 / 85; D = 64: 74 / 71
// so the turn lies near 32 rows (48 of the narrower ones) where the items fill
// the SMs, and moves up in proportion where they do not.  Over 4-bit pages:
//   8 items of 32768 tokens, D = 128: 32 rows 49 / 430, 128 rows 130 / 430
//                            D = 64:  32 rows 34 / 373, 128 rows 75 / 373
//   128 items of 4000 tokens, D = 128: 16 rows 46 / 64, 32 rows 75 / 65, 48 rows 102 / 65
//                             D = 64:  32 rows 47 / 56, 48 rows 60 / 56, 64 rows 76 / 56
//   512 items of 1000 tokens, D = 128: 32 rows 78 / 83, 48 rows 110 / 84
//                             D = 64:  32 rows 57 / 69, 48 rows 73 / 70, 64 rows 93 / 69
// which turns at nearly the same rows: near 26 of 128 channels where the items fill
// the SMs, so that 27 to 33 rows of such a batch take up to 15 % longer than by the
// prompt kernel, while 512 items of 1000 tokens still gain at 32.
constexpr int decode_rows(long long items, int D) {
  const int full = D == 64 ? 48 : 32;
  return items >= 133 ? full : static_cast<int>(full * 133 / items);
}
constexpr int paged_unit_tokens(int D) { return 4096 / D; }
// Requests a call may have: the prefix sums of the batch live in shared memory.
constexpr int kPagedMaxBatch = 4096;

}  // namespace kvq
