// kvq_rotary.cuh — turning heads by rotary angles (include/kvq.h, "Rotary
// positions"): the arithmetic that kvq_rotate and the paged appends share.
// Internal to csrc/.
#pragma once

#include <algorithm>

#include "kvq_paged.cuh"

namespace kvq {

// Quotients by one divisor: ceil(2^32 / d) overshoots n / d by less than n / 2^32,
// below 1 / d while n * d < 2^32 (m = 0 beyond, or for d = 1: a plain division).
struct Divisor {
  uint32_t d, m;
};
inline Divisor divisor(uint32_t d, unsigned long long most) {
  return {d, d > 1 && most * d < 1ull << 32 ? static_cast<uint32_t>(((1ull << 32) + d - 1) / d) : 0};
}
__device__ __forceinline__ uint32_t operator/(uint32_t n, const Divisor& v) {
  return v.m ? __umulhi(n, v.m) : n / v.d;
}

// x -> out, heads of D channels whose first `rot` turn by angles
// [token][rot / 2] (cos, sin).
struct RotateParams {
  const uint16_t* x;
  uint16_t* out;
  long long x_stride, out_stride;  // elements a token
  const float2* angles;
  int n_tokens, n_heads, D;
  int rot;          // even
  int interleaved;
  int tokens;       // of a CTA
  Divisor per, units;  // units of a token and of a head
};

// A unit of a head is what one thread turns: the channels of whole pairs, so
// that out may be x itself.  Where the layout's chunks of eight channels are
// aligned a unit is
//   kInterleaved  one chunk, its four pairs or (from rot on) its copy
//   kHalves       two chunks of eight pairs, or a chunk to copy
// and else (kSingle) four pairs of single channels, or eight channels to copy.
enum RotateKind { kInterleaved, kHalves, kSingle };
inline __host__ __device__ bool rotate_aligned(int rot, int interleaved) {
  return rot % (interleaved ? 8 : 16) == 0;
}
inline RotateKind rotate_kind(int rot, int interleaved) {
  return !rotate_aligned(rot, interleaved) ? kSingle : interleaved ? kInterleaved : kHalves;
}
inline int rotate_units(int D, int rot, int interleaved) {
  if (!rotate_aligned(rot, interleaved)) return (rot / 2 + 3) / 4 + (D - rot + 7) / 8;
  return interleaved ? D / 8 : rot / 16 + (D - rot) / 8;
}

template <bool BF16>
__device__ __forceinline__ float2 pair_to_float2(uint32_t w) {
  if constexpr (BF16) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  } else {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
}
template <bool BF16>
__device__ __forceinline__ uint32_t float2_to_pair(float lo, float hi) {
  if constexpr (BF16) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
  } else {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
template <bool BF16>
__device__ __forceinline__ float one_to_float(uint16_t x) {
  if constexpr (BF16) return __uint_as_float(static_cast<uint32_t>(x) << 16);
  else return __half2float(__ushort_as_half(x));
}
template <bool BF16>
__device__ __forceinline__ uint16_t float_to_one(float x) {
  if constexpr (BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(x));
  else return __half_as_ushort(__float2half_rn(x));
}

// The pair (a, b) turned by (cos, sin): every operation rounded by itself, as
// the header says, so that all callers give the same bits.
__device__ __forceinline__ float turn_a(float a, float b, float2 cs) {
  return __fsub_rn(__fmul_rn(a, cs.x), __fmul_rn(b, cs.y));
}
__device__ __forceinline__ float turn_b(float a, float b, float2 cs) {
  return __fadd_rn(__fmul_rn(b, cs.x), __fmul_rn(a, cs.y));
}

// Two consecutive angles (16-byte aligned when the first is even).
__device__ __forceinline__ float4 angles2(const float2* a) {
  return __ldg(reinterpret_cast<const float4*>(a));
}

// A word of two interleaved channels turned by (cos, sin).
template <bool BF16>
__device__ __forceinline__ uint32_t turn_word(uint32_t w, float2 cs) {
  const float2 x = pair_to_float2<BF16>(w);
  return float2_to_pair<BF16>(turn_a(x.x, x.y, cs), turn_b(x.x, x.y, cs));
}

// Eight interleaved channels by their four angles.
template <bool BF16>
__device__ __forceinline__ uint4 turn_interleaved(uint4 v, const float2* a) {
  const float4 p = angles2(a), q = angles2(a + 2);
  return make_uint4(turn_word<BF16>(v.x, make_float2(p.x, p.y)), turn_word<BF16>(v.y, make_float2(p.z, p.w)),
                    turn_word<BF16>(v.z, make_float2(q.x, q.y)), turn_word<BF16>(v.w, make_float2(q.z, q.w)));
}

// Words of two channels of the first half (va) and of the second (vb).
template <bool BF16>
__device__ __forceinline__ void turn_words(uint32_t& va, uint32_t& vb, float4 cs) {
  const float2 a = pair_to_float2<BF16>(va), b = pair_to_float2<BF16>(vb);
  const float2 c0 = make_float2(cs.x, cs.y), c1 = make_float2(cs.z, cs.w);
  va = float2_to_pair<BF16>(turn_a(a.x, b.x, c0), turn_a(a.y, b.y, c1));
  vb = float2_to_pair<BF16>(turn_b(a.x, b.x, c0), turn_b(a.y, b.y, c1));
}

// Eight pairs: channels i .. i + 7 (va) and i + rot / 2 .. (vb), a = their angles.
template <bool BF16>
__device__ __forceinline__ void turn_halves(uint4& va, uint4& vb, const float2* a) {
  turn_words<BF16>(va.x, vb.x, angles2(a));
  turn_words<BF16>(va.y, vb.y, angles2(a + 2));
  turn_words<BF16>(va.z, vb.z, angles2(a + 4));
  turn_words<BF16>(va.w, vb.w, angles2(a + 6));
}

// Channels [8 vec, 8 vec + 8) of a head after the turn; `own` holds them before,
// `head` is the whole head in memory (the pairs' other channels are read there).
template <bool BF16>
__device__ __forceinline__ uint4 turned_chunk(uint4 own, const uint16_t* head, int vec, const float2* a,
                                              int rot, int interleaved) {
  const int c0 = vec * 8;
  if (c0 >= rot) return own;
  const int half = rot >> 1;
  if (rotate_aligned(rot, interleaved)) {
    if (interleaved) return turn_interleaved<BF16>(own, a + (c0 >> 1));
    const bool second = c0 >= half;
    uint4 other = __ldg(reinterpret_cast<const uint4*>(head + (second ? c0 - half : c0 + half)));
    if (second) {
      turn_halves<BF16>(other, own, a + (c0 - half));
    } else {
      turn_halves<BF16>(own, other, a + c0);
    }
    return own;
  }
  uint32_t w[4] = {own.x, own.y, own.z, own.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int c = c0 + j;
    if (c >= rot) continue;
    const bool second = interleaved ? (c & 1) != 0 : c >= half;
    const int i = interleaved ? c >> 1 : second ? c - half : c;
    const int oc = interleaved ? c ^ 1 : second ? c - half : c + half;
    const float mine = one_to_float<BF16>(static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1))));
    // (the word itself may hold the partner already turned: read it from memory)
    const float theirs = one_to_float<BF16>(__ldg(head + oc));
    const float2 cs = __ldg(a + i);
    const uint32_t r = float_to_one<BF16>(second ? turn_b(theirs, mine, cs) : turn_a(mine, theirs, cs));
    w[j >> 1] = j & 1 ? (w[j >> 1] & 0xffffu) | (r << 16) : (w[j >> 1] & 0xffff0000u) | r;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The units of tokens [t0, t0 + p.tokens) by a CTA's THREADS threads, U at a time
// a thread so that as many loads are on their way.
template <bool BF16, RotateKind KIND, int THREADS>
__device__ __forceinline__ void rotate_tokens(const RotateParams& p, long long t0, int tid) {
  constexpr int U = KIND == kSingle ? 1 : 4;
  const int n = static_cast<int>(min(static_cast<long long>(p.tokens), p.n_tokens - t0));
  const uint32_t total = static_cast<uint32_t>(n) * p.per.d;
  const int half = p.rot >> 1;
  const bool copies = p.x != p.out;
  for (uint32_t i0 = tid; i0 < total; i0 += U * THREADS) {
    const uint16_t* x[U];
    uint16_t* out[U];
    const float2* a[U];
    int c[U];
    uint4 va[U], vb[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const uint32_t i = min(i0 + k * THREADS, total - 1);
      const uint32_t t = i / p.per, r = i - t * p.per.d, h = r / p.units, u = r - h * p.units.d;
      x[k] = p.x + (t0 + t) * p.x_stride + h * p.D;
      out[k] = p.out + (t0 + t) * p.out_stride + h * p.D;
      a[k] = p.angles + (t0 + t) * half;
      c[k] = static_cast<int>(u);
      if constexpr (KIND == kInterleaved) {
        c[k] = 8 * c[k];
        va[k] = *reinterpret_cast<const uint4*>(x[k] + c[k]);
      } else if constexpr (KIND == kHalves) {
        c[k] = c[k] < p.rot / 16 ? 8 * c[k] : p.rot + 8 * (c[k] - p.rot / 16);
        va[k] = *reinterpret_cast<const uint4*>(x[k] + c[k]);
        if (c[k] < half) vb[k] = *reinterpret_cast<const uint4*>(x[k] + c[k] + half);
      }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (i0 + k * THREADS >= total) break;
      if constexpr (KIND == kSingle) {
        const int turning = (half + 3) / 4;
        if (c[k] < turning) {
          for (int i = 4 * c[k]; i < min(4 * c[k] + 4, half); ++i) {
            const int ca = p.interleaved ? 2 * i : i, cb = p.interleaved ? 2 * i + 1 : i + half;
            const float xa = one_to_float<BF16>(x[k][ca]), xb = one_to_float<BF16>(x[k][cb]);
            const float2 cs = __ldg(a[k] + i);
            out[k][ca] = float_to_one<BF16>(turn_a(xa, xb, cs));
            out[k][cb] = float_to_one<BF16>(turn_b(xa, xb, cs));
          }
        } else if (copies) {
          const int c0 = p.rot + 8 * (c[k] - turning);
          for (int j = c0; j < min(c0 + 8, p.D); ++j) out[k][j] = x[k][j];
        }
        continue;
      }
      const bool turns = c[k] < p.rot;
      if constexpr (KIND == kInterleaved) {
        if (turns) va[k] = turn_interleaved<BF16>(va[k], a[k] + (c[k] >> 1));
      } else if (turns) {
        turn_halves<BF16>(va[k], vb[k], a[k] + c[k]);
        *reinterpret_cast<uint4*>(out[k] + c[k] + half) = vb[k];
      }
      if (turns || copies) *reinterpret_cast<uint4*>(out[k] + c[k]) = va[k];
    }
  }
}

// The same where the kind is known at run time only.
template <bool BF16, int THREADS>
__device__ __forceinline__ void rotate_any(const RotateParams& p, long long t0, int tid) {
  if (!rotate_aligned(p.rot, p.interleaved)) rotate_tokens<BF16, kSingle, THREADS>(p, t0, tid);
  else if (p.interleaved) rotate_tokens<BF16, kInterleaved, THREADS>(p, t0, tid);
  else rotate_tokens<BF16, kHalves, THREADS>(p, t0, tid);
}

// CTAs of `threads` that turn p's heads: enough units a CTA for every thread's
// loads in flight, fewer while that leaves SMs idle.
inline long long rotate_ctas(RotateParams* p, int threads) {
  const long long per = p->per.d, all = per * p->n_tokens;
  const long long want = std::min<long long>(8 * threads, std::max<long long>(threads, all / (152 * 4)));
  p->tokens = static_cast<int>(std::max<long long>(1, std::min<long long>(want / per, p->n_tokens)));
  p->per = divisor(p->per.d, per * p->tokens);
  p->units = divisor(p->units.d, per);
  return (p->n_tokens + p->tokens - 1) / p->tokens;
}

struct PagedStoreParams {
  uint8_t* pages[2];  // K, V: [n_pages][H][ps][D]
  float* scale[2];    // [n_pages][H]
  const void* x[2];   // k, v: token t, head h at t * stride + h * D
  long long stride[2];
  const int* slots;
  int n_tokens;
  int n_pages, H, lg_ps;
  int chunk;  // tokens a CTA looks at
  int* err;
  // kvq_paged_append: keys turn by their tokens' angles [n_tokens][rot / 2]
  // (rot 0: they are stored as they are)
  const float2* angles;
  int rot, interleaved;
  RotateParams q;  // the step's queries; n_heads 0: none
};

struct AnglesParams {
  const int* positions;
  const int64_t* turns;
  float2* angles;
  int n_tokens, half;
  float magnitude;
  Divisor lanes;  // threads of a token
};

// Checks a rotary description against heads of head_dim (KVQ_ERR_INVALID_ARG).
kvq_status check_rotary(const kvq_rotary* r, int head_dim, int n_tokens);
// Fills *p after checking the arguments of a call that turns heads.
kvq_status rotate_params(RotateParams* p, const kvq_rotary* rotary, const void* x, int dtype, long long x_stride,
                         void* out, long long out_stride, int n_tokens, int n_heads, int head_dim);
cudaError_t launch_rotary_angles(AnglesParams p, cudaStream_t st);
cudaError_t launch_paged_store(const PagedStoreParams& p, int D, int dtype, cudaStream_t st);
cudaError_t launch_rotate(const RotateParams& p, int dtype, cudaStream_t st);

}  // namespace kvq
