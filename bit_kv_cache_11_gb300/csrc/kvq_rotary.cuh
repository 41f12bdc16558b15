// kvq_rotary.cuh — turning heads by rotary angles (include/kvq.h, "Rotary
// positions"): the arithmetic that kvq_rotate and the paged appends share.
// Internal to csrc/.
#pragma once

#include "kvq_paged.cuh"

namespace kvq {

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
  int units;        // of a head, rotate_units()
};

// A unit of a head is what one thread turns: the channels of whole pairs, so
// that out may be x itself.  Where the layout's chunks of eight channels are
// aligned (rotate_aligned) a unit is
//   interleaved   one chunk, its four pairs or (from rot on) its copy
//   half          two chunks of eight pairs, or a chunk to copy
// and else four pairs of single channels, or eight channels to copy.
inline __host__ __device__ bool rotate_aligned(int rot, int interleaved) {
  return rot % (interleaved ? 8 : 16) == 0;
}
inline __host__ __device__ int rotate_units(int D, int rot, int interleaved) {
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

// Unit u of head h of token t.
template <bool BF16>
__device__ __forceinline__ void rotate_unit(const RotateParams& p, long long t, int h, int u) {
  const uint16_t* x = p.x + t * p.x_stride + static_cast<long long>(h) * p.D;
  uint16_t* out = p.out + t * p.out_stride + static_cast<long long>(h) * p.D;
  const float2* a = p.angles + t * (p.rot >> 1);
  const bool aligned = rotate_aligned(p.rot, p.interleaved);
  const bool copies = x != out;
  if (aligned && p.interleaved) {
    if (8 * u < p.rot || copies) {
      uint4 v = *reinterpret_cast<const uint4*>(x + 8 * u);
      if (8 * u < p.rot) v = turn_interleaved<BF16>(v, a + 4 * u);
      *reinterpret_cast<uint4*>(out + 8 * u) = v;
    }
    return;
  }
  const int half = p.rot >> 1;
  if (aligned) {
    if (u < p.rot / 16) {
      uint4 va = *reinterpret_cast<const uint4*>(x + 8 * u), vb = *reinterpret_cast<const uint4*>(x + half + 8 * u);
      turn_halves<BF16>(va, vb, a + 8 * u);
      *reinterpret_cast<uint4*>(out + 8 * u) = va;
      *reinterpret_cast<uint4*>(out + half + 8 * u) = vb;
    } else if (copies) {
      const int c = p.rot + 8 * (u - p.rot / 16);
      *reinterpret_cast<uint4*>(out + c) = *reinterpret_cast<const uint4*>(x + c);
    }
    return;
  }
  const int turning = (half + 3) / 4;
  if (u < turning) {
    for (int i = 4 * u; i < min(4 * u + 4, half); ++i) {
      const int ca = p.interleaved ? 2 * i : i, cb = p.interleaved ? 2 * i + 1 : i + half;
      const float xa = one_to_float<BF16>(x[ca]), xb = one_to_float<BF16>(x[cb]);
      const float2 cs = __ldg(a + i);
      out[ca] = float_to_one<BF16>(turn_a(xa, xb, cs));
      out[cb] = float_to_one<BF16>(turn_b(xa, xb, cs));
    }
  } else if (copies) {
    const int c0 = p.rot + 8 * (u - turning);
    for (int c = c0; c < min(c0 + 8, p.D); ++c) out[c] = x[c];
  }
}

struct AnglesParams {
  const int* positions;
  const int64_t* turns;
  float2* angles;
  int n_tokens, half;
  float magnitude;
};

// Checks a rotary description against heads of head_dim (KVQ_ERR_INVALID_ARG).
kvq_status check_rotary(const kvq_rotary* r, int head_dim, int n_tokens);
// Fills *p after checking the arguments of a call that turns heads.
kvq_status rotate_params(RotateParams* p, const kvq_rotary* rotary, const void* x, int dtype, long long x_stride,
                         void* out, long long out_stride, int n_tokens, int n_heads, int head_dim);
cudaError_t launch_rotary_angles(const AnglesParams& p, cudaStream_t st);
cudaError_t launch_rotate(const RotateParams& p, int dtype, cudaStream_t st);

}  // namespace kvq
