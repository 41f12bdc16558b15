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

// CTAs of `tokens` each (64 bits: token counts go up to 2^31 - 1).
inline long long ctas_of(int n_tokens, int tokens) { return (static_cast<long long>(n_tokens) + tokens - 1) / tokens; }

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
  int step;            // a thread's heads are h, h + step, ..., below n_heads
  int tokens;          // of a CTA
  Divisor per, units;  // threads of a token, units of a head
};

// A unit of a head is what one thread turns: the channels of whole pairs, so
// that out may be x itself.  Where the layout's chunks of eight channels are
// aligned a unit is
//   kInterleaved  one chunk, its four pairs or (from rot on) its copy
//   kHalves       two chunks of eight pairs, or a chunk to copy
// and else (kSingle) four pairs of single channels, or eight channels to copy, which
// takes three to five times as long on prompts (figures in kvq_rotary.cu).
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

// A word of two channels, with the other channels of their pairs: own cos + (-)
// other sin, the same roundings as turn_a (sign -1) and turn_b (1).
template <bool BF16>
__device__ __forceinline__ uint32_t turn_own(uint32_t own, uint32_t other, float4 cs, float sign) {
  const float2 x = pair_to_float2<BF16>(own), y = pair_to_float2<BF16>(other);
  return float2_to_pair<BF16>(__fadd_rn(__fmul_rn(x.x, cs.x), sign * __fmul_rn(y.x, cs.y)),
                              __fadd_rn(__fmul_rn(x.y, cs.z), sign * __fmul_rn(y.y, cs.w)));
}

// Channels [c0, c0 + 8) of `head`, in `own`, after the turn, channel by channel.
template <bool BF16>
__device__ __forceinline__ uint4 turn_single(uint4 own, const uint16_t* head, int c0, const float2* a, int rot,
                                             int interleaved) {
  const int half = rot >> 1;
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

// How a lane turns its chunk of a head, channels [8 vec, 8 vec + 8), where a head's
// chunks lie in consecutive lanes: the other channels of its pairs come from
// another lane, or (kSingle) from memory.
struct ChunkTurn {
  bool turns;   // the chunk has channels that turn
  bool pairs;   // aligned halves: the partner is a lane's whole chunk
  int src;      // that lane
  int angle;    // first angle
  bool second;  // of the two chunks of a pair
  __device__ __forceinline__ ChunkTurn(int vec, int lane, int rot, int interleaved) {
    const int c = vec * 8, half = rot >> 1;
    turns = c < rot;
    pairs = !interleaved && rotate_aligned(rot, interleaved);
    second = !interleaved && c >= half;
    angle = interleaved ? c >> 1 : second ? c - half : c;
    src = !turns || !pairs ? lane : second ? lane - (half >> 3) : lane + (half >> 3);
  }
};

// The chunk `own` of `head` after the turn by angles a [rot / 2].  Whole warps take
// part; a lane that is not `live` loads nothing.  Of two chunks whose channels are
// pairs, the first's lane turns the first four pairs and the second's the last four,
// so that each loads the half of the angles.
template <bool BF16>
__device__ __forceinline__ uint4 turn_chunk(uint4 own, const ChunkTurn& ct, const uint16_t* head, int vec,
                                            const float2* a, int rot, int interleaved, bool live) {
  if (ct.pairs) {
    const uint32_t x = __shfl_sync(~0u, ct.second ? own.x : own.z, ct.src);
    const uint32_t y = __shfl_sync(~0u, ct.second ? own.y : own.w, ct.src);
    uint32_t va[2] = {ct.second ? x : own.x, ct.second ? y : own.y};
    uint32_t vb[2] = {ct.second ? own.z : x, ct.second ? own.w : y};
    if (ct.turns && live) {
      a += ct.angle + (ct.second ? 4 : 0);
      turn_words<BF16>(va[0], vb[0], angles2(a));
      turn_words<BF16>(va[1], vb[1], angles2(a + 2));
    }
    const uint32_t z = __shfl_sync(~0u, ct.second ? va[0] : vb[0], ct.src);
    const uint32_t w = __shfl_sync(~0u, ct.second ? va[1] : vb[1], ct.src);
    if (!ct.turns) return own;
    return ct.second ? make_uint4(z, w, vb[0], vb[1]) : make_uint4(va[0], va[1], z, w);
  }
  if (!ct.turns || !live) return own;
  if (rotate_aligned(rot, interleaved)) return turn_interleaved<BF16>(own, a + ct.angle);
  return turn_single<BF16>(own, head, vec * 8, a, rot, interleaved);
}

// Heads of a thread.
constexpr int kHeads = 4;

// Tokens [t0, t0 + p.tokens) by a CTA's THREADS threads.  A thread turns one unit
// of kHeads heads of a token: their angles are loaded once, and the heads' loads
// are on their way together.  Measured (26298 tokens x 32 heads x 128, bf16): one
// head a thread 84 us (the angles' loads fill the L1), two 74, four 66.
template <bool BF16, RotateKind KIND, int THREADS>
__device__ __forceinline__ void rotate_tokens(const RotateParams& p, long long t0, int tid) {
  const int n = static_cast<int>(min(static_cast<long long>(p.tokens), p.n_tokens - t0));
  const uint32_t total = static_cast<uint32_t>(n) * p.per.d;
  const int half = p.rot >> 1, step = p.step * p.D;
  const bool copies = p.x != p.out;
  for (uint32_t i = tid; i < total; i += THREADS) {
    const uint32_t t = i / p.per, r = i - t * p.per.d, h0 = r / p.units, u = r - h0 * p.units.d;
    const int heads = min(kHeads, static_cast<int>((p.n_heads - h0 + p.step - 1) / p.step));  // h0, h0 + step, ...
    const uint16_t* x = p.x + (t0 + t) * p.x_stride + h0 * p.D;
    uint16_t* out = p.out + (t0 + t) * p.out_stride + h0 * p.D;
    const float2* a = p.angles + (t0 + t) * half;
    if constexpr (KIND == kSingle) {
      const int turning = (half + 3) / 4, v = static_cast<int>(u);
      for (int k = 0; k < heads; ++k, x += step, out += step) {
        if (v < turning) {
          for (int j = 4 * v; j < min(4 * v + 4, half); ++j) {
            const int ca = p.interleaved ? 2 * j : j, cb = p.interleaved ? 2 * j + 1 : j + half;
            const float xa = one_to_float<BF16>(x[ca]), xb = one_to_float<BF16>(x[cb]);
            const float2 cs = __ldg(a + j);
            out[ca] = float_to_one<BF16>(turn_a(xa, xb, cs));
            out[cb] = float_to_one<BF16>(turn_b(xa, xb, cs));
          }
        } else if (copies) {
          const int c0 = p.rot + 8 * (v - turning);
          for (int j = c0; j < min(c0 + 8, p.D); ++j) out[j] = x[j];
        }
      }
    } else {
      int c = 8 * static_cast<int>(u);
      if (KIND == kHalves && c >= half) c += half;
      const bool turns = c < p.rot;
      if (!turns && !copies) continue;
      uint4 va[kHeads], vb[kHeads];
#pragma unroll
      for (int k = 0; k < kHeads; ++k) {
        if (k < heads) {
          va[k] = *reinterpret_cast<const uint4*>(x + c + k * step);
          if (KIND == kHalves && turns) vb[k] = *reinterpret_cast<const uint4*>(x + c + half + k * step);
        }
      }
      float4 cs[4];
      if (turns) {
        a += KIND == kHalves ? c : c >> 1;
#pragma unroll
        for (int j = 0; j < (KIND == kHalves ? 4 : 2); ++j) cs[j] = angles2(a + 2 * j);
      }
#pragma unroll
      for (int k = 0; k < kHeads; ++k) {
        if (k >= heads) break;
        if (turns) {
          if constexpr (KIND == kHalves) {
            turn_words<BF16>(va[k].x, vb[k].x, cs[0]);
            turn_words<BF16>(va[k].y, vb[k].y, cs[1]);
            turn_words<BF16>(va[k].z, vb[k].z, cs[2]);
            turn_words<BF16>(va[k].w, vb[k].w, cs[3]);
            *reinterpret_cast<uint4*>(out + c + half + k * step) = vb[k];
          } else {
            va[k].x = turn_word<BF16>(va[k].x, make_float2(cs[0].x, cs[0].y));
            va[k].y = turn_word<BF16>(va[k].y, make_float2(cs[0].z, cs[0].w));
            va[k].z = turn_word<BF16>(va[k].z, make_float2(cs[1].x, cs[1].y));
            va[k].w = turn_word<BF16>(va[k].w, make_float2(cs[1].z, cs[1].w));
          }
        }
        *reinterpret_cast<uint4*>(out + c + k * step) = va[k];
      }
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

// CTAs of `threads` that turn p's heads: two rounds each (one or four: 66 and 67 us
// instead of 66 for the case above), one while that leaves SMs idle.
inline long long rotate_ctas(RotateParams* p, int threads) {
  p->step = (p->n_heads + kHeads - 1) / kHeads;
  const long long per = static_cast<long long>(p->step) * p->units.d, all = per * p->n_tokens;
  const long long want = std::min<long long>(2 * threads, std::max<long long>(threads, all / (152 * 4)));
  p->tokens = static_cast<int>(std::max<long long>(1, std::min<long long>(want / per, p->n_tokens)));
  p->per = divisor(static_cast<uint32_t>(per), per * p->tokens);
  p->units = divisor(p->units.d, per);
  return ctas_of(p->n_tokens, p->tokens);
}
// CTAs that make `rows` tokens' angles at a time: four rounds each where there are many.
inline long long angles_ctas(int n_tokens, int rows) {
  return std::min(ctas_of(n_tokens, rows), std::max(152LL * 8, ctas_of(n_tokens, 4 * rows)));
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
