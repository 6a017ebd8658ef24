// rotate.hpp -- rotary angles with several position axes, shared by the
// rotation kernel (rope_axes.hip) and the cache append (kv_append.hip).
//
// Pair i of a token turns by positions[axis(i)][token] * inv_freq[i] radians.
// In fp32 that product is off by half an ulp of the angle: 2^-8 rad at
// position 2^17 times inv_freq 1, and more beyond.  So it is formed as turns
// from a frequency of two fp32 terms, and the whole turns are taken off the
// leading product inside a fused multiply-add (|position| < 2^24 is exact in
// fp32): only the fraction of a turn, at most 1/2, is ever rounded.
#pragma once

#include "common.hpp"

namespace moe {

struct RotateArgs {
  const int32_t* pos;        // [axes][T]
  const int32_t* pair_axis;  // [half] or NULL (axis 0)
  const float* inv_freq;     // [half]
  int T, axes, half;         // half = rotary_dim / 2 pairs per head
  int interleaved, inverse;
};

constexpr double kInvTwoPi = 0.15915494309189533577;

// A frequency in turns per position, as two terms.
struct TurnFreq {
  float hi, lo;
};

__device__ __forceinline__ TurnFreq turn_freq(float inv_freq) {
  // 1 / (2 pi) as two fp32 terms; the first product's rounding is recovered
  constexpr float h = 0.15915494f, l = (float)(kInvTwoPi - (double)h);
  const float hi = inv_freq * h;
  return TurnFreq{hi, __builtin_fmaf(inv_freq, l, __builtin_fmaf(inv_freq, h, -hi))};
}

// {cos, sin} of the angle of position pos.  gfx950's sine and cosine take
// turns, and on [-1/2, 1/2] are within 2^-22.9 of the exact values (measured
// at every multiple of 2^-25 there); rounding the fraction adds at most
// 2^-23.3, and the two products and the sum of a rotation 2^-24 each, so that a
// rotated value is within 2^-21.7 (|u| + |v|).  A polynomial of the same error
// takes five times as long, and an append was bound by it.
__device__ __forceinline__ float2 rotate_cs(int pos, TurnFreq f, int inverse) {
  const float x = (float)pos;
  const float t = __builtin_fmaf(x, f.lo, __builtin_fmaf(x, f.hi, -__builtin_rintf(x * f.hi)));
  return make_float2(__builtin_amdgcn_cosf(t), __builtin_amdgcn_sinf(inverse ? -t : t));
}

// Axis of pair i; -1 (the pair is left unturned) when the map names none.
__device__ __forceinline__ int rotate_axis(const RotateArgs& r, int i) {
  if (!r.pair_axis) return 0;
  const int a = r.pair_axis[i];
  return (unsigned)a < (unsigned)r.axes ? a : -1;
}

// A head's values are handled as pairs of vectors of E values: vector g of a
// half and its counterpart half a stretch on, for the rotated values
// (stretch 2 half) and the passed ones behind them alike.  With halves pairing
// the two vectors hold the members of pairs E g..; interleaved, each holds E/2
// whole pairs, from E g / 2 and half / 2 + E g / 2 on.  Either way consecutive
// g are consecutive in memory.  First indices of pair-of-vectors g's two.
template <int E>
__device__ __forceinline__ void unit_groups(int g, int half, int D, int& p, int& q) {
  const int rot = half / E;
  if (g < rot) {
    p = E * g;
    q = half + E * g;
  } else {
    p = 2 * half + E * (g - rot);
    q = p + (D >> 1) - half;
  }
}

// Pair of {cos, sin} number i (0..E-1) of unit g.
template <int E>
__device__ __forceinline__ int unit_pair(int g, int i, int half, int interleaved) {
  return interleaved ? (i < E / 2 ? E / 2 * g + i : half / 2 + E / 2 * (g - 1) + i) : E * g + i;
}

// Rotates a unit in place (a: first vector, b: second); cs[i] is {cos, sin} of
// its pair number i.
template <int E>
__device__ __forceinline__ void rotate_unit(float* a, float* b, const float2* cs, int interleaved) {
  if (interleaved) {
#pragma unroll
    for (int j = 0; j < E / 2; ++j) {
      const float u0 = a[2 * j], v0 = a[2 * j + 1], u1 = b[2 * j], v1 = b[2 * j + 1];
      const float2 c0 = cs[j], c1 = cs[E / 2 + j];
      a[2 * j] = __builtin_fmaf(u0, c0.x, -(v0 * c0.y));
      a[2 * j + 1] = __builtin_fmaf(v0, c0.x, u0 * c0.y);
      b[2 * j] = __builtin_fmaf(u1, c1.x, -(v1 * c1.y));
      b[2 * j + 1] = __builtin_fmaf(v1, c1.x, u1 * c1.y);
    }
  } else {
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const float u = a[j], v = b[j];
      a[j] = __builtin_fmaf(u, cs[j].x, -(v * cs[j].y));
      b[j] = __builtin_fmaf(v, cs[j].x, u * cs[j].y);
    }
  }
}

// Values idx.. of the tensor at base: E of them (a multiple of a 16-byte load).
template <int XT, int E>
struct RawVec {
  i32x4 w[E * (XT == DT_BF16 ? 2 : 4) / 16];
};

template <int XT, int E>
__device__ __forceinline__ RawVec<XT, E> load_vec(const void* base, size_t idx) {
  RawVec<XT, E> r;
  const char* at = reinterpret_cast<const char*>(base) + idx * (XT == DT_BF16 ? 2 : 4);
#pragma unroll
  for (int k = 0; k < (int)(sizeof(r.w) / 16); ++k) r.w[k] = ld16(at + 16 * k);
  return r;
}

template <int XT, int E>
__device__ __forceinline__ void unpack_vec(const RawVec<XT, E>& r, float* v) {
#pragma unroll
  for (int j = 0; j < E; ++j) {
    if (XT == DT_BF16) {
      const uint32_t w = (uint32_t)r.w[j >> 3][(j >> 1) & 3];
      v[j] = __uint_as_float(j & 1 ? w & 0xffff0000u : w << 16);
    } else {
      v[j] = __int_as_float(r.w[j >> 2][j & 3]);
    }
  }
}

}  // namespace moe
