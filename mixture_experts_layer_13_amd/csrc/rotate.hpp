// rotate.hpp -- rotary angles with several position axes, shared by the
// rotation kernel (rope_axes.hip) and the cache append (kv_append.hip).
//
// Pair i of a token turns by positions[axis(i)][token] * inv_freq[i] radians.
// In fp32 that product is off by half an ulp of the angle: 2^-8 rad at
// position 2^17 times inv_freq 1, and more beyond.  Positions are whole numbers,
// so the whole turns of a frequency are whole turns of every angle: of
// inv_freq / 2 pi only the fraction is kept, as 64 bits, and the low 64 bits of
// its product with the position are the angle's fraction of a turn.  Whole
// numbers lose nothing, whatever the position and however many the turns (the
// reduction of an argument by a long 1 / 2 pi: Payne and Hanek, 1983).
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

// The fraction of a frequency in turns per position, in units of 2^-64.
struct TurnFreq {
  uint32_t hi, lo;
};

// Within one unit for |inv_freq| <= 2^32: 1 / 2 pi as two doubles (2^-108 of
// it), the first product's rounding recovered, whole turns off exactly.
__device__ __forceinline__ TurnFreq turn_freq(float inv_freq) {
#pragma clang fp contract(off)  // what `rest` recovers must have been rounded off
  constexpr double h = 0x1.45f306dc9c883p-3, l = -0x1.6b01ec5417056p-57;
  const double f = inv_freq, turns = f * h, rest = __builtin_fma(f, l, __builtin_fma(f, h, -turns));
  const double top = (turns - __builtin_rint(turns)) * 0x1p32, whole = __builtin_floor(top);
  const uint64_t u = ((uint64_t)(int64_t)whole << 32) +
                     (uint64_t)(int64_t)__builtin_rint(__builtin_fma(top - whole, 0x1p32, rest * 0x1p64));
  return TurnFreq{(uint32_t)(u >> 32), (uint32_t)u};
}

// A position as its magnitude, and the sign of its angles, with a turn's unit.
struct Place {
  uint32_t n;
  float unit;
};

__device__ __forceinline__ Place place_of(int pos, int inverse) {
  return Place{pos < 0 ? 0u - (uint32_t)pos : (uint32_t)pos, (pos < 0) != (inverse != 0) ? -0x1p-32f : 0x1p-32f};
}

// {cos, sin} of a place's angle.  The fraction of a turn is within 2^-32 of the
// exact one and rounded once, to fp32 in [-1/2, 1/2].  gfx950's sine and cosine
// take turns; with that rounding they are within 2^-22.34 of the exact values
// (measured at every one of the 2^32 fractions).  The two products and the sum of
// a rotation add at most 2^-23, so that a rotated value is within 2^-21.6
// (|u| + |v|).  A polynomial of the same error takes five times as long, and an
// append was bound by it.
__device__ __forceinline__ float2 rotate_cs(Place p, TurnFreq f) {
  const uint32_t turn = p.n * f.hi + __umulhi(p.n, f.lo);
  const float t = (float)(int32_t)turn * p.unit;
  return make_float2(__builtin_amdgcn_cosf(t), __builtin_amdgcn_sinf(t));
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
