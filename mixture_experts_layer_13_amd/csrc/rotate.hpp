// rotate.hpp -- rotary angles with several position axes, shared by the
// rotation kernel (rope_axes.hip) and the cache append (kv_append.hip).
//
// Pair i of a token turns by positions[axis(i)][token] * inv_freq[i] radians.
// In fp32 that product is off by half an ulp of the angle: 2^-8 rad at
// position 2^17 times inv_freq 1, and more beyond.  So it is formed and
// reduced in fp64 as turns (|position| < 2^24: the error stays below 2^-26
// rad), and only the fraction of a turn, at most 1/2, goes on in fp32.
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

// {cos, sin} of turns * 2 pi, the turn given in fp64.
__device__ __forceinline__ float2 rotate_cs(double turns, int inverse) {
  const float frac = (float)(turns - __builtin_rint(turns));
  float s, c;
  sincospif(2.0f * frac, &s, &c);
  return make_float2(c, inverse ? -s : s);
}

// Axis of pair i; -1 (the pair is left unturned) when the map names none.
__device__ __forceinline__ int rotate_axis(const RotateArgs& r, int i) {
  if (!r.pair_axis) return 0;
  const int a = r.pair_axis[i];
  return (unsigned)a < (unsigned)r.axes ? a : -1;
}

// Raw bits of 8 consecutive values at p: one 16-byte load for bf16, two for f32.
template <int XT>
__device__ __forceinline__ void load8(const void* base, size_t idx, i32x4 raw[2]) {
  if (XT == DT_BF16) {
    raw[0] = ld16(reinterpret_cast<const uint16_t*>(base) + idx);
  } else {
    raw[0] = ld16(reinterpret_cast<const float*>(base) + idx);
    raw[1] = ld16(reinterpret_cast<const float*>(base) + idx + 4);
  }
}

template <int XT>
__device__ __forceinline__ void unpack8(const i32x4 raw[2], float v[8]) {
  if (XT == DT_BF16) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = bf16_bits_to_f32((uint32_t)raw[0][j] & 0xffffu);
      v[2 * j + 1] = bf16_bits_to_f32((uint32_t)raw[0][j] >> 16);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = __int_as_float(raw[0][j]);
      v[4 + j] = __int_as_float(raw[1][j]);
    }
  }
}

// A unit is 16 values of one head: with halves pairing the first D/16 units'
// rotated part pairs values 8g.. with half + 8g.., interleaved and
// pass-through units are 16 consecutive values.  First indices of its two
// groups of 8 (rot_units = half / 8 units are rotated).
__device__ __forceinline__ void unit_groups(int g, int half, int interleaved, int& p, int& q) {
  const bool halves = !interleaved && g < (half >> 3);
  p = halves ? 8 * g : 16 * g;
  q = halves ? half + 8 * g : 16 * g + 8;
}

// Rotates a unit's 16 values in place (a = first group of 8, b = second);
// cs[j] is {cos, sin} of pair 8g + j.
__device__ __forceinline__ void rotate_unit(float a[8], float b[8], const float2* cs, int interleaved) {
  if (interleaved) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float u0 = a[2 * j], v0 = a[2 * j + 1], u1 = b[2 * j], v1 = b[2 * j + 1];
      const float2 c0 = cs[j], c1 = cs[4 + j];
      a[2 * j] = __builtin_fmaf(u0, c0.x, -(v0 * c0.y));
      a[2 * j + 1] = __builtin_fmaf(v0, c0.x, u0 * c0.y);
      b[2 * j] = __builtin_fmaf(u1, c1.x, -(v1 * c1.y));
      b[2 * j + 1] = __builtin_fmaf(v1, c1.x, u1 * c1.y);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float u = a[j], v = b[j];
      a[j] = __builtin_fmaf(u, cs[j].x, -(v * cs[j].y));
      b[j] = __builtin_fmaf(v, cs[j].x, u * cs[j].y);
    }
  }
}

}  // namespace moe
