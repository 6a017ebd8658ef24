// quant_blocks.hip -- E4M3 codes with one fp32 scale per row and 128 values,
// or per 128 x 128 block.
//
//   s = fl32(amax / 448), amax over the block's finite magnitudes; 1 if that is
//   0, at least 2^-126 (so that 1 / s is finite);
//   code = E4M3(fl32(x / s)), round to nearest even, saturating (infinities
//   too); a NaN gives the NaN code 0x7f.
// gated: x = SiLU(gate) * up in fp32, gate and up the two halves of a row.
//
// Bytes bound it (16384 x 7168 bf16 65 us, 5.4 TB/s; 8192 x 4096 fp32 28, 6.0), the
// gates' arithmetic where there are any (65536 x 1024 82, 4.1), and the launch when
// small (64 x 4096 3.2).
#include "block_gemm.hpp"
#include "common.hpp"
#include "launch.hpp"

namespace moe {

// Eight values of a row; zeros beyond it.
template <int DT>
__device__ __forceinline__ void load8(const void* base, size_t at, float (&v)[8]) {
  if constexpr (DT == DT_F32) {
    const i32x4 a = ld16(reinterpret_cast<const float*>(base) + at);
    const i32x4 b = ld16(reinterpret_cast<const float*>(base) + at + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __int_as_float(a[i]);
      v[4 + i] = __int_as_float(b[i]);
    }
  } else {
    const i32x4 a = ld16(reinterpret_cast<const uint16_t*>(base) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float((uint32_t)a[i] << 16);
      v[2 * i + 1] = __uint_as_float((uint32_t)a[i] & 0xffff0000u);
    }
  }
}

__device__ __forceinline__ float amax8(const float (&v)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = __builtin_fabsf(v[i]);
    m = fmaxf(m, a <= 3.40282347e+38f ? a : 0.0f);
  }
  return m;
}

// The largest magnitude's bits, NaN above infinity above all others.
__device__ __forceinline__ uint32_t largest_bits(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  return m;
}

__device__ __forceinline__ float block_scale(float amax) {
  return amax > 0.0f ? fmaxf(amax / 448.0f, 1.17549435e-38f) : 1.0f;
}

// e^v.  The exponent in two parts (an argument of 10 would lose four bits of the
// result to the rounding of v log2 e, and with them codes at a border): log2 e to 16
// bits times a bf16 value, or its half, is exact, of an fp32 value's product the rest
// comes from a fused multiply-add.  In u = 2^-24: the hardware's 2, this addition's 1
// and, for bf16, v^2 / 5000 that the first order leaves out: 4.3 at 80.
template <int DT>
__device__ __forceinline__ float exp_near(float v) {
  constexpr float kHi = DT == DT_F32 ? 1.44269502162933349609f : 1.442687988281250f;
  constexpr float kLo = DT == DT_F32 ? 1.334975816e-08f : 4.888495152e-06f;  // (log2 e - kHi) ln 2
  constexpr float kLn2 = 0.693147180559945309417f;
  const float t = v * kHi;
  float low = v * kLo;
  if constexpr (DT == DT_F32) low = __builtin_fmaf(__builtin_fmaf(v, kHi, -t), kLn2, low);
  const float e = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(e, low, e);
}

// SiLU(v) = v / (1 + e^-v), the quotient with one correction: within 7 u (with the
// product and the scale behind it 3.4 measured).  Beyond 80, where 1 + e^-80 is 1, it
// is v or v e^v, the power as a square since it may be subnormal: within 9 u where it
// is not (-inf gives the formula's NaN).
template <int DT>
__device__ __forceinline__ float silu_near(float v) {
  const float d = 1.0f + exp_near<DT>(-v);
  const float r = __builtin_amdgcn_rcpf(d), q = v * r;
  return __builtin_fmaf(__builtin_fmaf(-q, d, v), r, q);
}
template <int DT>
__device__ __forceinline__ float silu_far(float v) {
  const float e = exp_near<DT>(0.5f * v);
  return v > 0.0f ? v : v * e * e;
}

// v = SiLU(v) * w.  A value does not depend on the gates beside it.
template <int DT>
__device__ __forceinline__ void gate8(float (&v)[8], const float (&w)[8]) {
  constexpr float kNear = 80.0f;
  float most = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) most = fmaxf(most, __builtin_fabsf(v[i]));
  if (__builtin_expect(!(most <= kNear), 0)) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = (__builtin_fabsf(v[i]) <= kNear ? silu_near<DT>(v[i]) : silu_far<DT>(v[i])) * w[i];
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = silu_near<DT>(v[i]) * w[i];
}

// Codes of eight values, little-endian.
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float s) {
  const float r = 1.0f / s;
  const bool fast = e4m3_fast_scale(s, r);
  uint32_t lo = e4m3_codes4(v[0], v[1], v[2], v[3], s, r, fast), hi = e4m3_codes4(v[4], v[5], v[6], v[7], s, r, fast);
  // (those of NaN are saturated ones here, of either sign)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (v[i] != v[i]) lo = (lo & ~(0xffu << (8 * i))) | 0x7fu << (8 * i);
    if (v[4 + i] != v[4 + i]) hi = (hi & ~(0xffu << (8 * i))) | 0x7fu << (8 * i);
  }
  return make_uint2(lo, hi);
}

// The same where all values and their quotients are ordinary: one test for the
// eight, since what e4m3_codes4 tests four by four costs as much as the rest of
// it here (the kernel's VALU time is about that of its bytes).
__device__ __forceinline__ uint2 codes8_fast(const float (&v)[8], float s) {
  const float r = 1.0f / s;
  float q[8], least = 1.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q0 = v[i] * r;
    q[i] = __builtin_fmaf(__builtin_fmaf(-q0, s, v[i]), r, q0);
    least = fminf(least, __builtin_fabsf(q[i]));
  }
  if (__builtin_expect(!e4m3_fast_scale(s, r) || !(least >= 0x1p-9f), 0)) return codes8(v, s);
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = __builtin_amdgcn_fmed3f(q[i], -448.0f, 448.0f);
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
  return make_uint2((uint32_t)lo, (uint32_t)hi);
}

// One scale per row and block.  The blocks of all rows, row by row, are dealt out:
// 32 to a workgroup, eight lanes each (values 8 c and 64 + 8 c on of lane c), so
// that no lane is idle for rows of any length.  One block to eight lanes at a
// time: 16384 x 7168 bf16 68.0 us (5.2 TB/s, the copy's rate); two 74.2, four 83.6
// (fewer waves on a compute unit).  inv22, inv64: 2^22 and 2^64 over the blocks of
// a row, rounded up (inv64 0: one block).
template <int DT, bool GATED>
__global__ __launch_bounds__(256) void quant_rows_kernel(QuantArgs a, int KB, uint32_t inv22, uint64_t inv64) {
  const int lane = threadIdx.x & 63, c = lane & 7;
  const int limit = a.num_rows ? min(a.M, *a.num_rows) : a.M;
  const uint64_t first = (uint64_t)blockIdx.x * 32, row0 = inv64 ? __umul64hi(first, inv64) : first;
  const uint32_t x = (uint32_t)(first - row0 * KB) + (threadIdx.x >> 3);  // below 544: the product is exact
  const uint32_t down = inv64 ? (x * inv22) >> 22 : x;
  const int64_t row = (int64_t)(row0 + down);
  const int blk = (int)(x - down * KB);
  if (row >= limit) return;
  float v[2][8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[h][i] = 0.0f;
    const int col = blk * 128 + h * 64 + c * 8;
    if (col < a.K) {
      const size_t at = (size_t)row * a.x_stride + col;
      load8<DT>(a.x, at, v[h]);
      if constexpr (GATED) {
        float w[8];
        load8<DT>(a.x, at + a.K, w);
        gate8<DT>(v[h], w);
      }
    }
  }
  // the eight lanes of a block go together everywhere
  uint32_t most = max(largest_bits(v[0]), largest_bits(v[1]));
  most = max(most, (uint32_t)__builtin_amdgcn_mov_dpp((int)most, 0xB1, 0xf, 0xf, true));   // lanes 1 apart
  most = max(most, (uint32_t)__builtin_amdgcn_mov_dpp((int)most, 0x4E, 0xf, 0xf, true));   // 2 apart
  most = max(most, (uint32_t)__builtin_amdgcn_mov_dpp((int)most, 0x141, 0xf, 0xf, true));  // the other four of eight
  const bool odd = most >= 0x7f800000u;  // infinities or NaN: their magnitudes do not count
  float m = __uint_as_float(most);
  if (__builtin_expect(odd, 0)) {
    m = fmaxf(amax8(v[0]), amax8(v[1]));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, kWave));
  }
  const float s = block_scale(m);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int col = blk * 128 + h * 64 + c * 8;
    if (col < a.K)
      *reinterpret_cast<uint2*>(a.codes + (size_t)row * a.K + col) =
          __builtin_expect(odd, 0) ? codes8(v[h], s) : codes8_fast(v[h], s);
  }
  if (c == 0) a.scales[row * a.s_row + blk * a.s_block] = s;
}

// One scale per 128 x 128 block: a workgroup each, thread t the 8 columns
// t mod 16 of rows t / 16 + 16 q.
template <int DT>
__global__ __launch_bounds__(256) void quant_tiles_kernel(QuantArgs a) {
  __shared__ float part[4];
  const int col = blockIdx.y * 128 + (threadIdx.x & 15) * 8;
  const long long row0 = (long long)blockIdx.x * 128 + threadIdx.x / 16;
  float v[8][8], m = 0.0f;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[q][i] = 0.0f;
    if (row0 + 16 * q < a.M && col < a.K) load8<DT>(a.x, (size_t)(row0 + 16 * q) * a.x_stride + col, v[q]);
    m = fmaxf(m, amax8(v[q]));
  }
  m = wave_max(m);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
  __syncthreads();
  const float s = block_scale(fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3])));
#pragma unroll
  for (int q = 0; q < 8; ++q)
    if (row0 + 16 * q < a.M && col < a.K)
      *reinterpret_cast<uint2*>(a.codes + (size_t)(row0 + 16 * q) * a.K + col) = codes8(v[q], s);
  if (threadIdx.x == 0) a.scales[blockIdx.x * a.s_row + blockIdx.y * a.s_block] = s;
}

int launch_quant_blocks(const QuantArgs& a, int dt, bool gated, int block_rows, hipStream_t st) {
  QuantArgs c = a;
  int KB = (a.K + 127) / 128;
  if (block_rows == 128) {
    void* args[] = {&c};
    return (int)hipLaunchKernel(dt == DT_F32 ? (void*)quant_tiles_kernel<DT_F32> : (void*)quant_tiles_kernel<DT_BF16>,
                                dim3((unsigned)((a.M + 127) / 128), (unsigned)KB), dim3(256), args, 0, st);
  }
  uint32_t inv22 = ((1u << 22) + KB - 1) / KB;
  uint64_t inv64 = KB == 1 ? 0 : ~0ull / KB + 1;
  void* args[] = {&c, &KB, &inv22, &inv64};
  const void* k = dt == DT_F32 ? gated ? (void*)quant_rows_kernel<DT_F32, true> : (void*)quant_rows_kernel<DT_F32, false>
                  : gated      ? (void*)quant_rows_kernel<DT_BF16, true>
                               : (void*)quant_rows_kernel<DT_BF16, false>;
  const long long groups = ((long long)a.M * KB + 31) / 32;
  if (groups * 256 > kMaxThreads) return kTooManyTiles;
  return (int)hipLaunchKernel(k, dim3((unsigned)groups), dim3(256), args, 0, st);
}

}  // namespace moe
