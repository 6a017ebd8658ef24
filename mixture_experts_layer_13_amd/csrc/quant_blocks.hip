// quant_blocks.hip -- E4M3 codes with one fp32 scale per row and 128 values,
// or per 128 x 128 block.
//
//   s = fl32(amax / 448), amax over the block's finite magnitudes; 1 if that is
//   0, at least 2^-126 (so that 1 / s is finite);
//   code = E4M3(fl32(x / s)), round to nearest even, saturating (infinities
//   too); a NaN gives the NaN code 0x7f.
// gated: x = SiLU(gate) * up in fp32, gate and up the two halves of a row.
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

__device__ __forceinline__ float block_scale(float amax) {
  return amax > 0.0f ? fmaxf(amax / 448.0f, 1.17549435e-38f) : 1.0f;
}

// Codes of eight values, little-endian.
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float s) {
  const float r = 1.0f / s;
  const bool fast = e4m3_fast_scale(s, r);
  uint32_t lo = e4m3_codes4(v[0], v[1], v[2], v[3], s, r, fast), hi = e4m3_codes4(v[4], v[5], v[6], v[7], s, r, fast);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (v[i] != v[i]) lo |= 0x7fu << (8 * i);
    if (v[4 + i] != v[4 + i]) hi |= 0x7fu << (8 * i);
  }
  return make_uint2(lo, hi);
}

// One scale per row and block: a wave takes 512 columns (four blocks of 16
// lanes, 8 values a lane) of RPW rows.
template <int DT, bool GATED, int RPW>
__global__ __launch_bounds__(256) void quant_rows_kernel(QuantArgs a) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int limit = a.num_rows ? min(a.M, *a.num_rows) : a.M;
  const int row0 = ((int)blockIdx.x * 4 + wv) * RPW;
  const int col = blockIdx.y * 512 + lane * 8;
  float v[RPW][8];
#pragma unroll
  for (int r = 0; r < RPW; ++r) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[r][i] = 0.0f;
    if (row0 + r < limit && col < a.K) {
      const size_t at = (size_t)(row0 + r) * a.x_stride + col;
      load8<DT>(a.x, at, v[r]);
      if constexpr (GATED) {
        float u[8];
        load8<DT>(a.x, at + a.K, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[r][i] = silu(v[r][i]) * u[i];
      }
    }
  }
#pragma unroll
  for (int r = 0; r < RPW; ++r) {
    float m = amax8(v[r]);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, kWave));
    if (row0 + r >= limit || col >= a.K) continue;
    const float s = block_scale(m);
    *reinterpret_cast<uint2*>(a.codes + (size_t)(row0 + r) * a.K + col) = codes8(v[r], s);
    if ((lane & 15) == 0) a.scales[(row0 + r) * a.s_row + (col / 128) * a.s_block] = s;
  }
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

template <int DT>
static void* quant_rows_of(bool gated, bool many) {
  if (gated) return many ? (void*)quant_rows_kernel<DT, true, 4> : (void*)quant_rows_kernel<DT, true, 1>;
  return many ? (void*)quant_rows_kernel<DT, false, 4> : (void*)quant_rows_kernel<DT, false, 1>;
}

int launch_quant_blocks(const QuantArgs& a, int dt, bool gated, int block_rows, hipStream_t st) {
  QuantArgs c = a;
  void* args[] = {&c};
  if (block_rows == 128)
    return (int)hipLaunchKernel(dt == DT_F32 ? (void*)quant_tiles_kernel<DT_F32> : (void*)quant_tiles_kernel<DT_BF16>,
                                dim3((unsigned)((a.M + 127) / 128), (unsigned)((a.K + 127) / 128)), dim3(256), args, 0, st);
  const int parts = (a.K + 511) / 512;
  const bool many = (long long)a.M * parts >= 16384;
  const int per = many ? 16 : 4;
  return (int)hipLaunchKernel(dt == DT_F32 ? quant_rows_of<DT_F32>(gated, many) : quant_rows_of<DT_BF16>(gated, many),
                              dim3((unsigned)((a.M + per - 1) / per), (unsigned)parts), dim3(256), args, 0, st);
}

}  // namespace moe
