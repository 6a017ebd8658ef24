// permute.hip -- tokens into expert order and back, weighted, and the
// gradients of both.
//
// With f = t topk + j a pair, w its weight (1 without weights) and p(f) its
// place in the alignment's padded order (-1: dropped):
//   dispatch           rows[p(f)] = w_f x[t], rows of no pair 0
//   combine            out[t] = sum_j w_f rows[p(f)]
//   dispatch backward  dx[t] = sum_j w_f drows[p(f)],  dw_f = <x[t], drows[p(f)]>
//   combine backward   drows[p(f)] = w_f dout[t],      dw_f = <dout[t], rows[p(f)]>
// so there are two movements, token to rows (scatter) and rows to token
// (gather), each with or without the products that make dw.  Both go token by
// token: a token's row is read (or written) once, and its topk places come
// from pair_pos, so that nothing is added by two workgroups and every result
// is the same on every run.  Products and sums are fp32, in the order of j.
#include "common.hpp"
#include "launch.hpp"
#include "permute.hpp"

namespace moe {

constexpr int kPermWave = 4;  // waves of a workgroup

template <int DT, int VEC>
__device__ __forceinline__ void load_vec(const void* base, size_t at, float (&v)[VEC]) {
  if constexpr (DT == DT_F32) {
#pragma unroll
    for (int q = 0; q < VEC / 4; ++q) {
      const i32x4 d = ld16(reinterpret_cast<const float*>(base) + at + 4 * q);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * q + i] = __int_as_float(d[i]);
    }
  } else {
    uint32_t d[VEC / 2];
    const uint16_t* p = reinterpret_cast<const uint16_t*>(base) + at;
    if constexpr (VEC == 8) {
      const i32x4 r = ld16(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = (uint32_t)r[i];
    } else {
      const uint2 r = *reinterpret_cast<const uint2*>(p);
      d[0] = r.x;
      d[1] = r.y;
    }
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      v[2 * i] = __uint_as_float(d[i] << 16);
      v[2 * i + 1] = __uint_as_float(d[i] & 0xffff0000u);
    }
  }
}

template <int DT, int VEC>
__device__ __forceinline__ void store_vec(void* base, size_t at, const float (&v)[VEC]) {
  if constexpr (DT == DT_F32) {
#pragma unroll
    for (int q = 0; q < VEC / 4; ++q)
      st16(reinterpret_cast<float*>(base) + at + 4 * q,
           i32x4{__float_as_int(v[4 * q]), __float_as_int(v[4 * q + 1]), __float_as_int(v[4 * q + 2]),
                 __float_as_int(v[4 * q + 3])});
  } else {
    uint16_t* p = reinterpret_cast<uint16_t*>(base) + at;
    if constexpr (VEC == 8)
      st16(p, i32x4{(int)pack_bf16x2(v[0], v[1]), (int)pack_bf16x2(v[2], v[3]), (int)pack_bf16x2(v[4], v[5]),
                    (int)pack_bf16x2(v[6], v[7])});
    else
      *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  }
}

// Sum over the workgroup of G values per lane; thread i < G gets value i.
template <int G>
__device__ __forceinline__ float group_sums(float (&v)[G], float (*lds)[G]) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
#pragma unroll
  for (int i = 0; i < G; ++i) {
    const float s = wave_sum(v[i]);
    if (lane == 0) lds[wv][i] = s;
  }
  __syncthreads();
  float s = 0.0f;
  if (threadIdx.x < G)
    for (int q = 0; q < kPermWave; ++q) s += lds[q][threadIdx.x];
  __syncthreads();
  return s;
}

// Place of pair f among rows rows, -1 if it has none.
__device__ __forceinline__ int pair_place(const PermuteArgs& a, int f) {
  const int p = a.pair_pos[f];
  return p >= 0 && p < a.rows ? p : -1;
}

// Token to rows.  Workgroups below M: token blockIdx.x, the vectors of this
// blockIdx.y; the others zero the rows of no pair, 16 rows each.
template <int XT, int RT, bool DOT>
__global__ __launch_bounds__(kPermWave * 64) void scatter_kernel(PermuteArgs a) {
  constexpr int VEC = XT == DT_BF16 && RT == DT_BF16 ? 8 : 4;
  constexpr int G = 8;
  const int n = a.K / VEC, step = gridDim.y * blockDim.x;
  const int v0 = blockIdx.y * blockDim.x + threadIdx.x;
  if ((int)blockIdx.x >= a.M) {
    const int r0 = ((int)blockIdx.x - a.M) * 16;
    const int end = min(min(r0 + 16, a.rows), *a.num_padded);
    for (int r = r0; r < end; ++r) {
      const int f = a.sorted_ids[r];
      if (f >= 0 && f < a.P) continue;
      const float z[VEC] = {};
      for (int v = v0; v < n; v += step) store_vec<RT, VEC>(a.rows_out, (size_t)r * a.rows_out_stride + (size_t)v * VEC, z);
    }
    return;
  }
  const int t = blockIdx.x;
  __shared__ float sums[kPermWave][G];
  for (int j0 = 0; j0 < a.topk; j0 += G) {
    int p[G];
    float w[G], dot[G] = {};
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const int f = t * a.topk + j0 + j;
      p[j] = j0 + j < a.topk ? pair_place(a, f) : -1;
      w[j] = a.weights && p[j] >= 0 ? a.weights[f] : 1.0f;
    }
    for (int v = v0; v < n; v += step) {
      float x[VEC];
      load_vec<XT, VEC>(a.tok_in, (size_t)t * a.tok_in_stride + (size_t)v * VEC, x);
      float r[DOT ? G : 1][VEC];
      if constexpr (DOT) {
#pragma unroll
        for (int j = 0; j < G; ++j)
          if (p[j] >= 0) load_vec<RT, VEC>(a.rows_in, (size_t)p[j] * a.rows_in_stride + (size_t)v * VEC, r[j]);
      }
#pragma unroll
      for (int j = 0; j < G; ++j)
        if (p[j] >= 0) {
          float y[VEC];
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            y[i] = w[j] * x[i];
            if constexpr (DOT) dot[j] = __builtin_fmaf(x[i], r[j][i], dot[j]);
          }
          store_vec<RT, VEC>(a.rows_out, (size_t)p[j] * a.rows_out_stride + (size_t)v * VEC, y);
        }
    }
    if constexpr (DOT) {
      const float s = group_sums<G>(dot, sums);
      if ((int)threadIdx.x < G && j0 + (int)threadIdx.x < a.topk) a.dw[(size_t)t * a.topk + j0 + threadIdx.x] = s;
    }
  }
}

// Rows to token.
template <int XT, int RT, bool DOT>
__global__ __launch_bounds__(kPermWave * 64) void gather_kernel(PermuteArgs a) {
  constexpr int VEC = XT == DT_BF16 && RT == DT_BF16 ? 8 : 4;
  constexpr int G = 8;
  const int n = a.K / VEC, step = gridDim.y * blockDim.x;
  const int v0 = blockIdx.y * blockDim.x + threadIdx.x;
  const int t = blockIdx.x;
  __shared__ float sums[kPermWave][G];
  for (int j0 = 0; j0 < (DOT ? a.topk : 1); j0 += G) {
    float dot[G] = {};
    for (int v = v0; v < n; v += step) {
      float x[VEC], acc[VEC] = {};
      if constexpr (DOT) load_vec<XT, VEC>(a.tok_in, (size_t)t * a.tok_in_stride + (size_t)v * VEC, x);
      // the sum takes all pairs in the first round; the products G pairs a round
      for (int g = j0; g < (j0 ? min(j0 + G, a.topk) : a.topk); g += G) {
        float r[G][VEC];
        int p[G];
#pragma unroll
        for (int j = 0; j < G; ++j) {
          p[j] = g + j < a.topk ? pair_place(a, t * a.topk + g + j) : -1;
          if (p[j] >= 0) load_vec<RT, VEC>(a.rows_in, (size_t)p[j] * a.rows_in_stride + (size_t)v * VEC, r[j]);
        }
#pragma unroll
        for (int j = 0; j < G; ++j)
          if (p[j] >= 0) {
            const float w = a.weights ? a.weights[(size_t)t * a.topk + g + j] : 1.0f;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              acc[i] = __builtin_fmaf(w, r[j][i], acc[i]);
              if constexpr (DOT)
                if (g == j0) dot[j] = __builtin_fmaf(x[i], r[j][i], dot[j]);
            }
          }
      }
      if (j0 == 0) store_vec<XT, VEC>(a.tok_out, (size_t)t * a.tok_out_stride + (size_t)v * VEC, acc);
    }
    if constexpr (DOT) {
      const float s = group_sums<G>(dot, sums);
      if ((int)threadIdx.x < G && j0 + (int)threadIdx.x < a.topk) a.dw[(size_t)t * a.topk + j0 + threadIdx.x] = s;
    }
  }
}

template <bool DOT>
static void* scatter_of(int xt, int rt) {
  if (xt == DT_BF16)
    return rt == DT_BF16 ? (void*)scatter_kernel<DT_BF16, DT_BF16, DOT> : (void*)scatter_kernel<DT_BF16, DT_F32, DOT>;
  return rt == DT_BF16 ? (void*)scatter_kernel<DT_F32, DT_BF16, DOT> : (void*)scatter_kernel<DT_F32, DT_F32, DOT>;
}
template <bool DOT>
static void* gather_of(int xt, int rt) {
  if (xt == DT_BF16)
    return rt == DT_BF16 ? (void*)gather_kernel<DT_BF16, DT_BF16, DOT> : (void*)gather_kernel<DT_BF16, DT_F32, DOT>;
  return rt == DT_BF16 ? (void*)gather_kernel<DT_F32, DT_BF16, DOT> : (void*)gather_kernel<DT_F32, DT_F32, DOT>;
}

int launch_scatter(const PermuteArgs& a, int xt, int rt, hipStream_t st) {
  const int vec = xt == DT_BF16 && rt == DT_BF16 ? 8 : 4, parts = (a.K / vec + 255) / 256;
  const unsigned y = a.dw ? 1 : (unsigned)parts;
  PermuteArgs c = a;
  void* args[] = {&c};
  return (int)hipLaunchKernel(a.dw ? scatter_of<true>(xt, rt) : scatter_of<false>(xt, rt),
                              dim3((unsigned)(a.M + (a.rows + 15) / 16), y), dim3(kPermWave * 64), args, 0, st);
}

int launch_gather(const PermuteArgs& a, int xt, int rt, hipStream_t st) {
  const int vec = xt == DT_BF16 && rt == DT_BF16 ? 8 : 4, parts = (a.K / vec + 255) / 256;
  const unsigned y = a.dw ? 1 : (unsigned)parts;
  PermuteArgs c = a;
  void* args[] = {&c};
  return (int)hipLaunchKernel(a.dw ? gather_of<true>(xt, rt) : gather_of<false>(xt, rt), dim3((unsigned)a.M, y),
                              dim3(kPermWave * 64), args, 0, st);
}

}  // namespace moe
