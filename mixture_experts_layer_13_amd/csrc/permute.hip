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
//
// Bytes bound all of them (a large copy: 5.07 TB/s): 8192 tokens x 4096 bf16 top-8
// dispatch 135 us (5.0), combine 119 (5.1), dispatch's gradient 134 (5.0), combine's
// 246 (4.9, as many writes as reads); one pair in eight kept, 8192 x 7168, combine
// 36 (6.5, mostly reads); 64 tokens 3.4 to 6.9, launch and two loads in a row.
#include "common.hpp"
#include "launch.hpp"
#include "permute.hpp"

namespace moe {

constexpr int kPermWaves = 8;  // most waves of a workgroup
constexpr int kPairs = 8;      // pairs whose rows a thread has in flight

// VEC consecutive values of a row as they lie in memory, at most 16 bytes.
template <int DT, int VEC>
struct Raw8 {
  static constexpr int kWords = VEC * (DT == DT_F32 ? 4 : 2) / 4;
  uint32_t d[kWords];
  __device__ __forceinline__ void load(const void* base, size_t at) {
    const char* p = reinterpret_cast<const char*>(base) + at * (DT == DT_F32 ? 4 : 2);
    if constexpr (kWords == 4) {
      const i32x4 r = ld16(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = (uint32_t)r[i];
    } else {
      const uint2 r = *reinterpret_cast<const uint2*>(p);
      d[0] = r.x;
      d[1] = r.y;
    }
  }
  __device__ __forceinline__ float value(int i) const {
    if constexpr (DT == DT_F32) return __uint_as_float(d[i]);
    return __uint_as_float(i & 1 ? d[i / 2] & 0xffff0000u : d[i / 2] << 16);
  }
};

template <int DT, int VEC>
__device__ __forceinline__ void store_vec(void* base, size_t at, const float (&v)[VEC]) {
  if constexpr (DT == DT_F32) {
    static_assert(VEC == 4, "16 bytes");
    st16(reinterpret_cast<float*>(base) + at,
         i32x4{__float_as_int(v[0]), __float_as_int(v[1]), __float_as_int(v[2]), __float_as_int(v[3])});
  } else {
    uint16_t* p = reinterpret_cast<uint16_t*>(base) + at;
    if constexpr (VEC == 8)
      st16(p, i32x4{(int)pack_bf16x2(v[0], v[1]), (int)pack_bf16x2(v[2], v[3]), (int)pack_bf16x2(v[4], v[5]),
                    (int)pack_bf16x2(v[6], v[7])});
    else
      *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  }
}

// Places and weights of the pairs j0 .. j0 + kPairs - 1 of token t; -1: none.
struct Places {
  int p[kPairs];
  float w[kPairs];
  __device__ __forceinline__ Places(const PermuteArgs& a, int t, int j0) {
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      const size_t f = (size_t)t * a.topk + min(j0 + j, a.topk - 1);
      const int at = a.pair_pos[f];
      p[j] = j0 + j < a.topk && at >= 0 && at < a.rows ? at : -1;
      w[j] = a.weights ? a.weights[f] : 1.0f;
    }
  }
};

// The workgroup's sums of dot, to the pairs j0 .. of token t.  A wave's eight sums
// take ten exchanges: lanes 32, 16 and 8 apart first deal the values out among
// each other, then those of one value meet (48 if each were summed by itself).
__device__ __forceinline__ void store_dots(const PermuteArgs& a, int t, int j0, const float (&dot)[kPairs]) {
  static_assert(kPairs == 8, "three halvings");
  __shared__ float part[kPermWaves][kPairs];
  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  float v[kPairs];
#pragma unroll
  for (int j = 0; j < kPairs; ++j) v[j] = dot[j];
#pragma unroll
  for (int n = kPairs / 2, m = 32; n > 0; n /= 2, m /= 2)
#pragma unroll
    for (int j = 0; j < n; ++j) {
      const float keep = lane & m ? v[j + n] : v[j], give = lane & m ? v[j] : v[j + n];
      v[j] = keep + __shfl_xor(give, m, kWave);
    }
#pragma unroll
  for (int m = 4; m > 0; m /= 2) v[0] += __shfl_xor(v[0], m, kWave);
  if ((lane & 7) == 0) part[threadIdx.x >> 6][lane >> 3] = v[0];  // bits 5, 4, 3 of the lane: 4, 2, 1 of the pair
  __syncthreads();
  if ((int)threadIdx.x < min(kPairs, a.topk - j0)) {
    float s = 0.0f;
    for (int q = 0; q < waves; ++q) s += part[q][threadIdx.x];
    a.dw[(size_t)t * a.topk + j0 + threadIdx.x] = s;
  }
  __syncthreads();
}

template <int XT, int RT>
constexpr int perm_vec() {
  return XT == DT_BF16 && RT == DT_BF16 ? 8 : 4;
}

// Token to rows.  Workgroups below M: token blockIdx.x (the vectors of part
// blockIdx.y); the others zero the rows of no pair among 32.
template <int XT, int RT, bool DOT>
__global__ __launch_bounds__(kPermWaves * 64) void scatter_kernel(PermuteArgs a) {
  constexpr int VEC = perm_vec<XT, RT>();
  const int n = a.K / VEC, step = gridDim.y * blockDim.x;
  const int v0 = blockIdx.y * blockDim.x + threadIdx.x;
  if ((int)blockIdx.x >= a.M) {
    const int r0 = ((int)blockIdx.x - a.M) * 32, l = threadIdx.x & 31;
    const int end = min(a.rows, *a.num_padded);
    const int f = r0 + l < end ? a.sorted_ids[r0 + l] : 0;
    uint32_t empty = (uint32_t)__ballot(r0 + l < end && !(f >= 0 && f < a.P));
    const float z[VEC] = {};
    for (; empty; empty &= empty - 1) {
      const size_t r = r0 + __builtin_ctz(empty);
      for (int v = v0; v < n; v += step) store_vec<RT, VEC>(a.rows_out, r * a.rows_out_stride + (size_t)v * VEC, z);
    }
    return;
  }
  const int t = blockIdx.x;
  for (int j0 = 0; j0 < a.topk; j0 += kPairs) {
    const Places at(a, t, j0);
    float dot[kPairs] = {};
    for (int v = v0; v < n; v += step) {
      Raw8<XT, VEC> x;
      x.load(a.tok_in, (size_t)t * a.tok_in_stride + (size_t)v * VEC);
      Raw8<RT, VEC> r[DOT ? kPairs : 1];
      if constexpr (DOT) {
#pragma unroll
        for (int j = 0; j < kPairs; ++j)
          if (at.p[j] >= 0) r[j].load(a.rows_in, (size_t)at.p[j] * a.rows_in_stride + (size_t)v * VEC);
      }
#pragma unroll
      for (int j = 0; j < kPairs; ++j)
        if (at.p[j] >= 0) {
          float y[VEC];
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            y[i] = at.w[j] * x.value(i);
            if constexpr (DOT) dot[j] = __builtin_fmaf(x.value(i), r[j].value(i), dot[j]);
          }
          store_vec<RT, VEC>(a.rows_out, (size_t)at.p[j] * a.rows_out_stride + (size_t)v * VEC, y);
        }
    }
    if constexpr (DOT) store_dots(a, t, j0, dot);
  }
}

// Rows to token.  The token's pairs that have a place are listed first (of a rank's
// experts few are left), and their rows loaded four at a time for two vectors a
// thread, whatever topk is.
constexpr int kListed = 4;

template <int XT, int RT>
__global__ __launch_bounds__(kPermWaves * 64) void gather_kernel(PermuteArgs a) {
  constexpr int VEC = perm_vec<XT, RT>();
  __shared__ int place[64];
  __shared__ float weight[64];
  const int n = a.K / VEC, step = gridDim.y * blockDim.x;
  const int v0 = blockIdx.y * blockDim.x + threadIdx.x;
  const int t = blockIdx.x;
  int kept;
  {
    const int lane = threadIdx.x & 63;
    const size_t f = (size_t)t * a.topk + min(lane, a.topk - 1);
    const int p = a.pair_pos[f];
    const float w = a.weights ? a.weights[f] : 1.0f;
    const bool has = lane < a.topk && p >= 0 && p < a.rows;
    const uint64_t all = __ballot(has);
    kept = __popcll(all);
    if (has && threadIdx.x < 64) {
      const int at = __popcll(all & lanemask_lt(lane));
      place[at] = p;
      weight[at] = w;
    }
  }
  __syncthreads();
  for (int v = v0; v < n; v += 2 * step) {
    const int w = min(v + step, n - 1);  // the second vector, or one that is not stored
    float acc[2][VEC] = {};
    for (int i = 0; i < kept; i += kListed) {
      Raw8<RT, VEC> r[kListed][2];
      float wt[kListed];
#pragma unroll
      for (int q = 0; q < kListed; ++q) {
        const int at = min(i + q, kept - 1);
        const size_t row = (size_t)__builtin_amdgcn_readfirstlane(place[at]) * a.rows_in_stride;
        wt[q] = weight[at];
        if (i + q < kept) {
          r[q][0].load(a.rows_in, row + (size_t)v * VEC);
          r[q][1].load(a.rows_in, row + (size_t)w * VEC);
        }
      }
#pragma unroll
      for (int q = 0; q < kListed; ++q)
        if (i + q < kept)
#pragma unroll
          for (int c = 0; c < VEC; ++c) {
            acc[0][c] = __builtin_fmaf(wt[q], r[q][0].value(c), acc[0][c]);
            acc[1][c] = __builtin_fmaf(wt[q], r[q][1].value(c), acc[1][c]);
          }
    }
    store_vec<XT, VEC>(a.tok_out, (size_t)t * a.tok_out_stride + (size_t)v * VEC, acc[0]);
    if (v + step < n) store_vec<XT, VEC>(a.tok_out, (size_t)t * a.tok_out_stride + (size_t)w * VEC, acc[1]);
  }
}

// The same with the products for the weights' gradient.
template <int XT, int RT>
__global__ __launch_bounds__(kPermWaves * 64) void gather_dot_kernel(PermuteArgs a) {
  constexpr int VEC = perm_vec<XT, RT>();
  const int n = a.K / VEC, step = blockDim.x, t = blockIdx.x;
  // acc += the rows of `at` at vector v, dot += their products with x
  auto take = [&](const Places& at, int v, float (&acc)[VEC], bool products, float (&dot)[kPairs]) {
    Raw8<RT, VEC> r[kPairs];
    Raw8<XT, VEC> x;
    if (products) x.load(a.tok_in, (size_t)t * a.tok_in_stride + (size_t)v * VEC);
#pragma unroll
    for (int j = 0; j < kPairs; ++j)
      if (at.p[j] >= 0) r[j].load(a.rows_in, (size_t)at.p[j] * a.rows_in_stride + (size_t)v * VEC);
#pragma unroll
    for (int j = 0; j < kPairs; ++j)
      if (at.p[j] >= 0) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          acc[i] = __builtin_fmaf(at.w[j], r[j].value(i), acc[i]);
          if (products) dot[j] = __builtin_fmaf(x.value(i), r[j].value(i), dot[j]);
        }
      }
  };
  const Places first(a, t, 0);
  float dot[kPairs] = {}, unused[kPairs];
  for (int v = threadIdx.x; v < n; v += step) {
    float acc[VEC] = {};
    take(first, v, acc, true, dot);
    for (int j0 = kPairs; j0 < a.topk; j0 += kPairs) take(Places(a, t, j0), v, acc, false, unused);
    store_vec<XT, VEC>(a.tok_out, (size_t)t * a.tok_out_stride + (size_t)v * VEC, acc);
  }
  store_dots(a, t, 0, dot);
  for (int j0 = kPairs; j0 < a.topk; j0 += kPairs) {
    const Places at(a, t, j0);
    float more[kPairs] = {}, acc[VEC] = {};
    for (int v = threadIdx.x; v < n; v += step) take(at, v, acc, true, more);
    store_dots(a, t, j0, more);
  }
}

template <bool DOT>
static void* scatter_of(int xt, int rt) {
  if (xt == DT_BF16)
    return rt == DT_BF16 ? (void*)scatter_kernel<DT_BF16, DT_BF16, DOT> : (void*)scatter_kernel<DT_BF16, DT_F32, DOT>;
  return rt == DT_BF16 ? (void*)scatter_kernel<DT_F32, DT_BF16, DOT> : (void*)scatter_kernel<DT_F32, DT_F32, DOT>;
}
static void* gather_of(int xt, int rt) {
  if (xt == DT_BF16)
    return rt == DT_BF16 ? (void*)gather_kernel<DT_BF16, DT_BF16> : (void*)gather_kernel<DT_BF16, DT_F32>;
  return rt == DT_BF16 ? (void*)gather_kernel<DT_F32, DT_BF16> : (void*)gather_kernel<DT_F32, DT_F32>;
}
static void* gather_dot_of(int xt, int rt) {
  if (xt == DT_BF16)
    return rt == DT_BF16 ? (void*)gather_dot_kernel<DT_BF16, DT_BF16> : (void*)gather_dot_kernel<DT_BF16, DT_F32>;
  return rt == DT_BF16 ? (void*)gather_dot_kernel<DT_F32, DT_BF16> : (void*)gather_dot_kernel<DT_F32, DT_F32>;
}

// A token's vectors, `each` to a thread, over as few rounds of a workgroup of up to
// eight waves as will do; of few tokens without products, each wave's over a
// workgroup of its own.
static int permute_launch(const void* kernel, const PermuteArgs& a, int xt, int rt, int each, long long groups,
                          hipStream_t st) {
  const int vec = xt == DT_BF16 && rt == DT_BF16 ? 8 : 4;
  const int chunks = (a.K / vec + 63) / 64, rounds = (chunks + each * kPermWaves - 1) / (each * kPermWaves);
  int waves = (chunks + rounds * each - 1) / (rounds * each), parts = 1;
  if (!a.dw && (long long)a.M * waves < 4 * device_cu_count()) {
    parts = chunks;
    waves = 1;
  }
  PermuteArgs c = a;
  void* args[] = {&c};
  return (int)hipLaunchKernel(kernel, dim3((unsigned)groups, (unsigned)parts), dim3(waves * 64), args, 0, st);
}

// One vector a thread where its pairs' rows are many, two where they are few: smaller
// workgroups, of which more fit.  us with one | two: dispatch backward of 8192 tokens
// x 4096 bf16 topk 1 54.5 | 33.4, 3 69.5 | 59.8, 8 128.8 | 132.7; of 5003 x 1032 fp32
// topk 3 26.3 | 20.1; combine backward of 16384 x 2048 bf16 topk 1 76.8 | 49.9, 3
// 116.8 | 96.7, 8 213.6 | 227.4; dispatch of 16384 x 4096 bf16 topk 1 84.7 | 54.9, 3
// 140.0 | 106.9.
static int vectors_each(const PermuteArgs& a) { return a.topk <= 4 ? 2 : 1; }

int launch_scatter(const PermuteArgs& a, int xt, int rt, hipStream_t st) {
  return permute_launch(a.dw ? scatter_of<true>(xt, rt) : scatter_of<false>(xt, rt), a, xt, rt, vectors_each(a),
                        a.M + ((long long)a.rows + 31) / 32, st);
}

int launch_gather(const PermuteArgs& a, int xt, int rt, hipStream_t st) {
  return permute_launch(a.dw ? gather_dot_of(xt, rt) : gather_of(xt, rt), a, xt, rt, a.dw ? vectors_each(a) : 2, a.M,
                        st);
}

}  // namespace moe
