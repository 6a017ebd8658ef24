// rope_axes.hip -- rotary positions with several axes (time, height, width):
// out[t, h, :] = x[t, h, :] with pair i turned by the angle of the position
// axis that pair_axis names (rotate.hpp); values from rotary_dim on pass
// through.  x and out have strides of their own, so a head range of a fused
// projection is rotated where it lies, and out may be x.
//
// Bytes bound it: x is read and out written once.  A workgroup takes `tb`
// tokens; its threads issue the loads of up to kUnits units of 16 values
// each, compute the tokens' angles into LDS while these are in flight (one
// fp64 product and one sincospi per token and pair, shared by every head),
// and after one barrier rotate and store.  Each thread reads both halves of
// its pairs before it writes them, which is what allows out == x.
#include "launch.hpp"
#include "rotate.hpp"

namespace moe {

constexpr int kRaThreads = 256;
constexpr int kRaUnits = 4;           // units of 16 values a thread holds at once
constexpr int kRaMaxAngles = 4096;    // LDS: {cos, sin} of at most this many (token, pair)

struct RopeAxesArgs {
  const void* x;
  void* out;
  long long xs_t, xs_h, os_t, os_h;  // strides in elements
  int T, nH, D, tb;
  RotateArgs r;
};

template <int OT>
__device__ __forceinline__ void store8(void* base, size_t idx, const float v[8]) {
  if (OT == DT_BF16) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(base) + idx) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    float* p = reinterpret_cast<float*>(base) + idx;
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
  }
}

template <int XT, int OT>
__global__ __launch_bounds__(kRaThreads) void rope_axes_kernel(RopeAxesArgs a) {
  __shared__ float2 cs[kRaMaxAngles];
  const int t0 = blockIdx.x * a.tb;
  const int tn = a.T - t0 < a.tb ? a.T - t0 : a.tb;
  const int upd = a.D >> 4, upt = a.nH * upd, units = tn * upt;
  for (int base = 0; base < units; base += kRaThreads * kRaUnits) {
    i32x4 raw[kRaUnits][4];
    int tok[kRaUnits], hd[kRaUnits], gs[kRaUnits];
#pragma unroll
    for (int s = 0; s < kRaUnits; ++s) {
      const int u = base + s * kRaThreads + threadIdx.x;
      const int uu = u < units ? u : 0;
      tok[s] = uu / upt;
      const int r = uu - tok[s] * upt;
      hd[s] = r / upd;
      gs[s] = r - hd[s] * upd;
      int p, q;
      unit_groups(gs[s], a.r.half, a.r.interleaved, p, q);
      const size_t row = (size_t)(t0 + tok[s]) * a.xs_t + (size_t)hd[s] * a.xs_h;
      load8<XT>(a.x, row + p, raw[s]);
      load8<XT>(a.x, row + q, raw[s] + 2);
    }
    if (base == 0) {
      for (int i = threadIdx.x; i < tn * a.r.half; i += kRaThreads) {
        const int t = i / a.r.half, pr = i - t * a.r.half, ax = rotate_axis(a.r, pr);
        double turns = 0.0;
        if (ax >= 0)
          turns = (double)a.r.pos[(size_t)ax * a.r.T + t0 + t] * (double)a.r.inv_freq[pr] * kInvTwoPi;
        cs[i] = rotate_cs(turns, a.r.inverse);
      }
      __syncthreads();
    }
#pragma unroll
    for (int s = 0; s < kRaUnits; ++s) {
      if (base + s * kRaThreads + (int)threadIdx.x >= units) continue;
      float va[8], vb[8];
      unpack8<XT>(raw[s], va);
      unpack8<XT>(raw[s] + 2, vb);
      if (gs[s] < (a.r.half >> 3)) rotate_unit(va, vb, cs + tok[s] * a.r.half + 8 * gs[s], a.r.interleaved);
      int p, q;
      unit_groups(gs[s], a.r.half, a.r.interleaved, p, q);
      const size_t row = (size_t)(t0 + tok[s]) * a.os_t + (size_t)hd[s] * a.os_h;
      store8<OT>(a.out, row + p, va);
      store8<OT>(a.out, row + q, vb);
    }
  }
}

int launch_rope_axes(const void* x, int xt, long long xs_t, long long xs_h, const int32_t* pos, int axes,
                     const int32_t* pair_axis, const float* inv_freq, int T, int nH, int D, int R,
                     int interleaved, int inverse, void* out, int ot, long long os_t, long long os_h,
                     hipStream_t st) {
  RopeAxesArgs a{};
  a.x = x;
  a.out = out;
  a.xs_t = xs_t;
  a.xs_h = xs_h;
  a.os_t = os_t;
  a.os_h = os_h;
  a.T = T;
  a.nH = nH;
  a.D = D;
  a.r = RotateArgs{pos, pair_axis, inv_freq, T, axes, R / 2, interleaved, inverse};
  // tokens per workgroup: enough units for its threads, unless that would
  // leave compute units without a workgroup
  const int upt = nH * (D / 16);
  int tb = 1;
  while (tb < 64 && 2 * tb * upt <= kRaThreads * kRaUnits && 2 * tb * (R / 2) <= kRaMaxAngles &&
         (T + 2 * tb - 1) / (2 * tb) >= 2 * device_cu_count())
    tb *= 2;
  a.tb = tb;
  const dim3 grid((unsigned)((T + tb - 1) / tb)), block(kRaThreads);
  if (xt == DT_BF16 && ot == DT_BF16)
    hipLaunchKernelGGL((rope_axes_kernel<DT_BF16, DT_BF16>), grid, block, 0, st, a);
  else if (xt == DT_BF16)
    hipLaunchKernelGGL((rope_axes_kernel<DT_BF16, DT_F32>), grid, block, 0, st, a);
  else if (ot == DT_BF16)
    hipLaunchKernelGGL((rope_axes_kernel<DT_F32, DT_BF16>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((rope_axes_kernel<DT_F32, DT_F32>), grid, block, 0, st, a);
  return (int)hipGetLastError();
}

}  // namespace moe
