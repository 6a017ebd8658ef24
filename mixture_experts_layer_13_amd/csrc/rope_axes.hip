// rope_axes.hip -- rotary positions with several axes (time, height, width):
// out[t, h, :] = x[t, h, :] with pair i turned by the angle of the position
// axis that pair_axis names (rotate.hpp); values from rotary_dim on pass
// through.  x and out have strides of their own, so a head range of a fused
// projection is rotated where it lies, and out may be x.
//
// Bytes bound it: x is read and out written once.  A workgroup takes `tb`
// tokens; its threads issue the loads of up to kRaUnits pairs of 16-byte
// vectors each, compute the tokens' angles into LDS while these are in flight
// (once per token and pair, for every head), and after one barrier rotate and
// store.  Each thread reads both halves of its pairs before it writes them,
// which is what allows out == x.
// Measured: 8192 tokens, 32 heads of 128, bf16, three axes (134 MB): 27.6 us,
// 4.87 TB/s, a copy's rate (5.43) less the launch; 4099 x 20 x 80, f32, 64
// turned, interleaved (52 MB): 11.3 us, 4.6 TB/s, with angles per head instead
// of per token 20; 64 tokens: 3.8 us, the launch and two trips to memory.
#include "launch.hpp"
#include "rotate.hpp"

namespace moe {

constexpr int kRaThreads = 256;
constexpr int kRaUnits = 4;           // pairs of vectors a thread holds at once
constexpr int kRaMaxGrid = 1 << 20;   // workgroups of a launch; each takes every kRaMaxGrid-th run of tokens
constexpr int kRaMaxAngles = 4096;    // LDS: {cos, sin} of at most this many (token, pair)

struct RopeAxesArgs {
  const void* x;
  void* out;
  long long xs_t, xs_h, os_t, os_h;  // strides in elements
  int T, nH, D, tb;
  RotateArgs r;
};

template <int OT, int E>
__device__ __forceinline__ void store_vec(void* base, size_t idx, const float* v) {
  if (OT == DT_BF16) {
    uint32_t w[E / 2];
#pragma unroll
    for (int j = 0; j < E / 2; ++j) w[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
    uint16_t* p = reinterpret_cast<uint16_t*>(base) + idx;
    if (E == 8)
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[E / 2 - 2], w[E / 2 - 1]);
    else
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int j = 0; j < E; j += 4)
      *reinterpret_cast<float4*>(reinterpret_cast<float*>(base) + idx + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
  }
}

template <int XT, int OT>
__global__ __launch_bounds__(kRaThreads) void rope_axes_kernel(RopeAxesArgs a) {
  __shared__ float2 cs[kRaMaxAngles];
  constexpr int E = XT == DT_BF16 ? 8 : 4;  // values of a 16-byte load
  const int upd = a.D / (2 * E), upt = a.nH * upd;
  for (long long t0 = (long long)blockIdx.x * a.tb; t0 < a.T; t0 += (long long)gridDim.x * a.tb) {
    const int tn = a.T - t0 < a.tb ? (int)(a.T - t0) : a.tb, units = tn * upt;
    for (int base = 0; base < units; base += kRaThreads * kRaUnits) {
      RawVec<XT, E> ra[kRaUnits], rb[kRaUnits];
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
        unit_groups<E>(gs[s], a.r.half, a.D, p, q);
        const size_t row = (size_t)(t0 + tok[s]) * a.xs_t + (size_t)hd[s] * a.xs_h;
        ra[s] = load_vec<XT, E>(a.x, row + p);
        rb[s] = load_vec<XT, E>(a.x, row + q);
      }
      if (base == 0) {
        // a thread keeps one pair, and takes every `together`-th token
        const int together = kRaThreads / a.r.half, t1 = (int)threadIdx.x / a.r.half, pr = (int)threadIdx.x - t1 * a.r.half;
        if (t1 < together) {
          const int ax = rotate_axis(a.r, pr);
          const TurnFreq f = turn_freq(a.r.inv_freq[pr]);
          for (int t = t1; t < tn; t += together)
            cs[t * a.r.half + pr] =
                rotate_cs(place_of(ax >= 0 ? a.r.pos[(size_t)ax * a.r.T + t0 + t] : 0, a.r.inverse), f);
        }
        __syncthreads();
      }
#pragma unroll
      for (int s = 0; s < kRaUnits; ++s) {
        if (base + s * kRaThreads + (int)threadIdx.x >= units) continue;
        float va[E], vb[E];
        unpack_vec(ra[s], va);
        unpack_vec(rb[s], vb);
        if (gs[s] < a.r.half / E) {
          float2 w[E];
#pragma unroll
          for (int i = 0; i < E; ++i) w[i] = cs[tok[s] * a.r.half + unit_pair<E>(gs[s], i, a.r.half, a.r.interleaved)];
          rotate_unit<E>(va, vb, w, a.r.interleaved);
        }
        int p, q;
        unit_groups<E>(gs[s], a.r.half, a.D, p, q);
        const size_t row = (size_t)(t0 + tok[s]) * a.os_t + (size_t)hd[s] * a.os_h;
        store_vec<OT, E>(a.out, row + p, va);
        store_vec<OT, E>(a.out, row + q, vb);
      }
    }
    __syncthreads();  // the angles are read
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
  const int upt = nH * (D / (xt == DT_BF16 ? 16 : 8));
  int tb = 1;
  while (tb < 64 && 2 * tb * upt <= kRaThreads * kRaUnits && 2 * tb * (R / 2) <= kRaMaxAngles &&
         (T + 2 * tb - 1) / (2 * tb) >= 2 * device_cu_count())
    tb *= 2;
  a.tb = tb;
  const long long groups = ((long long)T + tb - 1) / tb;
  const dim3 grid((unsigned)(groups < kRaMaxGrid ? groups : kRaMaxGrid)), block(kRaThreads);
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
