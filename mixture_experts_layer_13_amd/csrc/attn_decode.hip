// attn_decode.hip -- the few-row attention (attn_decode.hpp) as a launch of its
// own, and the join of the parts that its workgroups leave.
#include "attn_decode.hpp"
#include "launch.hpp"

namespace moe {

template <int DT, int NR, int NS, bool OWN, bool STREAM>
__global__ __launch_bounds__(kDecThreads) void attn_decode_kernel(AttnArgs a) {
  __shared__ __align__(16) DecShared<DT> sh;
  attn_decode_run<DT, NR, NS, OWN, STREAM>(a, blockIdx.x, blockIdx.y, sh);
}

// Joins the parts of the sequence, if any, that began in workgroup blockIdx.x's
// run and went on into the next ones.  One workgroup per row: its lanes find
// the parts' common maximum, groups of DT / 4 lanes add up every GROUPS-th
// part, and LDS joins the groups.  Latency bounds it (4 us, most of it the
// launch and two trips to memory): what follows the header, the parts'
// maxima, sums and first kJoinAhead values of each lane, is loaded at once.
constexpr int kJoinAhead = 4;
template <int DT, int ROWS, int NS>
__global__ __launch_bounds__(kDecThreads) void attn_join_kernel(AttnArgs a) {
  constexpr int LANES = DT / 4, GROUPS = kDecThreads / LANES, ML = kAttnGroups / kDecThreads;
  __shared__ float weight[kAttnGroups];
  __shared__ float red[kDecWaves];
  __shared__ float4 acc[GROUPS][LANES];
  const int w0 = blockIdx.x, h = blockIdx.y, row = blockIdx.z;
  const int2 shared = a.part_seq[h * a.W + w0];
  const int b = shared.x, parts = shared.y;
  if (b < 0) return;
  const size_t slot = (size_t)h * a.W + w0;
  // part k: slot 1 (begins the sequence) of workgroup w0, slot 0 of the later ones
  auto part = [&](int k) { return ((slot + k) * 2 + (k == 0 ? 1 : 0)) * ROWS + row; };
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const Seq s = load_seq(a.b, a.c.lS, b);
  float2 ml[ML];
#pragma unroll
  for (int j = 0; j < ML; ++j) {
    const int k = threadIdx.x + j * kDecThreads;
    ml[j] = k < parts ? *reinterpret_cast<const float2*>(a.part_ml + part(k) * 2) : make_float2(-__builtin_inff(), 0.0f);
  }
  float4 first[kJoinAhead];
#pragma unroll
  for (int j = 0; j < kJoinAhead; ++j) {
    const int k = group + j * GROUPS;
    first[j] = *reinterpret_cast<const float4*>(a.part_o + part(k < parts ? k : 0) * DT + 4 * lane);
  }
  if (row >= s.q * a.G) return;

  float m = ml[0].x;
#pragma unroll
  for (int j = 1; j < ML; ++j) m = __builtin_fmaxf(m, ml[j].x);
  m = wave_max(m);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kDecWaves; ++k) m = __builtin_fmaxf(m, red[k]);
  const float mm = m == -__builtin_inff() ? 0.0f : m;
  float l = 0.0f;
#pragma unroll
  for (int j = 0; j < ML; ++j) {
    const float f = __builtin_amdgcn_exp2f(ml[j].x - mm);
    weight[threadIdx.x + j * kDecThreads] = f;  // 0 past the last part
    l += attn_lower(ml[j].y, mm - ml[j].x);
  }
  l = wave_sum(l);
  __syncthreads();  // weights written, maxima read
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = l;
  float4 o = make_float4(0, 0, 0, 0);
  auto add = [&](float f, const float4& v) {
    o.x += f * v.x;
    o.y += f * v.y;
    o.z += f * v.z;
    o.w += f * v.w;
  };
#pragma unroll
  for (int j = 0; j < kJoinAhead; ++j)
    if (group + j * GROUPS < parts) add(weight[group + j * GROUPS], first[j]);
#pragma unroll 4
  for (int k = group + kJoinAhead * GROUPS; k < parts; k += GROUPS)
    add(weight[k], *reinterpret_cast<const float4*>(a.part_o + part(k) * DT + 4 * lane));
  acc[group][lane] = o;
  __syncthreads();
  if (group != 0 || 4 * lane >= a.c.D) return;
  l = 0.0f;
#pragma unroll
  for (int k = 0; k < kDecWaves; ++k) l += red[k];
  float r[4] = {0, 0, 0, 0};
  for (int k = 0; k < GROUPS; ++k) {
    const float4 v = acc[k][lane];
    r[0] += v.x;
    r[1] += v.y;
    r[2] += v.z;
    r[3] += v.w;
  }
  const int qi = row / a.G;
  const size_t orow = (size_t)(s.q0 + qi) * a.nH + h * a.G + row - qi * a.G;
  attn_store4<NS>(a, orow, 4 * lane, r, l);
  if (lane == 0 && a.lse) a.lse[orow] = attn_lse(m, l);
}

template <int DT, int NR, int NS>
static int join_launch(const AttnArgs& a, hipStream_t st) {
  const int rows = 16 * NR < a.rows ? 16 * NR : a.rows;  // of a sequence, at most
  hipLaunchKernelGGL((attn_join_kernel<DT, 16 * NR, NS>), dim3((unsigned)a.W, (unsigned)a.c.H, (unsigned)rows),
                     dim3(kDecThreads), 0, st, a);
  return (int)hipGetLastError();
}

template <int DT, int NR, int NS>
static int dec_launch(const AttnArgs& a, hipStream_t st) {
  const bool own = (long long)a.b.max_pages << a.c.lS <= (a.b.B >= a.W ? 2 * kDecOwn : kDecOwn);
  const dim3 block(kDecThreads), grid((unsigned)(own ? a.b.B : a.W), (unsigned)a.c.H);
  // 64 sequences of 8192 tokens (1.07 GB): 169 us past the caches, 190 through
  // them; 500 of 500 to 900 (726 MB): 126 and 138; 21 MB in all, which the
  // last-level cache holds: 22.8 and 20.6
  const long long pool = 2LL * a.c.pages * a.c.H * a.c.D << a.c.lS;
  if (own && pool > kCacheBytes)
    hipLaunchKernelGGL((attn_decode_kernel<DT, NR, NS, true, true>), grid, block, 0, st, a);
  else if (own)
    hipLaunchKernelGGL((attn_decode_kernel<DT, NR, NS, true, false>), grid, block, 0, st, a);
  else if (pool > kCacheBytes)
    hipLaunchKernelGGL((attn_decode_kernel<DT, NR, NS, false, true>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((attn_decode_kernel<DT, NR, NS, false, false>), grid, block, 0, st, a);
  const int err = (int)hipGetLastError();
  return err || own ? err : join_launch<DT, NR, NS>(a, st);
}

template <int NS>
static int dec_pick(const AttnArgs& a, int rows, hipStream_t st) {
  if (a.c.D <= 64) {
    if (rows <= 16) return dec_launch<64, 1, NS>(a, st);
    if (rows <= 32) return dec_launch<64, 2, NS>(a, st);
    return dec_launch<64, 4, NS>(a, st);
  }
  if (a.c.D <= 128) return rows <= 16 ? dec_launch<128, 1, NS>(a, st) : dec_launch<128, 2, NS>(a, st);
  return dec_launch<256, 1, NS>(a, st);
}

// 16 NR rows; NR is bounded by the accumulators, NR * DT <= 256.
int attn_decode_rows(int D, int rows) {
  const int most = D <= 64 ? 64 : (D <= 128 ? 32 : 16);
  if (rows > most) return 0;
  return rows <= 16 ? 16 : (rows <= 32 ? 32 : 64);
}

int launch_attn_join16(const AttnArgs& a, bool f32, hipStream_t st) {
  if (a.c.D <= 64) return f32 ? join_launch<64, 1, 3>(a, st) : join_launch<64, 1, 1>(a, st);
  if (a.c.D <= 128) return f32 ? join_launch<128, 1, 3>(a, st) : join_launch<128, 1, 1>(a, st);
  return f32 ? join_launch<256, 1, 3>(a, st) : join_launch<256, 1, 1>(a, st);
}

int launch_attn_decode(const AttnArgs& a, int rows, bool f32, hipStream_t st) {
  return f32 ? dec_pick<3>(a, rows, st) : dec_pick<1>(a, rows, st);
}

}  // namespace moe
