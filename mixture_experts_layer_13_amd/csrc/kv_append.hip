// kv_append.hip -- new keys and values into the paged E4M3 cache, the keys
// rotated on the way (rotate.hpp).
//
// Per touched page and head, over the page's new tokens (keys after the
// rotation, in fp32: rotation and code are one rounding):
//   need = the smallest power of two with 448 need >= max |x|, at least 2^-64;
//   s'   = max(need, s) if earlier tokens of the sequence lie in the page,
//          else need;
//   codes of earlier tokens: E4M3(code * s / s'); new: E4M3(x / s').
// Scales are powers of two, so x / s' is exact, and a page whose scale grows
// is recoded by moving exponents: a code that stays normal keeps all its
// bits, where a scale of amax/448 would round it again with every growth.
// The scale costs no precision for that, E4M3's being relative over 2^14.
// A scale never shrinks while the page is in use, which makes the append of
// the same tokens at the same place the same cache bit for bit.
//
// One workgroup per (page, head) and per keys or values reads its tokens
// once, holds them in registers as fp32, reduces the maximum and stores the
// codes.  Values are stored channel by channel (paged.hpp): through LDS, 16
// bytes of a channel at a time, where a block of 16 tokens is all new; byte by
// byte otherwise, which leaves every other token's bytes alone.
#include "launch.hpp"
#include "paged.hpp"
#include "rotate.hpp"

namespace moe {

constexpr float kMinPageScale = 0x1p-64f;

struct AppendArgs {
  PagedArgs c;
  BatchArgs b;
  const void *k, *v;
  long long ks_t, ks_h, vs_t, vs_h;  // strides in elements
  RotateArgs r;                      // r.half == 0: no rotation
  int units;                         // upper bound of (sequence, page) pairs
};

// The smallest power of two s with 448 s >= amax: 448 = 1.75 * 2^8, so adding
// the distance from 1.75 to 2 carries into the exponent exactly above it.
__device__ __forceinline__ float page_scale(float amax) {
  const uint32_t e = (__float_as_uint(amax) + 0x1fffffu) >> 23;  // 448 * 2^(e - 135)
  return e <= 8u + 63u ? kMinPageScale : __uint_as_float((e - 8u) << 23);
}

// Four codes of y / s (r = 1 / s, exact: s is a power of two).  Saturates;
// a NaN gives a saturated code.
__device__ __forceinline__ uint32_t codes4(const float* y, float r) {
  float q[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) q[j] = __builtin_fminf(__builtin_fmaxf(y[j] * r, -448.0f), 448.0f);
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], v, true);
}

// Four codes times ratio, as codes.
__device__ __forceinline__ uint32_t recode4(uint32_t w, float ratio) {
  const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
  const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  const float y[4] = {lo[0], lo[1], hi[0], hi[1]};
  return codes4(y, ratio);
}

// XT: type of k and v; UPT: units of 16 values per thread.
template <int XT, int THREADS, int UPT>
__global__ __launch_bounds__(THREADS) void kv_append_kernel(AppendArgs a) {
  extern __shared__ __align__(16) uint8_t tile[];  // [S][D] codes of values
  __shared__ int scan[THREADS / 64];
  __shared__ int found[2];
  __shared__ float wmax[THREADS / 64];
  const int S = 1 << a.c.lS, D = a.c.D, h = blockIdx.y;
  const bool vals = blockIdx.z != 0;

  // the workgroup's sequence and page
  int b = blockIdx.x, rank = 0;
  if (a.b.cu_q) {
    if (threadIdx.x == 0) found[0] = -1;
    __syncthreads();
    int before = 0;
    for (int base = 0; base < a.b.B && before <= (int)blockIdx.x; base += THREADS) {
      int n = 0;
      if (base + (int)threadIdx.x < a.b.B) {
        const Seq s = load_seq(a.b, a.c.lS, base + threadIdx.x);
        const int p0 = s.kv - s.q > 0 ? s.kv - s.q : 0;
        if (s.q > 0 && s.lim > p0) n = ((s.lim - 1) >> a.c.lS) - (p0 >> a.c.lS) + 1;
      }
      int total;
      const int end = before + block_scan<THREADS>(n, scan, &total);
      if ((int)blockIdx.x >= end - n && (int)blockIdx.x < end) {
        found[0] = base + threadIdx.x;
        found[1] = blockIdx.x - (end - n);
      }
      before += total;
    }
    __syncthreads();
    b = found[0];
    rank = found[1];
    if (b < 0) return;
  }
  const Seq s = load_seq(a.b, a.c.lS, b);
  const int start = s.kv - s.q;  // token of the sequence's first row; rows of negative tokens are not kept
  const int p0 = start > 0 ? start : 0;
  if (s.q == 0 || s.lim <= p0) return;
  const int pg = (p0 >> a.c.lS) + rank;
  const int lo = p0 > (pg << a.c.lS) ? p0 : pg << a.c.lS;
  const int hi = s.lim < ((pg + 1) << a.c.lS) ? s.lim : (pg + 1) << a.c.lS;
  const int old = lo & (S - 1);  // earlier tokens in the page
  const int page = a.b.table[(size_t)b * a.b.max_pages + pg];
  if ((unsigned)page >= (unsigned)a.c.pages) return;
  const int row0 = s.q0 + lo - start, n = hi - lo;

  // the new tokens, in fp32
  const int upd = D >> 4, units = n * upd;
  const void* src = vals ? a.v : a.k;
  const long long st = vals ? a.vs_t : a.ks_t, sh = vals ? a.vs_h : a.ks_h;
  const int half = vals ? 0 : a.r.half;
  float x[UPT][16];
  float amax = 0.0f;
#pragma unroll
  for (int j = 0; j < UPT; ++j) {
    const int u = j * THREADS + threadIdx.x;
    if (u >= units) continue;
    const int tok = u / upd, g = u - tok * upd;
    int p, q;
    unit_groups(g, half, a.r.interleaved, p, q);
    const size_t base = (size_t)(row0 + tok) * st + (size_t)h * sh;
    i32x4 raw[4];
    load8<XT>(src, base + p, raw);
    load8<XT>(src, base + q, raw + 2);
    unpack8<XT>(raw, x[j]);
    unpack8<XT>(raw + 2, x[j] + 8);
    if (g < (half >> 3)) {
      float2 cs[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int pr = 8 * g + i, ax = rotate_axis(a.r, pr);
        double turns = 0.0;
        if (ax >= 0) {
          const int pos = a.r.pos ? a.r.pos[(size_t)ax * a.r.T + row0 + tok] : lo + tok;
          turns = (double)pos * (double)a.r.inv_freq[pr] * kInvTwoPi;
        }
        cs[i] = rotate_cs(turns, a.r.inverse);
      }
      rotate_unit(x[j], x[j] + 8, cs, a.r.interleaved);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float m = __builtin_fabsf(x[j][i]);
      amax = __builtin_fmaxf(amax, m < __builtin_inff() ? m : 0.0f);
    }
  }
  amax = wave_max(amax);
  if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) amax = __builtin_fmaxf(amax, wmax[w]);

  float* scale = (vals ? a.c.vs : a.c.ks) + (size_t)page * a.c.H + h;
  uint8_t* codes = (vals ? a.c.vc : a.c.kc) + ((size_t)page * a.c.H + h) * ((size_t)D << a.c.lS);
  const float was = old > 0 ? *scale : 0.0f;
  const float need = page_scale(amax);
  const float now = was > need ? was : need;
  const float rcp = 1.0f / now;
  if (old > 0 && now != was) {
    // recode what was there: whole 16-byte groups of keys; of values, the
    // bytes of earlier tokens (bytes past them go back unchanged, before the
    // new ones are stored)
    const float ratio = was / now;
    const int groups = vals ? ((old + 15) >> 4) * D : (old * D) >> 4;
    for (int i = threadIdx.x; i < groups; i += THREADS) {
      uint4 w = *reinterpret_cast<uint4*>(codes + 16 * (size_t)i);
      uint32_t* c = reinterpret_cast<uint32_t*>(&w);
      const int keep = vals ? old - 16 * (i / D) : 16;  // bytes of earlier tokens
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = keep - 4 * j;
        const uint32_t mask = k >= 4 ? 0xffffffffu : (k <= 0 ? 0u : (1u << (8 * k)) - 1u);
        c[j] = (recode4(c[j], ratio) & mask) | (c[j] & ~mask);
      }
      *reinterpret_cast<uint4*>(codes + 16 * (size_t)i) = w;
    }
  }
  __syncthreads();  // every thread has read *scale; recoded bytes are stored
  if (threadIdx.x == 0) *scale = now;

#pragma unroll
  for (int j = 0; j < UPT; ++j) {
    const int u = j * THREADS + threadIdx.x;
    if (u >= units) continue;
    const int tok = u / upd, g = u - tok * upd;
    int p, q;
    unit_groups(g, half, a.r.interleaved, p, q);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = codes4(x[j] + 4 * i, rcp);
    uint8_t* row = (vals ? tile + (size_t)tok * D : codes + (size_t)(old + tok) * D);
    *reinterpret_cast<uint2*>(row + p) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2*>(row + q) = make_uint2(w[2], w[3]);
  }
  if (!vals) return;
  __syncthreads();
  // values: one 16-byte group (block of 16 tokens, channel) per thread and step
  const int blk0 = old >> 4, blks = ((old + n - 1) >> 4) - blk0 + 1;
  for (int i = threadIdx.x; i < blks * D; i += THREADS) {
    const int blk = blk0 + i / D, d = i % D;
    uint8_t* to = codes + ((size_t)blk * D + d) * 16;
    const int t0 = 16 * blk - old;  // first token of the block, among the new ones
    if (t0 >= 0 && t0 + 16 <= n) {
      uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < 16; ++k) w[k >> 2] |= (uint32_t)tile[(size_t)(t0 + k) * D + d] << (8 * (k & 3));
      *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      for (int k = t0 < 0 ? -t0 : 0; k < 16 && t0 + k < n; ++k) to[k] = tile[(size_t)(t0 + k) * D + d];
    }
  }
}

template <int XT, int THREADS, int UPT>
static int append_launch(const AppendArgs& a, int rows, hipStream_t st) {
  const size_t lds = (size_t)rows * a.c.D;  // at most 32 KB
  hipLaunchKernelGGL((kv_append_kernel<XT, THREADS, UPT>), dim3((unsigned)a.units, (unsigned)a.c.H, 2), dim3(THREADS),
                     lds, st, a);
  return (int)hipGetLastError();
}

template <int XT>
static int append_pick(const AppendArgs& a, hipStream_t st) {
  const int S = 1 << a.c.lS;
  const int rows = a.b.cu_q ? S : 1;  // new tokens of a page, at most
  const int units = rows * (a.c.D / 16);
  if (units <= 64) return append_launch<XT, 64, 1>(a, rows, st);
  if (units <= 256) return append_launch<XT, 256, 1>(a, rows, st);
  if (units <= 512) return append_launch<XT, 256, 2>(a, rows, st);
  if (units <= 1024) return append_launch<XT, 512, 2>(a, rows, st);
  return append_launch<XT, 1024, 2>(a, rows, st);  // S <= 128, D <= 256: at most 2048 units
}

int launch_kv_append(const PagedArgs& c, const BatchArgs& b, const void* k, long long ks_t, long long ks_h,
                     const void* v, long long vs_t, long long vs_h, int xt, const RotateArgs& r,
                     hipStream_t st) {
  AppendArgs a{};
  a.c = c;
  a.b = b;
  a.k = k;
  a.v = v;
  a.ks_t = ks_t;
  a.ks_h = ks_h;
  a.vs_t = vs_t;
  a.vs_h = vs_h;
  a.r = r;
  // q tokens in a row touch at most (q - 2) / S + 2 pages
  a.units = b.cu_q ? (b.T >> c.lS) + 2 * (b.B < b.T ? b.B : b.T) : b.B;
  return xt == DT_BF16 ? append_pick<DT_BF16>(a, st) : append_pick<DT_F32>(a, st);
}

}  // namespace moe
