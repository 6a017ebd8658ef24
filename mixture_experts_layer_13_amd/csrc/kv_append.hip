// kv_append.hip -- new keys and values into the paged E4M3 cache, the keys
// rotated on the way (rotate.hpp).
//
// Per touched page and head, over the page's new tokens (keys after the
// rotation, in fp32: rotation and code are one rounding):
//   need = the smallest power of two with 448 need >= max |x|, kept within
//          2^-64 and 2^48, so that the attention's sums of codes, scales and
//          probabilities stay in fp32's range (values past 1.2e17 saturate);
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
// A workgroup takes one touched page and head, keys and values.  It reads its
// tokens once, 16 values per thread and unit, with every load in flight before
// the first is used, rotates keys in registers (a thread owns whole pairs),
// reduces the maxima and stores the codes.  Values are stored channel by
// channel (paged.hpp): through LDS, four channels by 16 tokens at a time
// transposed with byte permutes, where a block of 16 tokens is all new; byte by
// byte otherwise, which leaves every other token's bytes alone.
// Frequencies are made once per workgroup, by one thread each, while the tokens
// are on their way.
// Measured, page 64, 8 heads of 128, bf16: 65536 tokens at 4.6 TB/s (a copy:
// 5.43), bytes and the conversions' VALU together; 8192 tokens (50 MB) in
// 15.5 us, since its 1032 workgroups are all resident at once and load, then
// store, in step; one token of each of 64 sequences in 5 us, a chain of table,
// token, barrier and store.  Keys and values in workgroups of their own take
// 19 to 21 us for the 8192 tokens, a workgroup over all heads 26.
#include "launch.hpp"
#include "paged.hpp"
#include "rotate.hpp"

namespace moe {

constexpr int kAppendThreads = 1024;

struct AppendArgs {
  PagedArgs c;
  BatchArgs b;
  const void *k, *v;
  long long ks_t, ks_h, vs_t, vs_h;  // strides in elements
  RotateArgs r;                      // r.half == 0: no rotation
  int units;                         // upper bound of (sequence, page) pairs
  uint32_t upd_magic;                // t / (D / 16) = t upd_magic >> 20 for t < 1024
  int unit_toks, unit_rest;          // threads / (D / 16), and the remainder
};

// The smallest power of two s with 448 s >= amax: 448 = 1.75 * 2^8, so adding
// the distance from 1.75 to 2 carries into the exponent exactly above it.
__device__ __forceinline__ float page_scale(float amax) {
  const uint32_t e = (__float_as_uint(amax) + 0x1fffffu) >> 23;  // 448 * 2^(e - 135)
  return e <= 8u + 63u ? kMinPageScale : (e >= 8u + 175u ? kMaxPageScale : __uint_as_float((e - 8u) << 23));
}

// Four codes of y / s (r = 1 / s, exact: s is a power of two).  Saturates;
// a NaN gives a saturated code.
__device__ __forceinline__ uint32_t codes4(const float* y, float r) {
  float q[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) q[j] = __builtin_amdgcn_fmed3f(y[j] * r, -448.0f, 448.0f);
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

// 4 x 4 bytes transposed: byte j of out[i] = byte i of in[j].
__device__ __forceinline__ void transpose4(const uint32_t in[4], uint32_t out[4]) {
  const uint32_t a = __builtin_amdgcn_perm(in[1], in[0], 0x05010400u), b = __builtin_amdgcn_perm(in[1], in[0], 0x07030602u);
  const uint32_t c = __builtin_amdgcn_perm(in[3], in[2], 0x05010400u), d = __builtin_amdgcn_perm(in[3], in[2], 0x07030602u);
  out[0] = __builtin_amdgcn_perm(c, a, 0x05040100u);
  out[1] = __builtin_amdgcn_perm(c, a, 0x07060302u);
  out[2] = __builtin_amdgcn_perm(d, b, 0x05040100u);
  out[3] = __builtin_amdgcn_perm(d, b, 0x07060302u);
}

// XT: type of k and v; UPT: units of 16 values per thread.
template <int XT, int UPT>
__global__ __launch_bounds__(kAppendThreads) void kv_append_kernel(AppendArgs a) {
  extern __shared__ __align__(16) uint8_t tile[];  // [rows][D] codes of values
  __shared__ int scan[kAppendThreads / 64];
  __shared__ int found[6];
  __shared__ float wmax[2][kAppendThreads / 64];
  __shared__ TurnFreq turns[128];
  const int S = 1 << a.c.lS, D = a.c.D, TH = blockDim.x, t = threadIdx.x, unit = blockIdx.x, h = blockIdx.y;
  const int half = a.r.half;  // at most 128: two for each of 64 threads
  float inv[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) inv[j] = t + j * TH < half ? a.r.inv_freq[t + j * TH] : 0.0f;

  // the workgroup's sequence and page
  int b = unit, rank = 0;
  Seq s;
  if (a.b.cu_q) {
    if (t == 0) found[0] = -1;
    __syncthreads();
    int before = 0;
    for (int base = 0; base < a.b.B && before <= unit; base += TH) {
      int n = 0;
      if (base + t < a.b.B) {
        s = load_seq(a.b, a.c.lS, base + t);
        const int p0 = s.kv - s.q > 0 ? s.kv - s.q : 0;
        if (s.q > 0 && s.lim > p0) n = ((s.lim - 1) >> a.c.lS) - (p0 >> a.c.lS) + 1;
      }
      int total;
      const int end = before + block_scan<0>(n, scan, &total);
      if (unit >= end - n && unit < end) {
        found[0] = base + t;
        found[1] = unit - (end - n);
        found[2] = s.q0;
        found[3] = s.q;
        found[4] = s.kv;
        found[5] = s.lim;
      }
      before += total;
    }
    __syncthreads();
    b = found[0];
    rank = found[1];
    if (b < 0) return;
    s = Seq{found[2], found[3], found[4], found[5]};
  } else {
    s = load_seq(a.b, a.c.lS, b);
  }
  const int start = s.kv - s.q;  // token of the sequence's first row; rows of negative tokens are not kept
  const int p0 = start > 0 ? start : 0;
  if (s.q == 0 || s.lim <= p0) return;
  const int pg = (p0 >> a.c.lS) + rank;
  const int lo = p0 > (pg << a.c.lS) ? p0 : pg << a.c.lS;
  const int hi = s.lim < ((pg + 1) << a.c.lS) ? s.lim : (pg + 1) << a.c.lS;
  const int old = lo & (S - 1);  // earlier tokens in the page
  const int row0 = s.q0 + lo - start, n = hi - lo;
  const int page = a.b.table[(size_t)b * a.b.max_pages + pg];

  // the new tokens: every load first
  const int upd = D >> 4, units = n * upd, first = (int)((t * a.upd_magic) >> 20);
  RawVec<XT, 8> ka[UPT], kb[UPT], va[UPT], vb[UPT];
  int tok[UPT], gs[UPT], at_p[UPT], at_q[UPT], pos[UPT];
#pragma unroll
  for (int j = 0; j < UPT; ++j) {
    // unit j TH + t; past the last, the same values of token 0, which change no maximum
    int k = first + j * a.unit_toks, g = t - first * upd + j * a.unit_rest;
    k += g >= upd;
    g -= g >= upd ? upd : 0;
    tok[j] = k < n ? k : 0;
    gs[j] = g;
    unit_groups<8>(gs[j], half, D, at_p[j], at_q[j]);
    pos[j] = lo + tok[j];
    if (half && a.r.pos) pos[j] = a.r.pos[row0 + tok[j]];  // on the first axis
    const size_t krow = (size_t)(row0 + tok[j]) * a.ks_t + (size_t)h * a.ks_h;
    const size_t vrow = (size_t)(row0 + tok[j]) * a.vs_t + (size_t)h * a.vs_h + 8 * gs[j];
    ka[j] = load_vec<XT, 8>(a.k, krow + at_p[j]);
    kb[j] = load_vec<XT, 8>(a.k, krow + at_q[j]);
    va[j] = load_vec<XT, 8>(a.v, vrow);
    vb[j] = load_vec<XT, 8>(a.v, vrow + (D >> 1));
  }
  // the frequencies, once per workgroup, while the tokens are on their way
#pragma unroll
  for (int j = 0; j < 2; ++j)
    if (t + j * TH < half) turns[t + j * TH] = turn_freq(inv[j]);
  __syncthreads();
  if ((unsigned)page >= (unsigned)a.c.pages) return;
  const size_t at = (size_t)page * a.c.H + h;
  const float kwas = old > 0 ? a.c.ks[at] : 0.0f, vwas = old > 0 ? a.c.vs[at] : 0.0f;

  // in fp32, and the largest magnitudes
  float x[UPT][16], y[UPT][16], kmax = 0.0f, vmax = 0.0f;
  TurnFreq freq[8];
#pragma unroll
  for (int j = 0; j < UPT; ++j) {
    float2 cs[8];
    const bool turn = gs[j] < (half >> 3);
    if (turn) {
      const Place place = place_of(pos[j], a.r.inverse);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int pair = unit_pair<8>(gs[j], i, half, a.r.interleaved);
        if (XT == DT_F32 || j == 0 || a.unit_rest) freq[i] = turns[pair];  // else the same pairs as before
        Place p = place;
        if (a.r.pair_axis) {
          const int ax = rotate_axis(a.r, pair);
          p = place_of(ax < 0 ? 0 : (a.r.pos ? a.r.pos[(size_t)ax * a.r.T + row0 + tok[j]] : pos[j]), a.r.inverse);
        }
        cs[i] = rotate_cs(p, freq[i]);
      }
    }
    unpack_vec(ka[j], x[j]);
    unpack_vec(kb[j], x[j] + 8);
    unpack_vec(va[j], y[j]);
    unpack_vec(vb[j], y[j] + 8);
    if (turn) rotate_unit<8>(x[j], x[j] + 8, cs, a.r.interleaved);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      kmax = __builtin_fmaxf(kmax, __builtin_fabsf(x[j][i]));
      vmax = __builtin_fmaxf(vmax, __builtin_fabsf(y[j][i]));
    }
  }
  if (__any(kmax == __builtin_inff() || vmax == __builtin_inff())) {  // then of the finite ones
    kmax = vmax = 0.0f;
#pragma unroll
    for (int j = 0; j < UPT; ++j)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float k = __builtin_fabsf(x[j][i]), v = __builtin_fabsf(y[j][i]);
        kmax = __builtin_fmaxf(kmax, k < __builtin_inff() ? k : 0.0f);
        vmax = __builtin_fmaxf(vmax, v < __builtin_inff() ? v : 0.0f);
      }
  }
  kmax = wave_max(kmax);
  vmax = wave_max(vmax);
  if ((t & 63) == 0) {
    wmax[0][t >> 6] = kmax;
    wmax[1][t >> 6] = vmax;
  }
  __syncthreads();
  for (int w = 0; w < TH >> 6; ++w) {
    kmax = __builtin_fmaxf(kmax, wmax[0][w]);
    vmax = __builtin_fmaxf(vmax, wmax[1][w]);
  }

  uint8_t* kc = a.c.kc + at * ((size_t)D << a.c.lS);
  uint8_t* vc = a.c.vc + at * ((size_t)D << a.c.lS);
  const float kneed = page_scale(kmax), vneed = page_scale(vmax);
  const float know = kwas > kneed ? kwas : kneed, vnow = vwas > vneed ? vwas : vneed;
  if (old > 0 && know != kwas) {  // recode what was there
    const float ratio = kwas / know;
    for (int i = t; i < (old * D) >> 4; i += TH) {
      uint4 w = *reinterpret_cast<uint4*>(kc + 16 * (size_t)i);
      *reinterpret_cast<uint4*>(kc + 16 * (size_t)i) =
          make_uint4(recode4(w.x, ratio), recode4(w.y, ratio), recode4(w.z, ratio), recode4(w.w, ratio));
    }
  }
  if (old > 0 && vnow != vwas) {
    // the bytes of earlier tokens; those past them go back unchanged, before
    // the new ones are stored
    const float ratio = vwas / vnow;
    for (int i = t; i < ((old + 15) >> 4) * D; i += TH) {
      uint4 w = *reinterpret_cast<uint4*>(vc + 16 * (size_t)i);
      uint32_t* c = reinterpret_cast<uint32_t*>(&w);
      const int keep = old - 16 * (i / D);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = keep - 4 * j;
        const uint32_t mask = k >= 4 ? 0xffffffffu : (k <= 0 ? 0u : (1u << (8 * k)) - 1u);
        c[j] = (recode4(c[j], ratio) & mask) | (c[j] & ~mask);
      }
      *reinterpret_cast<uint4*>(vc + 16 * (size_t)i) = w;
    }
  }
  const float kr = 1.0f / know, vr = 1.0f / vnow;
#pragma unroll
  for (int j = 0; j < UPT; ++j) {
    if (j * TH + t >= units) continue;
    uint8_t* row = kc + (old + tok[j]) * D;
    *reinterpret_cast<uint2*>(row + at_p[j]) = make_uint2(codes4(x[j], kr), codes4(x[j] + 4, kr));
    *reinterpret_cast<uint2*>(row + at_q[j]) = make_uint2(codes4(x[j] + 8, kr), codes4(x[j] + 12, kr));
    row = tile + tok[j] * D + 8 * gs[j];
    *reinterpret_cast<uint2*>(row) = make_uint2(codes4(y[j], vr), codes4(y[j] + 4, vr));
    *reinterpret_cast<uint2*>(row + (D >> 1)) = make_uint2(codes4(y[j] + 8, vr), codes4(y[j] + 12, vr));
  }
  if (t == 0) {  // every thread has read the old ones, before the barrier above
    a.c.ks[at] = know;
    a.c.vs[at] = vnow;
  }
  __syncthreads();  // the codes are in LDS, the recoded bytes in the page
  const int blk0 = old >> 4, blks = ((old + n - 1) >> 4) - blk0 + 1, quads = D >> 2;
  for (int i = t; i < blks * quads; i += TH) {
    const int blk = i / quads, d = 4 * (i - blk * quads), t0 = 16 * (blk0 + blk) - old;  // its first token, among the new
    uint8_t* to = vc + ((blk0 + blk) * D + d) * 16;
    if (t0 >= 0 && t0 + 16 <= n) {
      uint32_t in[4][4], w[4][4];
#pragma unroll
      for (int k = 0; k < 16; ++k) in[k >> 2][k & 3] = *reinterpret_cast<uint32_t*>(tile + (t0 + k) * D + d);
#pragma unroll
      for (int k = 0; k < 4; ++k) transpose4(in[k], w[k]);
#pragma unroll
      for (int c = 0; c < 4; ++c) *reinterpret_cast<uint4*>(to + 16 * c) = make_uint4(w[0][c], w[1][c], w[2][c], w[3][c]);
    } else {
      for (int k = t0 < 0 ? -t0 : 0; k < 16 && t0 + k < n; ++k)
#pragma unroll
        for (int c = 0; c < 4; ++c) to[16 * c + k] = tile[(t0 + k) * D + d + c];
    }
  }
}

template <int XT>
static int append_pick(AppendArgs& a, hipStream_t st) {
  const int rows = a.b.cu_q ? 1 << a.c.lS : 1;  // new tokens of a page, at most
  const int units = rows * (a.c.D / 16);
  int TH = 64;  // two units a thread, at most
  while (2 * TH < units) TH *= 2;
  a.upd_magic = (1u << 20) / (a.c.D / 16) + 1;
  a.unit_toks = TH / (a.c.D / 16);
  a.unit_rest = TH % (a.c.D / 16);
  const size_t lds = (size_t)rows * a.c.D;  // at most 32 KB
  const dim3 grid((unsigned)a.units, (unsigned)a.c.H), block((unsigned)TH);
  if (units <= TH)
    hipLaunchKernelGGL((kv_append_kernel<XT, 1>), grid, block, lds, st, a);
  else
    hipLaunchKernelGGL((kv_append_kernel<XT, 2>), grid, block, lds, st, a);
  return (int)hipGetLastError();
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
