// attn_decode.hip -- attention over the paged E4M3 cache for few query rows:
// one token per sequence, or a few, times the query heads that share a KV
// head, up to 16 NR rows.
//
// The cache's bytes bound it: every code is read once, for all the rows that
// share the KV head.  The tiles of all sequences are laid end to end, and W
// workgroups per KV head take equal runs of them, so that a ragged batch, or
// one long sequence, fills the chip as evenly as equal ones.  Within a run the
// four waves take every fourth tile, each with its own running maximum, sum
// and accumulators, operands straight from memory (attention.hpp: no LDS, no
// transposition); they are joined through LDS at the end of a sequence.  A
// sequence that lies in one run is finished there; the others leave a part
// per workgroup, which attn_join_kernel joins.
#include "attention.hpp"
#include "launch.hpp"

namespace moe {

constexpr int kDecThreads = 256;
constexpr int kDecWaves = kDecThreads / 64;
constexpr int kDecMinTiles = kDecWaves;  // a shorter run would leave waves idle

// Tiles of sequence b that this kernel works on (0: none, or another kernel's).
__device__ __forceinline__ int dec_tiles(const AttnArgs& a, int rows_max, int b) {
  const Seq s = load_seq(a.b, a.c.lS, b);
  if (s.q <= 0 || s.q > rows_max / a.G) return 0;
  return view_of(a, s, 0, s.q).n;
}

__device__ __forceinline__ long long dec_run(long long total, int W) {
  const long long per = (total + W - 1) / W;
  return per < kDecMinTiles ? kDecMinTiles : per;
}

// Raw codes of one tile, and the scales of the lane's own 16 tokens.
template <int DT>
struct DecTile {
  i32x4 k[4][DT / 64];
  i32x4 v[DT / 16];
  float ks, vs;
  bool gone;  // the page of the lane's tokens is not in the cache
};

// Loads the lane's part of a tile.  Every load is unconditional, from an
// address clamped into the cache: what a lane must not use (blocks no row
// sees, pages outside the cache) it hides afterwards, keys by their scores,
// values by zeros, since a zero probability times a NaN code would be NaN.
template <int DT>
__device__ __forceinline__ void dec_load(const AttnArgs& a, const int32_t* table, const View& vw, int tile, int h,
                                         DecTile<DT>& r) {
  const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
  const int D = a.c.D, lS = a.c.lS, S = 1 << lS;
  const int tk = tile * kAttnTile + 16 * (m >> 2), tv = tile * kAttnTile + 16 * g;  // first tokens of the lane's blocks
  int pk, pv;
  attn_page(a, table, vw, tk, pk);
  r.gone = !attn_page(a, table, vw, tv, pv);
  {
    const size_t page = ((size_t)pk * a.c.H + h) << lS;
    const uint8_t* row = a.c.kc + (page + (tk & (S - 1)) + (m & 3)) * D;
#pragma unroll
    for (int c = 0; c < DT / 64; ++c) {
      const int d = g * (DT / 4) + 16 * c;
      const uint8_t* at = row + (d < D ? d : 0);
#pragma unroll
      for (int j = 0; j < 4; ++j) r.k[j][c] = ld16(at + 4 * j * D);
    }
  }
  const size_t at = (size_t)pv * a.c.H + h;
  const uint8_t* blk = a.c.vc + (at << lS) * D + (size_t)((tv & (S - 1)) * D + 16 * m);
#pragma unroll
  for (int i = 0; i < DT / 16; ++i) r.v[i] = ld16(blk + (16 * i < D ? 256 * i : 0));
  r.ks = a.c.ks[at];
  r.vs = a.c.vs[at];
  const int skip = vw.lo - tv, n = r.gone ? 0 : vw.hi - tv;
  if (skip > 0 || n < 16) {
#pragma unroll
    for (int i = 0; i < DT / 16; ++i) r.v[i] = keep_bytes(r.v[i], skip, n);
    if (r.gone) r.vs = 0.0f;
  }
}

template <int DT, int NR, int NS>
struct DecState {
  bf16x8 q[NR][DT / 32][NS];
  f32x4 o[NR][DT / 16];
  float m[NR], l[NR];
  int lo[NR], hi[NR];  // tokens that the lane's row sees
};

// Rows of the sequence into the B operand of the first product.
template <int DT, int NR, int NS>
__device__ __forceinline__ void dec_begin(const AttnArgs& a, const Seq& s, int h, DecState<DT, NR, NS>& st) {
  const int lane = threadIdx.x & 63, g = lane >> 4;
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const int row = 16 * r + (lane & 15), i = row / a.G, hd = h * a.G + row - i * a.G;
    const bool live = i < s.q;
    const size_t at = (size_t)(s.q0 + (live ? i : 0)) * a.qs_t + (size_t)(live ? hd : 0) * a.qs_h;
#pragma unroll
    for (int c = 0; c < DT / 32; ++c) {
      const int d = g * (DT / 4) + 8 * c;
      load_q8<NS>(a, at + d, live && d < a.c.D, st.q[r][c]);
    }
#pragma unroll
    for (int n = 0; n < DT / 16; ++n) st.o[r][n] = f32x4{0, 0, 0, 0};
    st.m[r] = -__builtin_inff();
    st.l[r] = 0.0f;
    const int p = s.kv - s.q + i;
    st.hi[r] = !live ? 0 : (a.causal && p + 1 < s.lim ? p + 1 : s.lim);
    st.lo[r] = a.window > 0 ? p - a.window + 1 : 0;
  }
}

template <int DT, int NR, int NS>
__device__ __forceinline__ void dec_tile(const AttnArgs& a, const View& vw, int tile, const DecTile<DT>& t,
                                         DecState<DT, NR, NS>& st) {
  const int lane = threadIdx.x & 63, g = lane >> 4;
  f32x4 s[NR][4];
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[r][j] = f32x4{0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int c = 0; c < DT / 32; ++c) {
      const bf16x8 k = codes_op(t.k[j][c >> 1][2 * (c & 1)], t.k[j][c >> 1][2 * (c & 1) + 1]);
#pragma unroll
      for (int r = 0; r < NR; ++r) s[r][j] = mfma_split<NS>(k, st.q[r][c], s[r][j]);
    }
  const int t0 = tile * kAttnTile + 16 * g;
  const float f = t.ks * a.scale2;
  bf16x8 p[NR][2][NS];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    float x[16], top = -__builtin_inff();
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      x[k] = s[r][k >> 2][k & 3] * f;
      if (t.gone || t0 + k < st.lo[r] || t0 + k >= st.hi[r]) x[k] = -__builtin_inff();
      top = __builtin_fmaxf(top, x[k]);
    }
    top = __builtin_fmaxf(top, __shfl_xor(top, 16, 64));
    top = __builtin_fmaxf(top, __shfl_xor(top, 32, 64));
    const float m = __builtin_fmaxf(st.m[r], top);
    const float base = m == -__builtin_inff() ? 0.0f : m;
    const float keep = __builtin_amdgcn_exp2f(st.m[r] - base);
    st.m[r] = m;
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      x[k] = __builtin_amdgcn_exp2f(x[k] - base);
      sum += x[k];
      x[k] *= t.vs;
    }
    st.l[r] = st.l[r] * keep + sum;
#pragma unroll
    for (int n = 0; n < DT / 16; ++n) st.o[r][n] *= keep;
    split_bf16<NS>(x, p[r][0]);
    split_bf16<NS>(x + 8, p[r][1]);
  }
#pragma unroll
  for (int n = 0; n < DT / 16; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const bf16x8 v = codes_op(t.v[n][2 * c], t.v[n][2 * c + 1]);
#pragma unroll
      for (int r = 0; r < NR; ++r) st.o[r][n] = mfma_split<NS>(v, p[r][c], st.o[r][n]);
    }
}

// Slot of a workgroup's part: a run holds at most one sequence that began
// before it (slot 0) and one that goes on after it (slot 1).
__device__ __forceinline__ size_t part_slot(const AttnArgs& a, int h, int w, int late) {
  return ((size_t)h * a.W + w) * 2 + late;
}

template <int DT, int NR, int NS>
__global__ __launch_bounds__(kDecThreads) void attn_decode_kernel(AttnArgs a) {
  constexpr int ROWS = 16 * NR, LD = DT + 4;
  __shared__ float jo[kDecWaves][16][LD];
  __shared__ float jm[kDecWaves][16], jl[kDecWaves][16];
  __shared__ int scan[kDecWaves];
  __shared__ int found[2];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4;
  const int w = blockIdx.x, h = blockIdx.y;

  // the run [begin, end) of this workgroup and the sequence it starts in
  long long total = 0;
  for (int base = 0; base < a.b.B; base += kDecThreads) {
    const int b = base + threadIdx.x;
    int t;
    block_scan<kDecThreads>(b < a.b.B ? dec_tiles(a, ROWS, b) : 0, scan, &t);
    total += t;
  }
  const long long run = dec_run(total, a.W);
  const long long begin = (long long)w * run;
  if (begin >= total) return;
  long long end = begin + run;
  if (end > total) end = total;
  long long before = 0;
  for (int base = 0; base < a.b.B && before <= begin; base += kDecThreads) {
    const int b = base + threadIdx.x;
    const int n = b < a.b.B ? dec_tiles(a, ROWS, b) : 0;
    int t;
    const long long e = before + block_scan<kDecThreads>(n, scan, &t);
    if (begin >= e - n && begin < e) {
      found[0] = b;
      found[1] = (int)(begin - (e - n));
    }
    before += t;
  }
  __syncthreads();
  int b = found[0], skip = found[1];
  long long left = end - begin;

  while (left > 0 && b < a.b.B) {
    const Seq s = load_seq(a.b, a.c.lS, b);
    const int n = dec_tiles(a, ROWS, b);
    if (n == 0) {
      ++b;
      continue;
    }
    const View vw = view_of(a, s, 0, s.q);
    const int count = n - skip < left ? n - skip : (int)left;
    const int32_t* table = a.b.table + (size_t)b * a.b.max_pages;
    DecState<DT, NR, NS> st;
    dec_begin<DT, NR, NS>(a, s, h, st);
    for (int i = wave; i < count; i += kDecWaves) {
      DecTile<DT> t;
      const int tile = vw.t0 + skip + i;
      dec_load<DT>(a, table, vw, tile, h, t);
      dec_tile<DT, NR, NS>(a, vw, tile, t, st);
    }
    const bool whole = skip == 0 && count == n;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      float l = st.l[r] + __shfl_xor(st.l[r], 16, 64);
      l += __shfl_xor(l, 32, 64);
      __syncthreads();  // the last join is read
#pragma unroll
      for (int k = 0; k < DT / 16; ++k)
        *reinterpret_cast<f32x4*>(&jo[wave][lane & 15][16 * k + 4 * g]) = st.o[r][k];
      if (g == 0) {
        jm[wave][lane] = st.m[r];
        jl[wave][lane] = l;
      }
      __syncthreads();
      const int col = threadIdx.x >> 4, row = 16 * r + col, qi = row / a.G;
      if (qi < s.q) {
        float m = -__builtin_inff();
#pragma unroll
        for (int k = 0; k < kDecWaves; ++k) m = __builtin_fmaxf(m, jm[k][col]);
        const float base = m == -__builtin_inff() ? 0.0f : m;
        float f[kDecWaves], sum = 0.0f;
#pragma unroll
        for (int k = 0; k < kDecWaves; ++k) {
          f[k] = __builtin_amdgcn_exp2f(jm[k][col] - base);
          sum += f[k] * jl[k][col];
        }
        const size_t orow = (size_t)(s.q0 + qi) * a.nH + h * a.G + row - qi * a.G;
        const size_t slot = part_slot(a, h, w, skip == 0);
        for (int d = 4 * (threadIdx.x & 15); d < a.c.D; d += 64) {
          float o[4] = {0, 0, 0, 0};
#pragma unroll
          for (int k = 0; k < kDecWaves; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] += f[k] * jo[k][col][d + j];
          if (whole)
            attn_store4<NS>(a, orow, d, o, sum);
          else
            *reinterpret_cast<float4*>(a.part_o + (slot * ROWS + row) * DT + d) = make_float4(o[0], o[1], o[2], o[3]);
        }
        if ((threadIdx.x & 15) == 0) {
          if (!whole)
            *reinterpret_cast<float2*>(a.part_ml + (slot * ROWS + row) * 2) = make_float2(m, sum);
          else if (a.lse)
            a.lse[orow] = attn_lse(m, sum);
        }
      }
    }
    left -= count;
    skip = 0;
    ++b;
  }
}

// Joins the parts of a sequence that several workgroups shared, and writes the
// rows of a sequence that sees nothing: zero, with lse -inf.
template <int DT, int NR, int NS>
__global__ __launch_bounds__(kDecThreads) void attn_join_kernel(AttnArgs a) {
  constexpr int ROWS = 16 * NR;
  __shared__ int scan[kDecWaves];
  const int b = blockIdx.x, h = blockIdx.y;
  const Seq s = load_seq(a.b, a.c.lS, b);
  if (s.q <= 0 || s.q > ROWS / a.G) return;
  const int n = view_of(a, s, 0, s.q).n;
  long long total = 0, at = 0;
  for (int base = 0; base < a.b.B; base += kDecThreads) {
    const int i = base + threadIdx.x;
    const int v = i < a.b.B ? dec_tiles(a, ROWS, i) : 0;
    int t;
    block_scan<kDecThreads>(v, scan, &t);
    total += t;
    block_scan<kDecThreads>(i < b ? v : 0, scan, &t);
    at += t;
  }
  const long long run = dec_run(total, a.W);
  const int w0 = (int)(at / run), w1 = n > 0 ? (int)((at + n - 1) / run) : w0;
  if (n > 0 && w0 == w1) return;  // finished by its workgroup
  const int rows = s.q * a.G;
  for (int i = threadIdx.x; i < rows * (a.c.D / 4); i += kDecThreads) {
    const int row = i / (a.c.D / 4), d = 4 * (i - row * (a.c.D / 4));
    float m = -__builtin_inff(), l = 0.0f, o[4] = {0, 0, 0, 0};
    if (n > 0) {
      for (int w = w0; w <= w1; ++w) {
        const float2 ml = *reinterpret_cast<const float2*>(
            a.part_ml + (part_slot(a, h, w, w == w0) * ROWS + row) * 2);
        m = __builtin_fmaxf(m, ml.x);
      }
      const float base = m == -__builtin_inff() ? 0.0f : m;
      for (int w = w0; w <= w1; ++w) {
        const size_t r = part_slot(a, h, w, w == w0) * ROWS + row;
        const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + r * 2);
        const float f = __builtin_amdgcn_exp2f(ml.x - base);
        const float4 v = *reinterpret_cast<const float4*>(a.part_o + r * DT + d);
        l += f * ml.y;
        o[0] += f * v.x;
        o[1] += f * v.y;
        o[2] += f * v.z;
        o[3] += f * v.w;
      }
    }
    const int qi = row / a.G;
    const size_t orow = (size_t)(s.q0 + qi) * a.nH + h * a.G + row - qi * a.G;
    attn_store4<NS>(a, orow, d, o, l);
    if (d == 0 && a.lse) a.lse[orow] = attn_lse(m, l);
  }
}

template <int DT, int NR, int NS>
static int dec_launch(const AttnArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((attn_decode_kernel<DT, NR, NS>), dim3((unsigned)a.W, (unsigned)a.c.H), dim3(kDecThreads), 0, st, a);
  const int err = (int)hipGetLastError();
  if (err) return err;
  hipLaunchKernelGGL((attn_join_kernel<DT, NR, NS>), dim3((unsigned)a.b.B, (unsigned)a.c.H), dim3(kDecThreads), 0, st, a);
  return (int)hipGetLastError();
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

int launch_attn_decode(const AttnArgs& a, int rows, bool f32, hipStream_t st) {
  return f32 ? dec_pick<3>(a, rows, st) : dec_pick<1>(a, rows, st);
}

}  // namespace moe
