// attn_decode.hpp -- attention over the paged E4M3 cache for few query rows:
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
// per workgroup, which attn_join_kernel joins.  Where the table cannot hold
// many tokens a sequence (kDecOwn), each has a workgroup of its own
// instead: no search, no parts, one launch.
// Measured, 32 query and 8 KV heads of 128, bf16: 64 sequences of 4096 to 12288
// tokens (1.075 GB) 169 us, 6.35 TB/s; 131071 tokens (268 MB) 48.5 us with the
// join, 5.5 TB/s; 1000 tokens, a workgroup a head, 10 us: a chain of table,
// codes and four tiles.  16 sequences of up to 5001 tokens, one KV head of 256,
// f32: 19 us for 21 MB, one tile a wave: search, codes, and the three products
// per term, in turn.
#pragma once

#include "attention.hpp"

namespace moe {

constexpr int kDecThreads = 256;
constexpr int kDecWaves = kDecThreads / 64;
constexpr int kDecMinTiles = kDecWaves;  // a shorter run would leave waves idle
// Tokens up to which a sequence has a workgroup of its own, 8 KV heads of 128:
// one sequence of 1000 tokens 11.2 us, shared out 13.7; of 1900 14.3 and 14.0.
// Twice as many where these fill the chip: 64 sequences of 1500 to 1900 tokens
// 43 and 50 us, of 2100 to 4000 77 and 73.
constexpr int kDecOwn = 1024;
constexpr long long kCacheBytes = 256LL << 20;  // last-level cache of the MI355X

__device__ __forceinline__ int dec_slots(int tiles) { return (tiles + kDecMinTiles - 1) / kDecMinTiles * kDecMinTiles; }

// Shortest runs, of kDecMinTiles tiles, that sequence b takes of this kernel (0:
// it sees nothing, or is another kernel's): runs and sequences both begin at
// whole ones, and none spans two sequences.  At most 2^22, so that those of 256
// sequences, which are scanned at once, stay in 32 bits; tiles would not.
__device__ __forceinline__ int dec_units(const AttnArgs& a, int rows_max, int b) {
  const Seq s = load_seq(a.b, a.c.lS, b);
  if (s.q <= 0 || s.q > rows_max / a.G) return 0;
  return dec_slots(view_of(a, s, 0, s.q).n) / kDecMinTiles;
}

// The first sequence after b that this kernel works on, or B: 64 at a time, as
// a batch may have many that see nothing between two that do (256 slots, the
// first and the last with 20000 tokens: 72 us one at a time, 26 so).
__device__ __forceinline__ int dec_next(const AttnArgs& a, int rows_max, int b) {
  for (++b; b < a.b.B; b += 64) {
    const int i = b + (threadIdx.x & 63);
    const uint64_t some = __ballot(i < a.b.B && dec_units(a, rows_max, i) > 0);
    if (some) return b + __builtin_ctzll(some);
  }
  return a.b.B;
}

// Raw codes of one tile, and the scales of the lane's own 16 tokens.
template <int DT>
struct DecTile {
  i32x4 k[4][DT / 64];
  i32x4 v[DT / 16];
  float ks, vs;
  bool gone;  // the page of the lane's tokens is not in the cache
};

// The lane's part of a tile: its pages (read a tile ahead), then its codes.
// Every load is unconditional, from an address clamped into the cache: what a
// lane must not use (blocks no row sees, pages outside the cache) it hides
// afterwards, keys by their scores, values by zeros, since a zero probability
// times a NaN code would be NaN.
struct DecPages {
  int k, v;  // as in the table: of the lane's key rows, and of its own 16 tokens
};

__device__ __forceinline__ DecPages dec_pages(const AttnArgs& a, const int32_t* table, int tile) {
  const int lane = threadIdx.x & 63;
  const int ik = (tile * kAttnTile + 16 * ((lane & 15) >> 2)) >> a.c.lS, iv = (tile * kAttnTile + 16 * (lane >> 4)) >> a.c.lS;
  return DecPages{table[ik < a.b.max_pages ? ik : 0], table[iv < a.b.max_pages ? iv : 0]};
}

// A load of codes: past the caches where the pool is larger than they are (it
// keeps the table, the queries and other kernels' data in them).
template <bool STREAM>
__device__ __forceinline__ i32x4 ld_codes(const uint8_t* p) {
  const i32x4* q = reinterpret_cast<const i32x4*>(p);
  return STREAM ? __builtin_nontemporal_load(q) : *q;
}

template <int DT, bool STREAM>
__device__ __forceinline__ void dec_load_k(const AttnArgs& a, const DecPages& pg, int tile, int h, DecTile<DT>& r) {
  const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4, D = a.c.D, lS = a.c.lS;
  const int t = tile * kAttnTile + 16 * (m >> 2);  // first token of the lane's block
  const uint32_t page = (uint32_t)pg.k < (uint32_t)a.c.pages ? pg.k : 0;
  const uint8_t* row = a.c.kc + ((((size_t)page * a.c.H + h) << lS) + (t & ((1 << lS) - 1)) + (m & 3)) * D;
#pragma unroll
  for (int c = 0; c < DT / 64; ++c) {
    // the four lanes of a row read 64 consecutive bytes: with a quarter of the
    // row each, 1.07 GB of heads of 256 took 220 us and now 172
    const int d = 64 * c + 16 * g;
    const uint8_t* at = row + (d < D ? d : 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) r.k[j][c] = ld_codes<STREAM>(at + 4 * j * D);
  }
}

template <int DT, bool STREAM>
__device__ __forceinline__ void dec_load_v(const AttnArgs& a, const DecPages& pg, const View& vw, int tile, int h,
                                           DecTile<DT>& r) {
  const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4, D = a.c.D, lS = a.c.lS;
  const int t = tile * kAttnTile + 16 * g;  // first token of the lane's block
  const uint32_t page = (uint32_t)pg.v < (uint32_t)a.c.pages ? pg.v : 0;
  r.gone = (uint32_t)pg.v >= (uint32_t)a.c.pages || t >= vw.hi || t + 16 <= vw.lo;
  const size_t at = (size_t)page * a.c.H + h;
  const uint8_t* blk = a.c.vc + (at << lS) * D + (size_t)((t & ((1 << lS) - 1)) * D + 16 * m);
  r.ks = a.c.ks[at];  // used before the values: loaded before them
  r.vs = a.c.vs[at];
#pragma unroll
  for (int i = 0; i < DT / 16; ++i) r.v[i] = ld_codes<STREAM>(blk + (16 * i < D ? 256 * i : 0));
}

template <int DT, int NR, int NS>
struct DecState {
  bf16x8 q[NR][DT / 32][NS];
  f32x4 o[NR][DT / 16];
  float m[NR], l[NR];
  int lo[NR], hi[NR];  // tokens that the lane's row sees
  int all_lo, all_hi;  // tokens that every row sees
};

// Rows of the sequence into the B operand of the first product.
template <int DT, int NR, int NS>
__device__ __forceinline__ void dec_begin(const AttnArgs& a, const Seq& s, int h, DecState<DT, NR, NS>& st) {
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const int p0 = s.kv - s.q;
  st.all_lo = a.window > 0 ? s.kv - a.window : 0;
  st.all_hi = a.causal && p0 + 1 < s.lim ? p0 + 1 : s.lim;
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const int row = 16 * r + (lane & 15), i = row / a.G, hd = h * a.G + row - i * a.G;
    const bool live = i < s.q;
    const size_t at = (size_t)(s.q0 + (live ? i : 0)) * a.qs_t + (size_t)(live ? hd : 0) * a.qs_h;
    QueryRaw<DT / 32, NS> raw;
    load_q<64, DT / 32, NS>(a, at, 16 * g, raw);
    make_q<64, DT / 32, NS>(a, raw, 16 * g, live, st.q[r]);
#pragma unroll
    for (int n = 0; n < DT / 16; ++n) st.o[r][n] = f32x4{0, 0, 0, 0};
    st.m[r] = -__builtin_inff();
    st.l[r] = 0.0f;
    const int p = s.kv - s.q + i;
    st.hi[r] = !live ? 0 : (a.causal && p + 1 < s.lim ? p + 1 : s.lim);
    st.lo[r] = a.window > 0 ? p - a.window + 1 : 0;
  }
}

// The tile in t.
template <int DT, int NR, int NS>
__device__ __forceinline__ void dec_tile(const AttnArgs& a, const View& vw, int tile, DecTile<DT>& t,
                                         DecState<DT, NR, NS>& st) {
  const int lane = threadIdx.x & 63, g = lane >> 4;
  f32x16 s[NR];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f32x4 x[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) x[r] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int c = 0; c < DT / 32; ++c) {
      const bf16x8 k = codes_op(t.k[j][c >> 1][2 * (c & 1)], t.k[j][c >> 1][2 * (c & 1) + 1]);
#pragma unroll
      for (int r = 0; r < NR; ++r) x[r] = mfma_split<NS>(k, st.q[r][c], x[r]);
    }
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[r][4 * j + i] = x[r][i];
  }
  const int t0 = tile * kAttnTile;
  const bool masked = t0 < st.all_lo || t0 + kAttnTile > st.all_hi || __any(t.gone);
  const float f = t.gone ? 1.0f : score_scale(a, t.ks), fv = t.gone ? 1.0f : page_scale_of(t.vs);
  const float lv = __builtin_amdgcn_logf(fv);
  float rv = __builtin_amdgcn_exp2f(-lv);
  float top[NR];
  bool grow = lv < kLowScale;
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    if (masked) attn_hide(s[r], t.gone, t0 + 16 * g, st.lo[r], st.hi[r]);
    top[r] = __builtin_fmaf(attn_top(s[r]), f, lv);
    grow |= top[r] > st.m[r] + kMaxSlack;
  }
  if (__any(grow)) {
    const bool low = __any(lv < kLowScale);
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const float m = __builtin_fmaxf(st.m[r], max32(max16(top[r])) - kMaxLow);
      if (m != -__builtin_inff()) {
        const float keep = __builtin_amdgcn_exp2f(st.m[r] - m);
        st.l[r] = attn_lower(st.l[r], m - st.m[r]);
        st.m[r] = m;
#pragma unroll
        for (int n = 0; n < DT / 16; ++n) st.o[r][n] *= keep;
        if (low) st.l[r] += attn_weights(s[r], f, m);
      }
    }
    if (low) rv = 0.0f;
  }
  bf16x8 p[NR][2][NS];
#pragma unroll
  for (int r = 0; r < NR; ++r)
    st.l[r] += rv * attn_probs<NS>(s[r], f, lv - (st.m[r] == -__builtin_inff() ? 0.0f : st.m[r]), p[r]);
  const int skip = vw.lo - (t0 + 16 * g), n_seen = t.gone ? 0 : vw.hi - (t0 + 16 * g);
  if (__any(skip > 0 || n_seen < 16)) {
#pragma unroll
    for (int i = 0; i < DT / 16; ++i) t.v[i] = keep_bytes(t.v[i], skip, n_seen);
  }
#pragma unroll
  for (int n = 0; n < DT / 16; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const bf16x8 v = value_op<NS>(t.v[n][2 * c], t.v[n][2 * c + 1]);
#pragma unroll
      for (int r = 0; r < NR; ++r) st.o[r][n] = mfma_value<NS>(v, p[r][c], st.o[r][n]);
    }
}

// Slot of a workgroup's part: a run holds at most one sequence that began
// before it (slot 0) and one that goes on after it (slot 1).
__device__ __forceinline__ size_t part_slot(const AttnArgs& a, int h, int w, int late) {
  return ((size_t)h * a.W + w) * 2 + late;
}

// LDS of a workgroup.
template <int DT>
struct DecShared {
  float o[kDecWaves][16][DT + 4];
  float m[kDecWaves][16], l[kDecWaves][16];
  int scan[kDecWaves], found[2];
};

// The rows of sequence b, if this kernel's, that see no token: zero, with lse
// -infinity.  By one thread: they are few.
__device__ __forceinline__ bool dec_empty(const AttnArgs& a, const Seq& s, int rows_max) {
  return s.q > 0 && s.q <= rows_max / a.G && view_of(a, s, 0, s.q).n == 0;
}
template <int NS>
__device__ __forceinline__ void dec_clear(const AttnArgs& a, int rows_max, int b, int h) {
  const Seq s = load_seq(a.b, a.c.lS, b);
  if (!dec_empty(a, s, rows_max)) return;
  const float zero[4] = {0, 0, 0, 0};
  for (int i = 0; i < s.q; ++i)
    for (int g = 0; g < a.G; ++g) {
      const size_t row = (size_t)(s.q0 + i) * a.nH + h * a.G + g;
      for (int d = 0; d < a.c.D; d += 4) attn_store4<NS>(a, row, d, zero, 0.0f);
      if (a.lse) a.lse[row] = -__builtin_inff();
    }
}

// Workgroup w of KV head h.  OWN: w is the sequence, whose workgroup then also
// writes rows that see nothing.  STREAM: codes are read past the caches.
template <int DT, int NR, int NS, bool OWN, bool STREAM>
__device__ __forceinline__ void attn_decode_run(const AttnArgs& a, int w, int h, DecShared<DT>& sh) {
  constexpr int ROWS = 16 * NR;
  auto& jo = sh.o;
  auto& jm = sh.m;
  auto& jl = sh.l;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4;

  // the run [begin, end) of this workgroup and the sequence it starts in
  int b = w, skip = 0;
  long long left = 1LL << 40, run = 0;
  int2 shared = make_int2(-1, 0);
  if (!OWN) {
    long long total = 0, before = 0;  // in shortest runs
    int n = 0, e = 0, t;
    for (int base = 0; base < a.b.B; base += kDecThreads) {
      n = base + (int)threadIdx.x < a.b.B ? dec_units(a, ROWS, base + threadIdx.x) : 0;
      e = block_scan<kDecWaves>(n, sh.scan, &t);
      total += t;
      const int own = base + (int)threadIdx.x;  // of the sequences that see nothing, every W-th is this workgroup's
      if (own < a.b.B && n == 0 && own % a.W == w) dec_clear<NS>(a, ROWS, own, h);
    }
    const long long per = total > 0 ? (total + a.W - 1) / a.W : 1, begin = w * per;
    if (begin >= total) {
      if (threadIdx.x == 0) a.part_seq[h * a.W + w] = shared;
      return;
    }
    run = per * kDecMinTiles;
    left = (total - begin < per ? total - begin : per) * kDecMinTiles;
    for (int base = 0; base < a.b.B && before <= begin; base += kDecThreads) {
      if (a.b.B > kDecThreads) {  // else the one scan above
        n = base + (int)threadIdx.x < a.b.B ? dec_units(a, ROWS, base + threadIdx.x) : 0;
        e = block_scan<kDecWaves>(n, sh.scan, &t);
      }
      if (begin >= before + e - n && begin < before + e) {
        sh.found[0] = base + threadIdx.x;
        sh.found[1] = (int)(begin - (before + e - n)) * kDecMinTiles;
      }
      before += t;
    }
    __syncthreads();
    b = __builtin_amdgcn_readfirstlane(sh.found[0]);
    skip = __builtin_amdgcn_readfirstlane(sh.found[1]);
  }

  while (left > 0 && b < a.b.B) {
    const Seq s = load_seq(a.b, a.c.lS, b);
    const View vw = view_of(a, s, 0, s.q);
    const bool mine = s.q > 0 && s.q <= ROWS / a.G;
    const int n = mine ? vw.n : 0;
    if (OWN && !mine) return;
    if (!OWN && n == 0) {
      b = dec_next(a, ROWS, b);
      continue;
    }
    const int count = n - skip < left ? n - skip : (int)left;
    const int32_t* table = a.b.table + (size_t)b * a.b.max_pages;
    DecState<DT, NR, NS> st;
    dec_begin<DT, NR, NS>(a, s, h, st);
    const int first = vw.t0 + skip;
    if (wave < count) {
      DecTile<DT> t;
      DecPages after = dec_pages(a, table, first + wave);
      for (int i = wave; i < count; i += kDecWaves) {
        const DecPages pages = after;
        after = dec_pages(a, table, first + i + kDecWaves);  // ahead of the codes, not behind them
        dec_load_k<DT, STREAM>(a, pages, first + i, h, t);
        dec_load_v<DT, STREAM>(a, pages, vw, first + i, h, t);
        // the three terms of f32 fill the registers, and the compiler would
        // load the values behind the first product: 1.07 GB, D 256, 224 us
        // against 180 (bf16 without: 172, with: 178)
        if (NS > 1) __builtin_amdgcn_sched_barrier(0);
        dec_tile<DT, NR, NS>(a, vw, first + i, t, st);
      }
    }
    const bool whole = skip == 0 && count == n;
    if (!OWN && skip == 0 && !whole) {  // so this run is not the last, and its length is `run`
      const long long at = run - left;
      shared = make_int2(b, (int)((at + dec_slots(n) - 1) / run) + 1);
    }
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const float l = sum32(sum16(st.l[r]));
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
          sum += attn_lower(jl[k][col], base - jm[k][col]);
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
    if (OWN) return;
    left -= dec_slots(n) - skip;
    skip = 0;
    ++b;
  }
  if (threadIdx.x == 0) a.part_seq[h * a.W + w] = shared;
}

}  // namespace moe
