// attn_tile.hip -- attention over the paged E4M3 cache for many query rows
// (prompts and chunks).
//
// A workgroup takes 128 consecutive rows of one sequence and KV head (the
// query heads of a token are consecutive rows, so all of them use the same
// keys and values) and walks the 64-token tiles that they see.  A tile's codes
// are converted to bf16 once and put into LDS in MFMA operand order, 16 bytes
// per lane and fragment, so that both the writes and the reads of a wave are
// contiguous; the next tile's codes are already in flight in registers while
// the waves work on this one.  Operand layout, transposed first product and
// running softmax: attention.hpp.
#include "attention.hpp"
#include "launch.hpp"

namespace moe {

constexpr int kTileThreads = 256;
constexpr int kTileWaves = kTileThreads / 64;
constexpr int kTileRT = 2;                               // 16-row tiles of a wave
constexpr int kTileRows = 16 * kTileRT * kTileWaves;     // rows of a workgroup

struct TileArgs {
  AttnArgs a;
  int rows_below;  // sequences of at most this many rows are another kernel's
  int units;       // upper bound of (sequence, row block) pairs
};

__device__ __forceinline__ int tile_blocks(const TileArgs& t, int b) {
  const Seq s = load_seq(t.a.b, t.a.c.lS, b);
  const long long rows = (long long)s.q * t.a.G;
  return rows <= t.rows_below ? 0 : (int)((rows + kTileRows - 1) / kTileRows);
}

// A thread's raw codes of one tile: keys as S^T tile j = wave, values as
// channels 16 (wave + 4 i) + m.
template <int DT>
struct TileRaw {
  i32x4 k[DT / 64];
  i32x4 v[DT / 64];
  float ks, vs;
  bool gone;
};

// Two workgroups a CU where the registers allow it: the matrix work of one
// covers the softmax of the other.
template <int DT, int NS>
__global__ __launch_bounds__(kTileThreads, DT <= 128 && NS == 1 ? 2 : 1) void attn_tile_kernel(TileArgs ta) {
  const AttnArgs& a = ta.a;
  constexpr int KC = DT / 32;              // contraction steps of the first product
  constexpr int FR = 4 * KC * 64;          // fragments (16 bytes a lane) of keys, and of values, in a tile
  extern __shared__ __align__(16) uint8_t smem[];
  bf16x8* frag = reinterpret_cast<bf16x8*>(smem);  // [2 buffers][keys [4 j][KC] | values [DT / 16][2]][64 lanes]
  __shared__ int scan[kTileWaves];
  __shared__ int found[2];
  __shared__ float bks[2][4], bvs[2][4];
  __shared__ int bgone[2][4];
  const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = blockIdx.x % a.c.H;  // heads in turn: with eight, each XCD's L2 keeps one head's codes

  // the row block: later blocks, which see more tokens, first
  const int unit = ta.units - 1 - (int)(blockIdx.x / a.c.H);
  if (threadIdx.x == 0) found[0] = -1;
  __syncthreads();
  int before = 0;
  for (int base = 0; base < a.b.B && before <= unit; base += kTileThreads) {
    const int b = base + threadIdx.x;
    const int n = b < a.b.B ? tile_blocks(ta, b) : 0;
    int t;
    const int e = before + block_scan<kTileThreads>(n, scan, &t);
    if (unit >= e - n && unit < e) {
      found[0] = b;
      found[1] = unit - (e - n);
    }
    before += t;
  }
  __syncthreads();
  const int b = __builtin_amdgcn_readfirstlane(found[0]);
  if (b < 0) return;
  const int row0 = __builtin_amdgcn_readfirstlane(found[1]) * kTileRows;
  const Seq s = load_seq(a.b, a.c.lS, b);
  const int rows = s.q * a.G - row0 < kTileRows ? s.q * a.G - row0 : kTileRows;
  const int i0 = row0 / a.G, i1 = (row0 + rows - 1) / a.G + 1;  // query tokens
  const View vw = view_of(a, s, i0, i1);
  const int32_t* table = a.b.table + (size_t)b * a.b.max_pages;
  const int D = a.c.D, lS = a.c.lS, S = 1 << lS;

  // queries, and what each row sees
  bf16x8 q[kTileRT][KC][NS];
  f32x4 o[kTileRT][DT / 16];
  float mx[kTileRT], l[kTileRT];
  int lo[kTileRT], hi[kTileRT];
#pragma unroll
  for (int r = 0; r < kTileRT; ++r) {
    const int row = row0 + (wave * kTileRT + r) * 16 + m, i = row / a.G, hd = h * a.G + row - i * a.G;
    const bool live = i < s.q;
    const size_t at = (size_t)(s.q0 + (live ? i : 0)) * a.qs_t + (size_t)(live ? hd : 0) * a.qs_h;
    load_q<KC, NS>(a, at, g * (DT / 4), live, q[r]);
#pragma unroll
    for (int n = 0; n < DT / 16; ++n) o[r][n] = f32x4{0, 0, 0, 0};
    mx[r] = -__builtin_inff();
    l[r] = 0.0f;
    const int p = s.kv - s.q + i;
    hi[r] = !live ? 0 : (a.causal && p + 1 < s.lim ? p + 1 : s.lim);
    lo[r] = a.window > 0 ? p - a.window + 1 : 0;
  }
  const int all_lo = a.window > 0 ? s.kv - s.q + i1 - a.window : 0;  // tokens [all_lo, all_hi) every row sees
  const int all_hi = a.causal && s.kv - s.q + i0 + 1 < s.lim ? s.kv - s.q + i0 + 1 : s.lim;

  // pages a tile ahead of codes, codes a tile ahead of fragments
  int pk = 0, pv = 0;
  bool okv = false;
  auto pages = [&](int tile) {
    attn_page(a, table, vw, tile * kAttnTile + 16 * (m >> 2), pk);
    okv = attn_page(a, table, vw, tile * kAttnTile + 16 * g, pv);
  };
  TileRaw<DT> raw;
  auto load = [&](int tile) {
    const int tk = tile * kAttnTile + 16 * (m >> 2), tv = tile * kAttnTile + 16 * g;
    const uint8_t* row = a.c.kc + ((((size_t)pk * a.c.H + h) << lS) + (tk & (S - 1)) + (m & 3) + 4 * wave) * D;
    const size_t at = (size_t)pv * a.c.H + h;
    const uint8_t* blk = a.c.vc + (at << lS) * D + (size_t)((tv & (S - 1)) * D + 16 * m);
#pragma unroll
    for (int c = 0; c < DT / 64; ++c) {
      const int d = g * (DT / 4) + 16 * c, n = 16 * (wave + 4 * c);
      raw.k[c] = ld16(row + (d < D ? d : 0));
      raw.v[c] = ld16(blk + (n < D ? 16 * n : 0));
    }
    raw.ks = a.c.ks[at];
    raw.vs = a.c.vs[at];
    raw.gone = !okv;
  };
  auto store = [&](int tile, int buf) {
    const int skip = vw.lo - (tile * kAttnTile + 16 * g), n = raw.gone ? 0 : vw.hi - (tile * kAttnTile + 16 * g);
    if (skip > 0 || n < 16) {
#pragma unroll
      for (int c = 0; c < DT / 64; ++c) raw.v[c] = keep_bytes(raw.v[c], skip, n);
    }
    bf16x8* kf = frag + buf * 2 * FR;
    bf16x8* vf = kf + FR;
#pragma unroll
    for (int c = 0; c < DT / 64; ++c) {
      kf[(wave * KC + 2 * c) * 64 + lane] = codes_op(raw.k[c][0], raw.k[c][1]);
      kf[(wave * KC + 2 * c + 1) * 64 + lane] = codes_op(raw.k[c][2], raw.k[c][3]);
      vf[((wave + 4 * c) * 2) * 64 + lane] = codes_op(raw.v[c][0], raw.v[c][1]);
      vf[((wave + 4 * c) * 2 + 1) * 64 + lane] = codes_op(raw.v[c][2], raw.v[c][3]);
    }
    if (wave == 0 && m == 0) {
      bks[buf][g] = raw.gone ? 0.0f : raw.ks * a.scale2;
      bvs[buf][g] = raw.gone ? 1.0f : raw.vs;
      bgone[buf][g] = raw.gone;
    }
  };

  if (vw.n > 0) {
    pages(vw.t0);
    load(vw.t0);
    if (vw.n > 1) pages(vw.t0 + 1);
    store(vw.t0, 0);
    if (vw.n > 1) {
      load(vw.t0 + 1);
      if (vw.n > 2) pages(vw.t0 + 2);
    }
    __syncthreads();
  }
  for (int i = 0; i < vw.n; ++i) {
    const int tile = vw.t0 + i, t0 = tile * kAttnTile, buf = i & 1;
    const bf16x8* kf = frag + buf * 2 * FR;
    const bf16x8* vf = kf + FR;
    f32x4 sc[kTileRT][4];
#pragma unroll
    for (int r = 0; r < kTileRT; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j) sc[r][j] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int c = 0; c < KC; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bf16x8 k = kf[(j * KC + c) * 64 + lane];
#pragma unroll
        for (int r = 0; r < kTileRT; ++r) sc[r][j] = mfma_split<NS>(k, q[r][c], sc[r][j]);
      }
    const float f = bks[buf][g], fv = bvs[buf][g];
    const bool out = bgone[buf][g] != 0;
    const bool masked = t0 < all_lo || t0 + kAttnTile > all_hi || __any(out);
    if (i + 1 < vw.n) {
      store(tile + 1, buf ^ 1);
      if (i + 2 < vw.n) {
        load(tile + 2);
        if (i + 3 < vw.n) pages(tile + 3);
      }
    }

    float top[kTileRT];
    bool grow = false;
#pragma unroll
    for (int r = 0; r < kTileRT; ++r) {
      top[r] = attn_top(sc[r], masked, out, t0 + 16 * g, lo[r], hi[r], f);
      grow |= top[r] > mx[r] + kMaxSlack;
    }
    if (__any(grow)) {
#pragma unroll
      for (int r = 0; r < kTileRT; ++r) {
        const float mn = __builtin_fmaxf(mx[r], row_max(top[r]));
        const float keep = mn == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(mx[r] - mn);
        mx[r] = mn;
        l[r] *= keep;
#pragma unroll
        for (int n = 0; n < DT / 16; ++n) o[r][n] *= keep;
      }
    }
    const float lv = __builtin_amdgcn_logf(fv), rv = __builtin_amdgcn_exp2f(-lv);
    bf16x8 p[kTileRT][2][NS];
#pragma unroll
    for (int r = 0; r < kTileRT; ++r)
      l[r] += rv * attn_probs<NS>(sc[r], masked, f, lv - (mx[r] == -__builtin_inff() ? 0.0f : mx[r]), p[r]);
#pragma unroll
    for (int n = 0; n < DT / 16; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const bf16x8 v = vf[(n * 2 + c) * 64 + lane];
#pragma unroll
        for (int r = 0; r < kTileRT; ++r) o[r][n] = mfma_split<NS>(v, p[r][c], o[r][n]);
      }
    __syncthreads();  // this buffer may be written, the other one read
  }

#pragma unroll
  for (int r = 0; r < kTileRT; ++r) {
    const float sum = row_sum(l[r]);
    const int row = row0 + (wave * kTileRT + r) * 16 + m, i = row / a.G;
    if (i >= s.q) continue;
    const size_t orow = (size_t)(s.q0 + i) * a.nH + h * a.G + row - i * a.G;
#pragma unroll
    for (int n = 0; n < DT / 16; ++n) {
      const float v[4] = {o[r][n][0], o[r][n][1], o[r][n][2], o[r][n][3]};
      if (16 * n < D) attn_store4<NS>(a, orow, 16 * n + 4 * g, v, sum);
    }
    if (g == 0 && a.lse) a.lse[orow] = attn_lse(mx[r], sum);
  }
}

template <int DT, int NS>
static int tile_launch(const TileArgs& t, hipStream_t st) {
  const size_t lds = (size_t)kAttnTile * DT * 2 * 2 * 2;  // two tiles' keys and values in bf16
  if (lds > 32768) {  // with the static part past 64 KB, or near it
    static OncePerDevice once;
    const int err = once.run([&] {
      return (int)hipFuncSetAttribute(reinterpret_cast<const void*>(attn_tile_kernel<DT, NS>),
                                      hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    });
    if (err) return err;
  }
  hipLaunchKernelGGL((attn_tile_kernel<DT, NS>), dim3((unsigned)t.units * t.a.c.H), dim3(kTileThreads), lds, st, t);
  return (int)hipGetLastError();
}

int launch_attn_tile(const AttnArgs& a, int rows_below, int units, bool f32, hipStream_t st) {
  const TileArgs t{a, rows_below, units};
  if (a.c.D <= 64) return f32 ? tile_launch<64, 3>(t, st) : tile_launch<64, 1>(t, st);
  if (a.c.D <= 128) return f32 ? tile_launch<128, 3>(t, st) : tile_launch<128, 1>(t, st);
  return f32 ? tile_launch<256, 3>(t, st) : tile_launch<256, 1>(t, st);
}

int attn_tile_rows() { return kTileRows; }

}  // namespace moe
