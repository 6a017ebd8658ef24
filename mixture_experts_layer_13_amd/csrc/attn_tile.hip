// attn_tile.hip -- attention over the paged E4M3 cache for many query rows
// (prompts and chunks).
//
// A workgroup takes 128 consecutive rows of one sequence and KV head (the
// query heads of a token are consecutive rows, so all of them use the same
// keys and values) and walks the 64-token tiles that they see.  A tile's codes
// are converted to MFMA operands once and put into LDS in operand order, 16 bytes
// per lane and fragment, so that both the writes and the reads of a wave are
// contiguous; the next tile's codes are already in flight in registers while
// the waves work on this one.  Operand layout, transposed first product and
// running softmax: attention.hpp.
// Measured, a causal prompt of 8192 tokens, 32 query and 8 KV heads of 128,
// bf16, page 64: 530 to 562 us by the card's clock, 1.0 PFLOP/s (a library
// product of 8192^3: 1.23).  The
// matrix pipe is busy for half of the cycles and the VALU for as much again
// (per score a multiply-add, an exponential of four issue slots, a sum, half a
// conversion, and the maximum), at a clock of 1.75 to 2.0 GHz under this load;
// the two overlap as far as two workgroups a CU allow.  Pages below 64 tokens
// 560 to 577 us.  Twelve chunks of up to 701 tokens over up to 6001, window 1024,
// 16 / 4 heads of 64, page 16: 48.5 to 50 us, two or three workgroups a CU, so that
// the chip waits for the CUs with three; over all of it the VALU issues in 0.37
// of the cycles and the matrix pipe is busy in 0.14.  f32 queries of heads above
// 128 spill 75 to 86 registers (4096 tokens, 16 / 4 heads of 256: 494 us, bf16
// 202, for three times the products).
#include "attn_decode.hpp"
#include "launch.hpp"

namespace moe {

constexpr int kTileThreads = 256;
constexpr int kTileWaves = kTileThreads / 64;
constexpr int kTileRows = 32 * kTileWaves;  // rows of a workgroup

struct TileArgs {
  AttnArgs a;
  int rows_below;  // sequences of at most this many rows are not worked on here
  int units;       // upper bound of (sequence, row block) pairs
  int decode;      // workgroups, before those, that take the sequences of up to 16 rows
};

__device__ __forceinline__ int tile_blocks(const TileArgs& t, int b) {
  const Seq s = load_seq(t.a.b, t.a.c.lS, b);
  const long long rows = (long long)s.q * t.a.G;
  return rows <= t.rows_below ? 0 : (int)((rows + kTileRows - 1) / kTileRows);
}

// A thread's raw codes of one tile.  With j = wave % 2: of keys, DT / 4 bytes of
// its row of MFMA tile j; of values, channels 32 (wave / 2 + 2 i) + l % 32 of
// the 16 tokens of block 2 (l / 32) + j.
template <int DT>
struct TileRaw {
  i32x4 k[DT / 64];
  i32x4 v[DT / 64];
  float ks, vs;
  bool gone;
};

struct TilePages {
  int k, v;
};

// Two workgroups a CU where the registers allow it: the matrix work of one
// covers the softmax of the other.
// UNI: pages of 64 tokens or more, so that a tile lies in one: its page, scales
// and addresses are the workgroup's, not the lane's.
template <int DT, int NS, bool UNI>
__global__ __launch_bounds__(kTileThreads, DT <= 128 && NS == 1 ? 2 : 1) void attn_tile_kernel(TileArgs ta) {
  const AttnArgs& a = ta.a;
  constexpr int KC = DT / 16;          // contraction steps of the first product
  constexpr int FR = 2 * KC * 64;      // fragments (16 bytes a lane) of keys, and of values, in a tile
  extern __shared__ __align__(16) uint8_t smem[];
  bf16x8* frag = reinterpret_cast<bf16x8*>(smem);  // [2 buffers][keys [2 j][KC] | values [DT / 32][4]][64 lanes]
  if ((int)blockIdx.x < ta.decode) {
    // single tokens among the prompts: in the same launch, beside the row
    // blocks (a batch of 12 chunks and single tokens: 7 us of 55)
    attn_decode_run<DT, 1, NS, false, false>(a, blockIdx.x / a.c.H, blockIdx.x % a.c.H,
                                             *reinterpret_cast<DecShared<DT>*>(smem));
    return;
  }
  const int block = blockIdx.x - ta.decode;
  __shared__ int scan[kTileWaves];
  __shared__ int found[2];
  __shared__ float bks[2][4], bvs[2][4];  // of the tile's blocks (UNI: not used)
  __shared__ int bgone[2][4], bany[2][2];
  const int lane = threadIdx.x & 63, m = lane & 31, g = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = block % a.c.H;  // heads in turn: with eight, each XCD's L2 keeps one head's codes

  // the row block: later blocks, which see more tokens, first
  const int unit = ta.units - 1 - block / a.c.H;
  if (threadIdx.x == 0) found[0] = -1;
  __syncthreads();
  int before = 0;
  for (int base = 0; base < a.b.B && before <= unit; base += kTileThreads) {
    const int b = base + threadIdx.x;
    const int n = b < a.b.B ? tile_blocks(ta, b) : 0;
    int t;
    const int e = before + block_scan<kTileWaves>(n, scan, &t);
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

  // queries, and what the lane's row sees
  bf16x8 q[KC][NS];
  f32x16 o[DT / 32];
  float mx = -__builtin_inff(), l = 0.0f;
  const int row = row0 + wave * 32 + m, qi = row / a.G, hd = h * a.G + row - qi * a.G;
  const bool live = qi < s.q;
  QueryRaw<KC, NS> qraw;
  load_q<32, KC, NS>(a, (size_t)(s.q0 + (live ? qi : 0)) * a.qs_t + (size_t)(live ? hd : 0) * a.qs_h, 16 * g, qraw);
#pragma unroll
  for (int n = 0; n < DT / 32; ++n)
#pragma unroll
    for (int k = 0; k < 16; ++k) o[n][k] = 0.0f;
  const int p0 = s.kv - s.q;
  const int hi = !live ? 0 : (a.causal && p0 + qi + 1 < s.lim ? p0 + qi + 1 : s.lim);
  const int lo = a.window > 0 ? p0 + qi - a.window + 1 : 0;
  const int all_lo = a.window > 0 ? p0 + i1 - a.window : 0;  // tokens [all_lo, all_hi) every row sees
  const int all_hi = a.causal && p0 + i0 + 1 < s.lim ? p0 + i0 + 1 : s.lim;

  // pages a tile ahead of codes, codes kAhead tiles ahead of fragments; past the
  // last tile all three go on with what is at hand, unused, so that the loop
  // has no branches (addresses are clamped into the cache)
  const int j = wave & 1, bk = 16 * (2 * ((m >> 2) & 1) + j), bv = 16 * (2 * g + j);  // first tokens of the blocks
  const uint32_t page_bytes = (uint32_t)(a.c.H * D) << lS;                            // at most 2^23
  const uint8_t* kbase = a.c.kc + (size_t)((h << lS) * D);
  const uint8_t* vbase = a.c.vc + (size_t)((h << lS) * D);
  uint32_t koff[DT / 64], voff[DT / 64];  // the lane's place in a tile (UNI) or in its block
#pragma unroll
  for (int c = 0; c < DT / 64; ++c) {
    const int d = 32 * ((wave >> 1) * (DT / 64) + c) + 16 * g, n = 32 * ((wave >> 1) + 2 * c) + m;
    koff[c] = (4 * (m >> 3) + (m & 3) + (UNI ? bk : 0)) * D + (d < D ? d : 0);
    voff[c] = (UNI ? bv * D : 0) + (n < D ? 16 * n : 0);
  }
  auto pages = [&](int tile) {  // as in the table (UNI: v only)
    const int ik = (tile * kAttnTile + (UNI ? 0 : bk)) >> lS, iv = (tile * kAttnTile + (UNI ? 0 : bv)) >> lS;
    TilePages p{};
    if (!UNI) p.k = table[ik < a.b.max_pages ? ik : 0];
    p.v = table[iv < a.b.max_pages ? iv : 0];
    return p;
  };
  // two tiles' codes in flight where the registers hold them: the loop is
  // shorter than a load from memory takes
  constexpr int kAhead = DT <= 128 && NS == 1 ? 2 : 1;
  TileRaw<DT> codes[kAhead];
  auto load = [&](TileRaw<DT>& raw, const TilePages& pg, int tile) {
    const int t0 = tile * kAttnTile;
    const uint32_t page = UNI ? __builtin_amdgcn_readfirstlane(pg.v) : pg.v, pages = a.c.pages;
    const uint32_t v = page < pages ? page : 0, k = UNI ? v : ((uint32_t)pg.k < pages ? pg.k : 0);
    raw.gone = page >= pages || (!UNI && (t0 + bv >= vw.hi || t0 + bv + 16 <= vw.lo));
    const uint8_t* kp = kbase + ((uint64_t)k * page_bytes + (uint32_t)(((t0 + (UNI ? 0 : bk)) & (S - 1)) * D));
    const uint8_t* vp = vbase + ((uint64_t)v * page_bytes + (uint32_t)(((t0 + (UNI ? 0 : bv)) & (S - 1)) * D));
#pragma unroll
    for (int c = 0; c < DT / 64; ++c) {
      raw.k[c] = ld16(kp + koff[c]);
      raw.v[c] = ld16(vp + voff[c]);
    }
    const uint64_t at = (uint64_t)v * (uint32_t)a.c.H + h;
    raw.ks = a.c.ks[at];
    raw.vs = a.c.vs[at];
  };
  auto trim = [&](TileRaw<DT>& raw, int tile) {  // zeros for the values of tokens that no row sees
    const int t0 = tile * kAttnTile;
    if (t0 < vw.lo || t0 + kAttnTile > vw.hi || (UNI ? raw.gone : __any(raw.gone))) {
      const int skip = vw.lo - (t0 + bv), n = raw.gone ? 0 : vw.hi - (t0 + bv);
#pragma unroll
      for (int c = 0; c < DT / 64; ++c) raw.v[c] = keep_bytes(raw.v[c], skip, n);
    }
  };
  // one of the DT / 16 fragments that the thread makes of its codes
  auto store = [&](const TileRaw<DT>& raw, int buf, int x) {
    bf16x8* kf = frag + buf * 2 * FR + (j * KC + (wave >> 1) * (DT / 32)) * 64 + lane;
    bf16x8* vf = frag + buf * 2 * FR + FR + ((wave >> 1) * 4 + 2 * j) * 64 + lane;
    const int c = x >> 2, e = 2 * (x & 1);
    if (x & 2)
      vf[(8 * c + (x & 1)) * 64] = value_op<NS>(raw.v[c][e], raw.v[c][e + 1]);
    else
      kf[(2 * c + (x & 1)) * 64] = codes_op(raw.k[c][e], raw.k[c][e + 1]);
  };
  // scale of the scores and of the values of the lane's two blocks, and
  // whether they are hidden: from LDS, or (UNI) from the next tile's load
  float f0 = 1.0f, f1 = 1.0f, v0 = 1.0f, v1 = 1.0f;
  bool out0 = false, out1 = false;
  auto store_scales = [&](const TileRaw<DT>& raw, int buf) {
    const float f = raw.gone ? 1.0f : score_scale(a, raw.ks), v = raw.gone ? 1.0f : page_scale_of(raw.vs);
    if (UNI) {
      f0 = f1 = f;
      v0 = v1 = v;
      out0 = out1 = raw.gone;
    } else if (wave < 2) {
      const int any = __any(raw.gone);
      if (m == 0) {
        bks[buf][2 * g + j] = f;
        bvs[buf][2 * g + j] = v;
        bgone[buf][2 * g + j] = raw.gone;
        bany[buf][j] = any;
      }
    }
  };

  TilePages next{};  // pages of the tile that is loaded next
  if (vw.n > 0) {
    TileRaw<DT> first;
    TilePages p[1 + kAhead];
#pragma unroll
    for (int k = 0; k <= kAhead; ++k) p[k] = pages(vw.t0 + k);
    next = pages(vw.t0 + 1 + kAhead);
    load(first, p[0], vw.t0);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) load(codes[k], p[1 + k], vw.t0 + 1 + k);
    trim(first, vw.t0);
#pragma unroll
    for (int x = 0; x < KC; ++x) store(first, 0, x);
    store_scales(first, 0);
  }
  make_q<32, KC, NS>(a, qraw, 16 * g, live, q);
  __syncthreads();

  // tile i; raw: the codes of tile i + 1, then of tile i + 1 + kAhead
  auto body = [&](int i, TileRaw<DT>& raw) {
    const int tile = vw.t0 + i, t0 = tile * kAttnTile, buf = i & 1;
    const bf16x8* kf = frag + buf * 2 * FR + lane;
    const bf16x8* vf = kf + FR;
    trim(raw, tile + 1);

    // first product: fragments are read AHEAD steps early, and the next
    // tile's are made from its codes between the steps
    constexpr int AHEAD = NS == 1 ? 4 : 2;
    bf16x8 kq[AHEAD][2];
    f32x16 sc[2];
#pragma unroll
    for (int c = 0; c < AHEAD; ++c) {
      kq[c][0] = kf[c * 64];
      kq[c][1] = kf[(KC + c) * 64];
    }
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int k = 0; k < 16; ++k) sc[x][k] = 0.0f;
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int c = 0; c < KC; ++c) {
      sc[0] = mfma_split<NS>(kq[c % AHEAD][0], q[c], sc[0]);
      sc[1] = mfma_split<NS>(kq[c % AHEAD][1], q[c], sc[1]);
      if (c + AHEAD < KC) {
        kq[c % AHEAD][0] = kf[(c + AHEAD) * 64];
        kq[c % AHEAD][1] = kf[(KC + c + AHEAD) * 64];
      }
      store(raw, buf ^ 1, c);
      __builtin_amdgcn_sched_barrier(0);
    }
    bool masked = t0 < all_lo || t0 + kAttnTile > all_hi;
    const float cf0 = UNI ? f0 : bks[buf][2 * g], cf1 = UNI ? f1 : bks[buf][2 * g + 1];
    const float cv0 = UNI ? v0 : bvs[buf][2 * g], cv1 = UNI ? v1 : bvs[buf][2 * g + 1];
    const bool cout0 = UNI ? out0 : bgone[buf][2 * g] != 0, cout1 = UNI ? out1 : bgone[buf][2 * g + 1] != 0;
    masked |= UNI ? out0 : __builtin_amdgcn_readfirstlane(bany[buf][0] | bany[buf][1]) != 0;
    store_scales(raw, buf ^ 1);
    load(raw, next, tile + 1 + kAhead);
    next = pages(tile + 2 + kAhead);

    const int t = t0 + 32 * g;
    if (masked) {
      attn_hide(sc[0], cout0, t, lo, hi);
      attn_hide(sc[1], cout1, t + 16, lo, hi);
    }
    const float lv0 = __builtin_amdgcn_logf(cv0), lv1 = UNI ? lv0 : __builtin_amdgcn_logf(cv1);
    const float top = UNI ? __builtin_fmaf(__builtin_fmaxf(attn_top(sc[0]), attn_top(sc[1])), cf0, lv0)
                          : __builtin_fmaxf(__builtin_fmaf(attn_top(sc[0]), cf0, lv0),
                                            __builtin_fmaf(attn_top(sc[1]), cf1, lv1));
    float rv0 = __builtin_amdgcn_exp2f(-lv0), rv1 = UNI ? rv0 : __builtin_amdgcn_exp2f(-lv1);
    if (__any(top > mx + kMaxSlack || (UNI ? lv0 : __builtin_fminf(lv0, lv1)) < kLowScale)) {
      const bool low = __any((UNI ? lv0 : __builtin_fminf(lv0, lv1)) < kLowScale);
      const float mn = __builtin_fmaxf(mx, max32(top) - kMaxLow);
      if (mn != -__builtin_inff()) {
        const float keep = __builtin_amdgcn_exp2f(mx - mn);
        l = attn_lower(l, mn - mx);
        mx = mn;
#pragma unroll
        for (int n = 0; n < DT / 32; ++n) o[n] *= keep;
        if (low) l += attn_weights(sc[0], cf0, mx) + attn_weights(sc[1], cf1, mx);
      }
      if (low) rv0 = rv1 = 0.0f;
    }
    const float base = mx == -__builtin_inff() ? 0.0f : mx;
    bf16x8 p[2][2][NS];
    const float s0 = attn_probs<NS>(sc[0], cf0, lv0 - base, p[0]);
    const float s1 = attn_probs<NS>(sc[1], UNI ? cf0 : cf1, lv1 - base, p[1]);
    l += UNI ? rv0 * (s0 + s1) : rv0 * s0 + rv1 * s1;
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int n = 0; n < DT / 32; ++n) o[n] = mfma_value<NS>(vf[(n * 4 + c) * 64], p[c >> 1][c & 1], o[n]);
    __syncthreads();  // this buffer may be written, the other one read
  };
  for (int i = 0; i < vw.n; i += kAhead) {
    body(i, codes[0]);
    if (kAhead > 1 && i + 1 < vw.n) body(i + 1, codes[kAhead - 1]);
  }

  l = sum32(l);
  if (!live) return;
  const size_t orow = (size_t)(s.q0 + qi) * a.nH + hd;
#pragma unroll
  for (int n = 0; n < DT / 32; ++n)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float v[4] = {o[n][4 * k], o[n][4 * k + 1], o[n][4 * k + 2], o[n][4 * k + 3]};
      const int d = 32 * n + 8 * k + 4 * g;
      if (d < D) attn_store4<NS>(a, orow, d, v, l);
    }
  if (g == 0 && a.lse) a.lse[orow] = attn_lse(mx, l);
}

template <int DT, int NS, bool UNI>
static int tile_launch(const TileArgs& t, hipStream_t st) {
  const size_t lds = (size_t)kAttnTile * DT * 2 * 2 * 2;  // two tiles' keys and values in bf16
  if (lds > 32768) {  // with the static part past 64 KB, or near it
    static OncePerDevice once;
    const int err = once.run([&] {
      return (int)hipFuncSetAttribute(reinterpret_cast<const void*>(attn_tile_kernel<DT, NS, UNI>),
                                      hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    });
    if (err) return err;
  }
  hipLaunchKernelGGL((attn_tile_kernel<DT, NS, UNI>), dim3((unsigned)(t.decode + t.units * t.a.c.H)), dim3(kTileThreads), lds, st, t);
  return (int)hipGetLastError();
}

template <int DT>
static int tile_pick(const TileArgs& t, bool f32, hipStream_t st) {
  if (t.a.c.lS >= 6) return f32 ? tile_launch<DT, 3, true>(t, st) : tile_launch<DT, 1, true>(t, st);
  return f32 ? tile_launch<DT, 3, false>(t, st) : tile_launch<DT, 1, false>(t, st);
}

int launch_attn_tile(const AttnArgs& a, int rows_below, int units, bool f32, hipStream_t st) {
  // few-row sequences of up to 16 rows run in this launch too; wider ones
  // need more registers than a tile and have a launch of their own
  const bool both = rows_below == 16;
  const TileArgs t{a, rows_below, units, both ? a.W * a.c.H : 0};
  int err = rows_below > 16 ? launch_attn_decode(a, rows_below, f32, st) : 0;
  if (err) return err;
  if (a.c.D <= 64)
    err = tile_pick<64>(t, f32, st);
  else
    err = a.c.D <= 128 ? tile_pick<128>(t, f32, st) : tile_pick<256>(t, f32, st);
  return err || !both ? err : launch_attn_join16(a, f32, st);
}

int attn_tile_rows() { return kTileRows; }

}  // namespace moe
