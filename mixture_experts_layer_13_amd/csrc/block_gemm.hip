// block_gemm.hip -- block-scaled E4M3 product for many rows, of a whole batch
// or of the rows of each expert:
//   out[m, n] = sum_b as[m, b] ws[n / 128, b] sum_{k in block b} a[m, k] w[n, k]
//
// A workgroup computes TN columns of out (weight rows) x TM rows of a; its
// WN x WM waves own (TN / WN) x (TM / WM) each, weights on the MFMA row
// operand.  With KS > 1 there are so many sets of waves, each with a ring of
// its own and every KS-th block along K; their sums are added in order.  One
// 16x16x128 MFMA starts from zero and holds a whole block of 128 along K, so
// its four results a lane are added to the accumulators with one fused
// multiply-add each, the scale of the token (a lane's column) times that of
// the weight block (the same for all of a wave).
//
// Operands come through an LDS ring of two or four stages by direct-to-LDS
// loads, 128 bytes of each row a stage, both scales with them.  Row r's 16-byte
// column c lies at physical column c ^ (r / 2) mod 8: the fragment reads (lane l
// row l mod 16, columns l / 16 and 4 more) find every bank once (no conflicts
// counted in the loop).
//
// What bounds it: 8192 x 4096 x 7168 takes 197 to 240 us by the card and its heat (2.0
// to 2.4 PFLOP/s; a library's product with one scale for each tensor 186), the matrix pipe
// busy 0.58 of the cycles at 1.78 GHz, the clock that full load leaves: 32 compute
// units alone take 1.36 us for a 256 x 256 x 128 block, the whole chip 1.75.  Hence
// 256 x 256 (the fewest LDS and L2 bytes a product) where there are enough rows, one
// fused multiply-add a sum and block, and nothing else in the loop.  Measured and
// slower: 32 x 32 x 64 instructions (225 us against 211), all fragments of a block
// read ahead, the stage's two operands freed apart with a second barrier.
// Few tiles: a four-stage ring, one workgroup a compute unit; two stages of 128 x 128
// leave room for two workgroups, whose barriers and ends overlap.
#include <algorithm>

#include "block_gemm.hpp"
#include "block_load.hpp"
#include "common.hpp"
#include "launch.hpp"

namespace moe {

template <int TN, int TM, int WN, int WM>
struct BTile {
  static constexpr int kWaves = WN * WM;
  static constexpr int NI = TN / WN / 16, MJ = TM / WM / 16;  // blocks of 16 of a wave
  static constexpr int WLoads = TN / 8 / kWaves, ALoads = TM / 8 / kWaves;  // ring loads of a wave (8 rows each)
  static constexpr int Loads = WLoads + ALoads + 1;                         // and one of scales
  static constexpr int kCodes = (TN + TM) * 128;
  static constexpr int kStage = kCodes + (TM + 64) * 4;  // codes, scales of the rows of a, of the weight blocks
  static_assert(TN % (8 * kWaves) == 0 && TM % (8 * kWaves) == 0, "whole loads");
  static_assert(128 % (TN / WN) == 0, "a wave's weight rows share their scale");
  static_assert(TM % 64 == 0 && TM / 64 < kWaves, "a wave for 64 rows' scales, and one more");
  static_assert(NI % 2 == 0, "two operands of weights in turn");
};

// Tile number blockIdx.x: the workgroups of an XCD (dealt out round-robin) take
// consecutive tiles, in groups of spans times all of N, so that the rows and weights
// that they share meet in that XCD's L2: of a batch kGroup spans, of experts kGroup
// or up to as many again less one, none of two experts.
constexpr int kGroup = 4;
template <int TM>
__device__ __forceinline__ bool b_tile(const BlockGemmArgs& g, int ntn, RowSpan& s, int& nt) {
  RowSpans<TM> all;
  const int spans = g.ids ? all.total(g) : (g.M + TM - 1) / TM, total = spans * ntn;
  if ((int)blockIdx.x >= total) return false;
  const int xcd = blockIdx.x % 8, per = total / 8, rem = total % 8;
  const int t = xcd * per + min(xcd, rem) + (int)blockIdx.x / 8;
  if (!g.ids) {
    const int grp = t / (kGroup * ntn), r = t % (kGroup * ntn), gs = min(kGroup, spans - grp * kGroup);
    nt = r / gs;
    s = all.at(g, grp * kGroup + r % gs);
    return true;
  }
  const auto x = all.expert_of(g, t / ntn, true);
  // its spans in groups of `small`, and of one more the first `more`
  const int groups = max(x.spans / kGroup, 1), small = x.spans / groups, more = x.spans % groups;
  int u = t - x.span * ntn, at = more * (small + 1);
  const bool large = u < at * ntn;
  const int gs = large ? small + 1 : small;
  if (large)
    at = 0;
  else
    u -= at * ntn;
  const int r = u % (gs * ntn);
  nt = r / gs;
  s = all.span(x, at + u / (gs * ntn) * gs + r % gs);
  return true;
}

template <int TN, int TM, int WN, int WM, int STAGES, int KS, int OT, bool MOVED, bool PAST>
__global__ __launch_bounds__(KS * WN * WM * 64) void block_gemm_kernel(BlockGemmArgs g, int ntn) {
  using B = BTile<TN, TM, WN, WM>;
  constexpr int NI = B::NI, MJ = B::MJ, S = NI * MJ;
  constexpr int LAG = 2, RING = 4;  // a step's sums are added LAG steps later
  static_assert(S % RING == 0 && LAG < RING, "sums of a block's last steps are found by the next block");
  constexpr bool WIDE = OT == DT_F32;
  __shared__ __attribute__((aligned(16))) char ring0[KS * B::kStage];
  __shared__ __attribute__((aligned(16))) char ring1[KS * B::kStage];
  __shared__ __attribute__((aligned(16))) char ring2[STAGES > 2 ? KS * B::kStage : 16];
  __shared__ __attribute__((aligned(16))) char ring3[STAGES > 2 ? KS * B::kStage : 16];
  static_assert(STAGES == 2 || STAGES == 4, "fragments and scales take turns with every block");
  static_assert((STAGES - 1) * B::Loads < 64, "counted waits");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = KS > 1 ? wave / B::kWaves : 0, wv = wave - part * B::kWaves;
  char* const stage0 = ring0 + part * B::kStage;
  char* const stage1 = ring1 + part * B::kStage;
  char* const stage2 = ring2 + (STAGES > 2 ? part * B::kStage : 0);
  char* const stage3 = ring3 + (STAGES > 2 ? part * B::kStage : 0);
  const int steps = (g.KB + KS - 1) / KS;  // blocks of each part, the last one's perhaps past the end
  const int wn = wv % WN, wm = wv / WN;
  const int l16 = lane & 15, grp = lane >> 4;

  RowSpan s;
  int nt;
  if (!b_tile<TM>(g, ntn, s, nt)) return;
  if (s.rows <= 0) return;
  const int n0 = nt * TN;

  // Sources.  A load takes eight rows, lane l 16-byte column l mod 8 of row l / 8
  // as they will lie in LDS; its buffer ends with the last real row of this
  // wave's, and the columns past K of a last, partial block are sent past every
  // buffer.
  const int nrows = min(TN, g.N - n0), w0 = wv * B::WLoads * 8, a0 = wv * B::ALoads * 8;
  const uint8_t* wbase = g.w + ((size_t)s.e * g.N + n0 + w0) * g.K;
  const uint32_t wbytes = (uint32_t)max(nrows - w0, 0) * g.K;
  const uint8_t* abase = MOVED ? g.a : g.a + (size_t)(s.row0 + a0) * g.a_stride;
  const uint32_t abytes = MOVED         ? (uint32_t)((size_t)(g.M - 1) * g.a_stride + g.K)
                          : s.rows > a0 ? (uint32_t)((s.rows - a0 - 1) * g.a_stride + g.K)
                                        : 0u;
  auto lcol = [&](int odd) { return ((lane ^ (lane >> 4) ^ (4 * odd)) & 7) * 16; };  // of row blocks 2 q + odd
  uint32_t woff[2], aoff[MOVED ? B::ALoads : 2];
#pragma unroll
  for (int q = 0; q < 2; ++q) woff[q] = (uint32_t)(lane >> 3) * g.K + lcol(q);
  auto source = [&](int r) { return r < s.rows ? source_row(g, s.row0 + r, g.ids ? g.ids[s.row0 + r] : 0) : -1; };
  if constexpr (MOVED) {
    static_assert(B::ALoads <= 8, "a lane for each row that this wave loads");
    const int mine = source(a0 + (lane & (8 * B::ALoads - 1)));
#pragma unroll
    for (int q = 0; q < B::ALoads; ++q) {
      const int at = __shfl(mine, q * 8 + (lane >> 3), kWave);
      aoff[q] = at >= 0 ? (uint32_t)(at * g.a_stride) + lcol((wv * B::ALoads + q) & 1) : kNowhere;
    }
  } else {
#pragma unroll
    for (int q = 0; q < 2; ++q) aoff[q] = (uint32_t)((lane >> 3) * g.a_stride) + lcol(q);
  }
  // scales: wave q takes rows 64 q .. of the tile (any row's where there is
  // none: its products are not kept), the waves behind these the weight blocks'
  const bool rowscales = wv < TM / 64;
  uint32_t soff;
  if (rowscales) {
    int r = min(wv * 64 + lane, s.rows - 1);
    if (MOVED) r = max(source(r), 0);
    soff = (uint32_t)(r * g.as_m) * 4;
  } else {
    soff = (uint32_t)min(n0 / 128 + lane, g.NB - 1) * g.KB * 4;
  }
  const float* sbase = rowscales ? (MOVED ? g.as : g.as + (size_t)s.row0 * g.as_m) : g.ws + (size_t)s.e * g.NB * g.KB;
  const long long sstep = rowscales ? g.as_b : 1;
  const int sdst = B::kCodes + (rowscales ? wv * 256 : TM * 4);

  // Load v of this part's block number `step` into a stage; of blocks past the last
  // one, zeros (the buffer is empty).  A buffer's end holds for both offsets together.
  auto load = [&](auto vc, int step, char* stage) {
    constexpr int v = decltype(vc)::value;
    const int b = step * KS + part;
    const int k = b * 128;
    const bool real = b < g.KB;
    if constexpr (v < B::WLoads) {
      const int blk = wv * B::WLoads + v, odd = B::WLoads % 2 ? blk & 1 : v & 1;
      const uint32_t cut = k + lcol(odd) >= g.K ? kNowhere : 0u;
      b_dma16<PAST ? kPastCaches : 0>(b_rsrc(wbase, real ? wbytes : 0u), stage + blk * 1024,
                                      (odd ? woff[1] : woff[0]) | cut, v * 8 * g.K + k);
    } else if constexpr (v < B::WLoads + B::ALoads) {
      constexpr int q = v - B::WLoads;
      const int blk = wv * B::ALoads + q, odd = B::ALoads % 2 ? blk & 1 : q & 1;
      const uint32_t cut = k + lcol(odd) >= g.K ? kNowhere : 0u;
      const auto res = b_rsrc(abase, real ? abytes : 0u);
      char* dst = stage + TN * 128 + blk * 1024;
      if constexpr (MOVED)
        b_dma16(res, dst, aoff[q] | cut, k);
      else
        b_dma16(res, dst, (odd ? aoff[1] : aoff[0]) | cut, q * 8 * (int)g.a_stride + k);
    } else {
      b_dma4(b_rsrc(sbase + (long long)b * sstep, real ? kMost : 0u), stage + sdst, soff);
    }
  };

  // which of this wave's rows are real
  constexpr int WTN = TN / WN, WTM = TM / WM;
  static_assert(WTM <= 64, "a bit for each");
  const uint64_t real = __ballot((lane & (WTM - 1)) == lane && source(WTM * wm + lane) >= 0);

  f32x4 acc[NI][MJ] = {};
  const int nb = WTN * wn, mb = WTM * wm;  // this wave's first rows
  const int wsat = TM + (n0 % 128 + nb) / 128;
  BOperand16<false> af[2], bf[2][MJ];  // codes as read
  BOperand16<WIDE> wa, wb[MJ];         // WIDE: those at hand, converted before their first product
  float sc[2][MJ] = {};
  f32x4 t[RING] = {};
  // a lane's codes of row l16: 16-byte columns grp and 4 + grp
  const int f0 = l16 * 128 + ((grp ^ (l16 >> 1)) & 7) * 16;
  const int fa = nb * 128 + f0, fb = (TN + mb) * 128 + f0;
  auto read_a = [&](int i, const char* stage, BOperand16<false>& o) {
    const char* p = stage + 16 * i * 128;
    o.set(ld16(p + fa), ld16(p + (fa ^ 64)));
  };
  auto read_b = [&](int j, const char* stage, BOperand16<false>& o) {
    const char* p = stage + 16 * j * 128;
    o.set(ld16(p + fb), ld16(p + (fb ^ 64)));
  };
  auto read_s = [&](const char* stage, float (&o)[MJ]) {
    const float* as = reinterpret_cast<const float*>(stage + B::kCodes);
    const float ws = as[wsat];
#pragma unroll
    for (int j = 0; j < MJ; ++j) o[j] = as[mb + 16 * j + l16] * ws;
  };
  // Block b, in stage cur (P: its parity).  Its steps are an MFMA each, the
  // additions of LAG steps before under it.  The wave's reads of cur end a row
  // block before its products do; there, behind a barrier that all of block
  // b + 1 (in nxt) has landed for, cur is free for block b + STAGES and the first
  // fragments of block b + 1 are read under the last products.  The loads into
  // the stage of block b - 1 (prv), begun behind its barrier, end here, spread
  // out: a bunch of them would hold up the wave's MFMAs at the issue.
  constexpr int EARLY = B::Loads - (S - MJ) > 2 ? B::Loads - (S - MJ) : 2;
  constexpr int GAP = (S - MJ) / (B::Loads - EARLY) >= 2 ? 2 : 1;
  static_assert((B::Loads - EARLY - 1) * GAP < S - MJ, "all loads of a block come before its barrier");
  auto add = [&](auto qc, float f) {  // the sums of step q, of this block or the last
    constexpr int q = (decltype(qc)::value + S) % S;
#pragma unroll
    for (int v = 0; v < 4; ++v)
      acc[q / MJ][q % MJ][v] = __builtin_fmaf(t[q % RING][v], f, acc[q / MJ][q % MJ][v]);
  };
  auto block = [&](auto par, int b, char* cur, char* nxt, char* prv) {
    constexpr int P = decltype(par)::value;
    b_for<0, S>([&](auto qc) {
      constexpr int q = decltype(qc)::value, i = q / MJ, j = q % MJ;
      if constexpr (q == S - MJ) {
        b_wait_vmcnt<(STAGES - 2) * B::Loads>();
        b_barrier();
        read_s(nxt, sc[P ^ 1]);
      }
      if constexpr (WIDE) {
        if constexpr (j == 0) wa.set(af[i & 1]);
        if constexpr (i == 0) wb[j].set(bf[P][j]);
        t[q % RING] = block_sums16(wa, wb[j]);
      } else {
        t[q % RING] = block_sums16(af[i & 1], bf[P][j]);
      }
      if constexpr (j == 0 && i + 1 < NI) read_a(i + 1, cur, af[(i + 1) & 1]);
      if constexpr (i == NI - 1) {
        if constexpr (j == 0) read_a(0, nxt, af[0]);
        read_b(j, nxt, bf[P ^ 1][j]);
        b_for<j * EARLY / MJ, (j + 1) * EARLY / MJ>([&](auto v) { load(v, b + STAGES, cur); });
      } else if constexpr (q % GAP == 0 && q / GAP < B::Loads - EARLY) {
        load(std::integral_constant<int, EARLY + q / GAP>{}, b + STAGES - 1, prv);
      }
      constexpr int d = (q + S - LAG) % S;
      add(std::integral_constant<int, d>{}, q >= LAG ? sc[P][d % MJ] : sc[P ^ 1][d % MJ]);
      __builtin_amdgcn_sched_barrier(0);
    });
  };

  constexpr int kAhead = (STAGES - 2) * B::Loads + EARLY;  // loads behind block 0's
  b_for<0, B::Loads>([&](auto v) { load(v, 0, stage0); });
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  if constexpr (STAGES > 2) {
    b_for<0, B::Loads>([&](auto v) { load(v, 1, stage1); });
    b_for<0, B::Loads>([&](auto v) { load(v, 2, stage2); });
  }
  b_for<0, EARLY>([&](auto v) { load(v, STAGES - 1, STAGES > 2 ? stage3 : stage1); });
  b_wait_vmcnt<kAhead>();  // block 0
  b_barrier();
  read_s(stage0, sc[0]);
  read_a(0, stage0, af[0]);
#pragma unroll
  for (int j = 0; j < MJ; ++j) read_b(j, stage0, bf[0][j]);
  const std::integral_constant<int, 0> even{};
  const std::integral_constant<int, 1> odd{};
  int b = 0;
  if (!real) {  // none of this wave's rows of a is real: it loads and keeps the barriers
    b_for<EARLY, B::Loads>([&](auto v) { load(v, STAGES - 1, STAGES > 2 ? stage3 : stage1); });
    for (; b < steps; ++b) {
      b_wait_vmcnt<(STAGES - 2) * B::Loads>();
      b_barrier();
      char* const cur = b % STAGES == 0 ? stage0 : b % STAGES == 1 ? stage1 : b % STAGES == 2 ? stage2 : stage3;
      b_for<0, B::Loads>([&](auto v) { load(v, b + STAGES, cur); });
    }
    b_wait_vmcnt<0>();
  }
  // whole turns of the ring, then what is left, once: a path from one stage's
  // block to its own next would make the compiler wait for loads before its reads
  for (; b + STAGES <= steps; b += STAGES) {
    if constexpr (STAGES == 2) {
      block(even, b, stage0, stage1, stage1);
      block(odd, b + 1, stage1, stage0, stage0);
    } else {
      block(even, b, stage0, stage1, stage3);
      block(odd, b + 1, stage1, stage2, stage0);
      block(even, b + 2, stage2, stage3, stage1);
      block(odd, b + 3, stage3, stage0, stage2);
    }
  }
  if (b < steps) {
    block(even, b, stage0, stage1, STAGES == 2 ? stage1 : stage3);
    if constexpr (STAGES > 2) {
      if (b + 1 < steps) {
        block(odd, b + 1, stage1, stage2, stage0);
        if (b + 2 < steps) block(even, b + 2, stage2, stage3, stage1);
      }
    }
  }
  b_wait_vmcnt<0>();  // no load may land after the workgroup's LDS is released
  auto rest = [&](const float (&f)[MJ]) {
    b_for<S - LAG, S>([&](auto q) { add(q, f[q % MJ]); });
  };
  if (steps & 1)
    rest(sc[0]);
  else
    rest(sc[1]);

  if constexpr (KS > 1) {  // the parts' sums, in order, to the first one's waves
    static_assert((KS - 1) * B::kWaves * S * 1024 <= KS * B::kStage, "sums in one ring");
    f32x4* sums = reinterpret_cast<f32x4*>(ring0) + lane;
    b_barrier();
    if (part) {
#pragma unroll
      for (int q = 0; q < S; ++q) sums[(((part - 1) * B::kWaves + wv) * S + q) * 64] = acc[q / MJ][q % MJ];
    }
    b_barrier();
    if (part) return;
#pragma unroll
    for (int p = 0; p < KS - 1; ++p)
#pragma unroll
      for (int q = 0; q < S; ++q) acc[q / MJ][q % MJ] += sums[((p * B::kWaves + wv) * S + q) * 64];
  }

  // Value v of lane l of block (i, j): column 16 i + 4 (l / 16) + v of row
  // 16 j + l mod 16.  bf16 rows go through this wave's part of LDS (behind a
  // barrier: the others may still read theirs), 16-byte column c of row r at
  // c ^ r, so that a store writes whole row pieces of the wave.
  zero_rows<OT, TN>(g, s, n0, WN * WM * 64);
  b_barrier();
  if (OT == DT_BF16 && g.vec && n0 + nb + WTN <= g.N) {
    constexpr int kRowBytes = WTN * 2, kPieces = kRowBytes / 16, kRowsAtOnce = 64 / kPieces;
    static_assert(WTM * kRowBytes * (B::kWaves / 2) <= B::kStage, "half of the waves in each of two stages");
    char* mine = (wv < B::kWaves / 2 ? stage0 : stage1) + (wv % (B::kWaves / 2)) * WTM * kRowBytes;
#pragma unroll
    for (int j = 0; j < MJ; ++j) {
      const bool kept = real >> (16 * j + l16) & 1;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const f32x4 v = kept ? acc[i][j] : f32x4{};
        const int c = (2 * i + (grp >> 1)) ^ (l16 & (kPieces - 1));
        *reinterpret_cast<uint2*>(mine + (16 * j + l16) * kRowBytes + c * 16 + (grp & 1) * 8) =
            make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
      }
    }
    const int c = lane % kPieces;
#pragma unroll
    for (int q = 0; q < WTM / kRowsAtOnce; ++q) {
      const int r = q * kRowsAtOnce + lane / kPieces;
      const i32x4 v = ld16(mine + r * kRowBytes + (c ^ (r & 15 & (kPieces - 1))) * 16);
      if (mb + r < s.rows)
        st16(reinterpret_cast<uint16_t*>(g.out) + (size_t)(s.row0 + mb + r) * g.out_stride + n0 + nb + c * 8, v);
    }
    return;
  }
  // Rows that do not begin on 16 bytes: 16 at a time through LDS as well, a lane a
  // column, so that a store writes 64 values in a row (3766 x 6429 x 400 fp32 100 us
  // with each lane its four, 62).
  if (!g.vec) {
    constexpr int kRow = WTN + 4, kCols = WTN < 64 ? WTN : 64;
    static_assert(16 * kRow * 4 * (B::kWaves / 2) <= B::kStage, "half of the waves in each of two stages");
    float* mine =
        reinterpret_cast<float*>((wv < B::kWaves / 2 ? stage0 : stage1) + (wv % (B::kWaves / 2)) * 16 * kRow * 4);
#pragma unroll
    for (int j = 0; j < MJ; ++j) {
      const bool kept = real >> (16 * j + l16) & 1;
#pragma unroll
      for (int i = 0; i < NI; ++i)
        *reinterpret_cast<f32x4*>(mine + l16 * kRow + 16 * i + 4 * grp) = kept ? acc[i][j] : f32x4{};
#pragma unroll
      for (int q = 0; q < 16 * WTN / 64; ++q) {
        const int r = q * 64 / WTN + (WTN < 64 ? lane / kCols : 0), c = q * 64 % WTN + lane % kCols;
        const float v = mine[r * kRow + c];
        if (mb + 16 * j + r < s.rows && n0 + nb + c < g.N) {
          const size_t at = (size_t)(s.row0 + mb + 16 * j + r) * g.out_stride + n0 + nb + c;
          if constexpr (OT == DT_BF16)
            reinterpret_cast<uint16_t*>(g.out)[at] = (uint16_t)f32_to_bf16_bits(v);
          else
            reinterpret_cast<float*>(g.out)[at] = v;
        }
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < MJ; ++j) {
    const int r = mb + 16 * j + l16;
    if (r >= s.rows) continue;
    const bool kept = real >> (16 * j + l16) & 1;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const f32x4 v = kept ? acc[i][j] : f32x4{};
      const int n = n0 + nb + 16 * i + 4 * grp;
      const size_t at = (size_t)(s.row0 + r) * g.out_stride + n;
      if constexpr (OT == DT_BF16) {
        uint16_t* p = reinterpret_cast<uint16_t*>(g.out) + at;
        if (n + 4 <= g.N)
          *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        else
          for (int c = 0; c < 4 && n + c < g.N; ++c) p[c] = (uint16_t)f32_to_bf16_bits(v[c]);
      } else {
        float* p = reinterpret_cast<float*>(g.out) + at;
        if (n + 4 <= g.N)
          *reinterpret_cast<f32x4*>(p) = v;
        else
          for (int c = 0; c < 4 && n + c < g.N; ++c) p[c] = v[c];
      }
    }
  }
}

template <int TN, int TM, int WN, int WM, int STAGES, int OT, bool PAST = false, int KS = 1>
static int block_gemm_launch(const BlockGemmArgs& g, hipStream_t st) {
  BlockGemmArgs c = g;
  int ntn = (g.N + TN - 1) / TN;
  const long long tiles = row_spans(g, TM) * ntn;
  if (tiles * KS * WN * WM * 64 > kMaxThreads) return kTooManyTiles;
  void* args[] = {&c, &ntn};
  return (int)hipLaunchKernel(g.ids && g.topk ? (void*)block_gemm_kernel<TN, TM, WN, WM, STAGES, KS, OT, true, PAST>
                                              : (void*)block_gemm_kernel<TN, TM, WN, WM, STAGES, KS, OT, false, PAST>,
                              dim3((unsigned)tiles), dim3(KS * WN * WM * 64), args, 0, st);
}

// Which kernel: by the workgroups that each makes of the call, against the
// compute units, and the time of a round of them.  us for N = K = 4096, bf16 out, in a graph:
//   M            128   256   512  1024  2048  4096
//   few rows    11.0  17.1  29.2
//   64 x 64     13.4  13.5  21.9  39.6
//   64 x 128    18.2  18.0  18.6  33.9
//   128 x 128   23.9  23.6  23.7  24.4  53.3  99.3   (four stages, one a CU)
//   128 x 128   32.3  32.0  32.2  32.5  43.4  87.3   (two stages, two a CU)
//   256 x 256   51.1  52.0  51.2  50.9  52.3  65.2
// fp32 out (operands twice as wide, half the rate; in two parts: waves that share out
// the blocks of K, as conversions and waits of more waves overlap):
//   M                       200   512  1024  2048  4096 | 1037 x 1544 x 2000
//   64 x 64                20.2  29.8  55.6   104   200   17.2
//   64 x 64, two parts     16.6  32.6  61.1                19.5
//   64 x 128, two parts    23.2  25.6  48.9                14.1
//   128 x 128              35.2  35.6  41.1  80.3   158   20.6
//   128 x 128, two parts   30.7  32.2  36.7  76.4   143   18.5
//   256 x 128              57.7  57.2  58.1  67.1   134   29.3
// (with M = 200 and K = 512 one part 5.7, two 6.2; 2000 x 2000 x 400 11.7 and 14.5.)
// Rows of experts, of uneven numbers (falling like 1 / (rank + 3)), by their average:
// us for 64 experts x 2048 x 4096 | 16 x 1408 x 2048
//   rows           8            16           32           64          128          256          512
//   few (16)    113 | 13.1   139 | 15.8   200 | 21     343 | 29
//   few (32)    115 | 13.7   129 | 14.6   159 | 18     254 | 26
//   64 x 64     122 | 12.8   132 | 13.3   133 | 13.5   157 | 13.3   242 | 23     413 | 38
//   128 x 128   140 | 12.8   141 | 13.0   157 | 13.8   147 | 14.3   187 | 16     287 | 28   (four stages)
//   128 x 128                142 | 15.9   166 | 16.2   165 | 17.2   183 | 18     279 | 25     485 | 44
//   256 x 256                147 | 21.4   149 | 22.4   190 | 23.0   196 | 29     217 | 31     358 | 36
int launch_block_product(const BlockGemmArgs& g, int ot, hipStream_t st) {
  const long long cu = device_cu_count();
  // rows of a batch, or of the average expert
  const long long m = g.ids ? (std::min(g.pairs, g.R) + g.E - 1) / g.E : g.M;
  auto tiles = [&](int tn, int tm) { return ((long long)g.N + tn - 1) / tn * spans_estimate(g, tm); };
  if (tiles(32, 64) <= cu || (!g.ids && m <= 64)) return launch_block_rows(g, ot, (int)std::min(m, 64LL), st);
  if (g.ids && m <= 16) {
    // Tiles of 64 x 64 are fewer workgroups, which counts where each has to look its
    // rows up.  us of few rows | 64 x 64 past the caches, 64 experts x 2048, average 2, 8
    // and 12 rows: K 512 in blocks of 16 16 | 17, 29 | 27, 32 | 29, of 256 33 | 25, 60 | 40,
    // 66 | 40; K 4096 53 | 63, 103 | 99, 114 | 106, of 256 76 | 77, 149 | 123, 164 | 131.
    if (m <= (ot == DT_F32 ? 12 : 8) && (g.bm == 16 || tiles(64, 64) <= cu)) return launch_block_rows(g, ot, 16, st);
    const bool past = weights_past_caches(g);
    if (ot == DT_F32)
      return past ? block_gemm_launch<64, 64, 2, 2, 4, DT_F32, true>(g, st)
                  : block_gemm_launch<64, 64, 2, 2, 4, DT_F32>(g, st);
    return past ? block_gemm_launch<64, 64, 2, 2, 4, DT_BF16, true>(g, st)
                : block_gemm_launch<64, 64, 2, 2, 4, DT_BF16>(g, st);
  }
  // rounds of tiles over the chip, of `two` (hundredths of a 256 x 256 tile's time)
  // with two on a compute unit, of `one` with one; where two do not fit, one round
  auto rounds = [&](int tn, int tm, int one, int two) {
    const long long t = tiles(tn, tm), last = t % (2 * cu);
    if (!two) return t <= cu ? one : 1LL << 30;
    return t / (2 * cu) * two + (last == 0 ? 0 : last <= cu ? one : two);
  };
  if (ot == DT_F32) {
    const long long none = 1LL << 30, a = rounds(64, 64, 19, 27);
    const long long b = (tiles(128, 128) + cu - 1) / cu * 41, c = (tiles(256, 128) + cu - 1) / cu * 66;
    if (g.ids && m <= 96) return block_gemm_launch<64, 64, 2, 2, 4, DT_F32>(g, st);
    // in two parts along K where that is one round and K is long
    const bool parts = g.KB >= 12;
    const long long a2 = parts ? rounds(64, 64, 16, 0) : none, b2 = parts ? rounds(128, 128, 37, 0) : none;
    const long long d2 = parts ? rounds(64, 128, 25, 0) : none;
    const long long best = std::min({a2, d2, a, b2, b, c});
    if (best == a2) return block_gemm_launch<64, 64, 2, 2, 4, DT_F32, false, 2>(g, st);
    if (best == d2) return block_gemm_launch<64, 128, 2, 2, 2, DT_F32, false, 2>(g, st);
    if (best == a || g.N <= 64) return block_gemm_launch<64, 64, 2, 2, 4, DT_F32>(g, st);
    if (best == b2) return block_gemm_launch<128, 128, 2, 2, 2, DT_F32, false, 2>(g, st);
    if (best == b) return block_gemm_launch<128, 128, 2, 4, 4, DT_F32>(g, st);
    return block_gemm_launch<256, 128, 4, 2, 2, DT_F32>(g, st);
  }
  if (g.N <= 64 || (g.ids && m <= 48)) return block_gemm_launch<64, 64, 2, 2, 4, DT_BF16>(g, st);
  if (g.ids && m <= 96) return block_gemm_launch<128, 128, 2, 4, 4, DT_BF16>(g, st);
  // experts' last tiles, of less work than the others, fill the last of several rounds
  const long long n = tiles(256, 256);
  const long long t256 = g.ids && m < 192 ? 1LL << 30 : g.ids && n >= 2 * cu ? n * 100 / cu : (n + cu - 1) / cu * 100;
  const long long t64 = tiles(64, 64) <= 2 * cu ? rounds(64, 64, 21, 31) : 1LL << 30, t64x128 = rounds(64, 128, 28, 0);
  const long long t128one = rounds(128, 128, 37, 0), t128 = rounds(128, 128, 50, 67);
  const long long best = std::min({t64, t64x128, t128one, t128, t256});
  if (best == t64) return block_gemm_launch<64, 64, 2, 2, 4, DT_BF16>(g, st);
  if (best == t64x128) return block_gemm_launch<64, 128, 2, 2, 4, DT_BF16>(g, st);
  if (best == t128one) return block_gemm_launch<128, 128, 2, 4, 4, DT_BF16>(g, st);
  if (best == t128) return block_gemm_launch<128, 128, 2, 4, 2, DT_BF16>(g, st);
  return block_gemm_launch<256, 256, 2, 4, 2, DT_BF16>(g, st);
}

}  // namespace moe
