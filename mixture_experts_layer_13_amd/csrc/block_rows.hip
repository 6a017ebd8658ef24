// block_rows.hip -- block-scaled E4M3 product for few rows (one to 64 of a
// batch or of an expert): the weights are read once and decide the time.
//
// A workgroup computes 16 NB columns of out (weight rows) for up to 16 MB rows
// of a.  Its waves share out the blocks of 128 along K, wave w those that are w
// modulo their number, each with an LDS ring of its own (STAGES blocks of its
// weight rows and rows of a, by direct-to-LDS loads of whole 128-byte lines):
// no wave waits for another until the end, and all of the ring but the block at
// hand is in flight.  One 16x16x128 MFMA makes a block's sums from nothing;
// they are added, times both scales, in fp32.  The waves' sums meet in LDS, in
// the order of the waves.
//
// What bounds it: the weights' bytes and, for few of them, one chain of loads and
// barriers: 1 x 4096 x 4096 6.5 us (2.6 TB/s; an empty kernel is 3), 61 x 7168 x
// 2048 7.4, 64 experts of 8 rows x 2048 x 4096 97 (5.6 TB/s).  Weights straight to
// registers, which no other wave wants, were slower (64 x 4096 x 4096 13.2 against
// 10.0; the experts 105 against 100): too few of a wave's bytes are in flight.
#include "block_gemm.hpp"
#include "block_load.hpp"
#include "common.hpp"
#include "launch.hpp"

namespace moe {

template <int NB, int MB, int WAVES, int STAGES>
struct BRing {
  static constexpr int kCodes = (NB + MB) * 2048, kStage = kCodes + 256;  // codes, scales of the rows of a
  static constexpr int Loads = 2 * (NB + MB) + 1;
  static constexpr int kParts = WAVES * NB * MB * 1024;
  static constexpr int kOne = WAVES * kStage;  // a stage of all waves
  static_assert(MB <= 4, "the rows' scales are one load");
  static_assert(Loads * (STAGES - 1) < 64, "counted waits");
};

template <int NB, int MB, int WAVES, int STAGES, bool PAST, int OT>
__global__ __launch_bounds__(WAVES * 64) void block_rows_kernel(BlockGemmArgs g, int ntn) {
  using R = BRing<NB, MB, WAVES, STAGES>;
  constexpr bool WIDE = OT == DT_F32;
  // an array for each stage, so that the compiler sees that the reads of one
  // never meet the loads into the others
  __shared__ __attribute__((aligned(16))) char ring0[R::kOne];
  __shared__ __attribute__((aligned(16))) char ring1[R::kOne];
  __shared__ __attribute__((aligned(16))) char ring2[STAGES > 2 ? R::kOne : 16];
  __shared__ __attribute__((aligned(16))) char ring3[STAGES > 3 ? R::kOne : 16];
  __shared__ __attribute__((aligned(16))) char parts[R::kParts > R::kOne ? R::kParts : 16];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, grp = lane >> 4;
  const int span = blockIdx.x / ntn, n0 = (int)(blockIdx.x % ntn) * 16 * NB;
  // of blocks that are spans: the pairs are asked for before what the span is has come
  int pair = g.ids && g.bm == 16 * MB ? g.ids[min(span * 16 * MB + lane, g.R - 1)] : 0;
  const RowSpan s = RowSpans<16 * MB>().at(g, span);
  if (s.rows <= 0) return;
  if (g.ids && g.bm != 16 * MB) pair = g.ids[min(s.row0 + lane, g.R - 1)];
  const int source = lane < s.rows ? source_row(g, s.row0 + lane, pair) : -1;  // of row `lane` of the span
  const uint64_t real = __ballot(source >= 0);

  // sources, as in the tile kernel (block_gemm.hip)
  const int nrows = min(16 * NB, g.N - n0);
  const uint8_t* wbase = g.w + ((size_t)s.e * g.N + n0) * g.K;
  const uint32_t wbytes = (uint32_t)nrows * g.K;
  const bool moved = g.ids && g.topk;
  const uint8_t* abase = moved ? g.a : g.a + (size_t)s.row0 * g.a_stride;
  const float* asbase = moved ? g.as : g.as + (size_t)s.row0 * g.as_m;
  const uint32_t abytes = (uint32_t)((size_t)((moved ? g.M : s.rows) - 1) * g.a_stride + g.K);
  const float* ws = g.ws + ((size_t)s.e * g.NB + n0 / 128) * g.KB;
  auto lcol = [&](int odd) { return ((lane ^ (lane >> 4) ^ (4 * odd)) & 7) * 16; };
  const uint32_t woff = (uint32_t)(lane >> 3) * g.K;
  uint32_t aoff[2 * MB], soff;
  b_for<0, 2 * MB>([&](auto q) {
    const int r = 8 * q + (lane >> 3);
    const int at = __shfl(source, r, kWave);
    aoff[q] = at >= 0 ? (uint32_t)((moved ? at : r) * g.a_stride) + lcol(q & 1) : kNowhere;
  });
  soff = (uint32_t)((moved ? max(source, 0) : min(lane, s.rows - 1)) * g.as_m) * 4;
  char* const own0 = ring0 + wv * R::kStage;
  char* const own1 = ring1 + wv * R::kStage;
  char* const own2 = ring2 + (STAGES > 2 ? wv * R::kStage : 0);
  char* const own3 = ring3 + (STAGES > 3 ? wv * R::kStage : 0);

  // block b into a stage; of blocks past the last one, zeros
  auto fetch = [&](int b, char* stage) {
    const int k = b * 128;
    const bool real = b < g.KB;
    const uint32_t cut0 = k + lcol(0) >= g.K ? kNowhere : 0u, cut1 = k + lcol(1) >= g.K ? kNowhere : 0u;
    b_for<0, 2 * NB>([&](auto q) {
      b_dma16<PAST ? kPastCaches : 0>(b_rsrc(wbase, real ? wbytes : 0u), stage + q * 1024,
                                      (woff + lcol(q & 1)) | (q & 1 ? cut1 : cut0), q * 8 * g.K + k);
    });
    b_for<0, 2 * MB>([&](auto q) {
      b_dma16(b_rsrc(abase, real ? abytes : 0u), stage + NB * 2048 + q * 1024, aoff[q] | (q & 1 ? cut1 : cut0), k);
    });
    b_dma4(b_rsrc(asbase + (long long)b * g.as_b, real ? kMost : 0u), stage + R::kCodes, soff);
  };

  f32x4 acc[NB][MB] = {};
  const int f0 = l16 * 128 + ((grp ^ (l16 >> 1)) & 7) * 16;
  auto multiply = [&](int b, const char* stage) {
    const float w1 = ws[min(b, g.KB - 1)];
    BOperand16<WIDE> wf[NB], af[MB];
    float sc[MB];
#pragma unroll
    for (int i = 0; i < NB; ++i) wf[i].set(ld16(stage + i * 2048 + f0), ld16(stage + i * 2048 + (f0 ^ 64)));
#pragma unroll
    for (int j = 0; j < MB; ++j) {
      af[j].set(ld16(stage + (NB + j) * 2048 + f0), ld16(stage + (NB + j) * 2048 + (f0 ^ 64)));
      sc[j] = reinterpret_cast<const float*>(stage + R::kCodes)[16 * j + l16];
    }
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int j = 0; j < MB; ++j) {
        const f32x4 t = block_sums16(wf[i], af[j]);
        const float f = sc[j] * w1;
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(t[r], f, acc[i][j][r]);
      }
  };
  auto step = [&](int b, char* stage) {
    b_wait_vmcnt<R::Loads * (STAGES - 1)>();  // this block; the others of the ring stay in flight
    multiply(b, stage);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4) | (0 << 8));  // lgkmcnt(0): read, before it is filled anew
    fetch(b + STAGES * WAVES, stage);
  };

  fetch(wv, own0);
  fetch(wv + WAVES, own1);
  if constexpr (STAGES > 2) fetch(wv + 2 * WAVES, own2);
  if constexpr (STAGES > 3) fetch(wv + 3 * WAVES, own3);
  for (int b = wv; b < g.KB; b += STAGES * WAVES) {
    step(b, own0);
    step(b + WAVES, own1);
    if constexpr (STAGES > 2) step(b + 2 * WAVES, own2);
    if constexpr (STAGES > 3) step(b + 3 * WAVES, own3);
  }
  b_wait_vmcnt<0>();  // no load may land in what follows
  zero_rows<OT, 16 * NB>(g, s, n0, WAVES * 64);
  if constexpr (R::kParts <= R::kOne) __syncthreads();
  f32x4(*part)[NB * MB][64] = reinterpret_cast<f32x4(*)[NB * MB][64]>(R::kParts > R::kOne ? parts : ring0);
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) part[wv][i * MB + j][lane] = acc[i][j];
  __syncthreads();
  // result: value r of lane l of block (i, j) is column 16 i + 4 (l / 16) + r
  // of row 16 j + l mod 16
  for (int q = threadIdx.x; q < NB * MB * 64; q += WAVES * 64) {
    const int blk = q >> 6, ln = q & 63, i = blk / MB, j = blk % MB;
    f32x4 t = part[0][blk][ln];
#pragma unroll
    for (int v = 1; v < WAVES; ++v) t += part[v][blk][ln];
    const int r = 16 * j + (ln & 15), n = n0 + 16 * i + 4 * (ln >> 4);
    if (r >= s.rows) continue;
    if (!(real >> r & 1)) t = f32x4{};
    const size_t at = (size_t)(s.row0 + r) * g.out_stride + n;
    if constexpr (OT == DT_BF16) {
      uint16_t* p = reinterpret_cast<uint16_t*>(g.out) + at;
      if (g.vec && n + 4 <= g.N)
        *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(t[0], t[1]), pack_bf16x2(t[2], t[3]));
      else
        for (int c = 0; c < 4 && n + c < g.N; ++c) p[c] = (uint16_t)f32_to_bf16_bits(t[c]);
    } else {
      float* p = reinterpret_cast<float*>(g.out) + at;
      if (g.vec && n + 4 <= g.N)
        *reinterpret_cast<f32x4*>(p) = t;
      else
        for (int c = 0; c < 4 && n + c < g.N; ++c) p[c] = t[c];
    }
  }
}

template <int NB, int MB, int WAVES, int STAGES, bool PAST, int OT>
static int block_rows_start(const BlockGemmArgs& g, hipStream_t st) {
  BlockGemmArgs c = g;
  int ntn = (g.N + 16 * NB - 1) / (16 * NB);
  const long long tiles = row_spans(g, 16 * MB) * ntn;
  if (tiles * WAVES * 64 > kMaxThreads) return kTooManyTiles;
  void* args[] = {&c, &ntn};
  return (int)hipLaunchKernel((void*)block_rows_kernel<NB, MB, WAVES, STAGES, PAST, OT>, dim3((unsigned)tiles),
                              dim3(WAVES * 64), args, 0, st);
}

template <int NB, int MB, int WAVES, int STAGES>
static int block_rows_launch(const BlockGemmArgs& g, int ot, hipStream_t st) {
  const bool past = weights_past_caches(g);
  if (ot == DT_BF16)
    return past ? block_rows_start<NB, MB, WAVES, STAGES, true, DT_BF16>(g, st)
                : block_rows_start<NB, MB, WAVES, STAGES, false, DT_BF16>(g, st);
  return past ? block_rows_start<NB, MB, WAVES, STAGES, true, DT_F32>(g, st)
              : block_rows_start<NB, MB, WAVES, STAGES, false, DT_F32>(g, st);
}

// Narrow tiles and many waves where that gives every compute unit a workgroup and
// not many more (1 x 4096 x 4096 6.5 us, 64 x 4096 x 4096 10.0), else wider ones,
// small enough in LDS that three are on a compute unit: the next one's first
// loads run while another ends (64 experts x 2048 x 4096, eight rows each: 99.7 us,
// 5.4 TB/s; 119 with one on a compute unit).
int launch_block_rows(const BlockGemmArgs& g, int ot, int rows, hipStream_t st) {
  const long long cu = device_cu_count();
  const int mb = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
  const long long spans = spans_estimate(g, 16 * mb), n16 = ((long long)g.N + 15) / 16 * spans, n32 = (n16 + 1) / 2;
  if (mb == 1)
    return n16 <= 2 * cu ? block_rows_launch<1, 1, 8, 2>(g, ot, st) : block_rows_launch<2, 1, 4, 2>(g, ot, st);
  if (mb == 2)
    return n16 <= 2 * cu ? block_rows_launch<1, 2, 8, 2>(g, ot, st) : block_rows_launch<2, 2, 4, 2>(g, ot, st);
  if (n16 <= cu) return block_rows_launch<1, 4, 4, 2>(g, ot, st);
  return n32 <= cu ? block_rows_launch<2, 4, 4, 2>(g, ot, st) : block_rows_launch<2, 4, 2, 2>(g, ot, st);
}

}  // namespace moe
