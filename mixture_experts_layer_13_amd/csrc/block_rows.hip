// block_rows.hip -- block-scaled E4M3 product for few rows (one to 64 of a
// batch or of an expert): the weights are read once and decide the time.
//
// A workgroup computes 16 NB columns of out (weight rows) for up to 16 MB rows
// of a.  Its waves share out the blocks of 128 along K: the weights go
// straight from memory into the MFMA operand (lane l row l mod 16, bytes
// 16 (l / 16) and 64 + 16 (l / 16) on of the block), the rows of a likewise
// (they come from the L2), one 16x16x128 MFMA makes a block's sums from
// nothing and they are added, times both scales, in fp32.  The waves' sums
// meet in LDS, in the order of the waves.
#include "block_gemm.hpp"
#include "common.hpp"
#include "launch.hpp"

namespace moe {

// Bytes 16 g .. and 64 + 16 g .. of block b of a row; zeros past K.
template <bool WIDE>
__device__ __forceinline__ BOperand<WIDE> load_block(const uint8_t* row, int b, int g, int K, bool real) {
  const int c0 = b * 128 + g * 16, c1 = c0 + 64;
  i32x4 lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
  if (real && c0 < K) lo = ld16(row + c0);
  if (real && c1 < K) hi = ld16(row + c1);
  BOperand<WIDE> o;
  o.set(lo, hi);
  return o;
}

template <int NB, int MB, int WAVES, int OT>
__global__ __launch_bounds__(WAVES * 64) void block_rows_kernel(BlockGemmArgs g, int ntn) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, l16 = lane & 15, grp = lane >> 4;
  const RowSpan s = row_span<16 * MB>(g, blockIdx.x / ntn);
  if (s.rows <= 0) return;
  const int n0 = (int)(blockIdx.x % ntn) * 16 * NB;
  __shared__ f32x4 part[WAVES][NB * MB][64];
  const uint8_t* w = g.w + (size_t)s.e * g.N * g.K;
  const float* ws = g.ws + (size_t)s.e * g.NB * g.KB + (size_t)(n0 / 128) * g.KB;

  const uint8_t* wrow[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) wrow[i] = w + (size_t)min(n0 + 16 * i + l16, g.N - 1) * g.K;
  const uint8_t* arow[MB];
  const float* asr[MB];
  bool real[MB];
#pragma unroll
  for (int j = 0; j < MB; ++j) {
    const int r = 16 * j + l16;
    const int at = r < s.rows ? source_row(g, s.row0 + r) : -1;
    real[j] = at >= 0;
    arow[j] = g.a + (size_t)max(at, 0) * g.a_stride;
    asr[j] = g.as + (size_t)max(at, 0) * g.as_m;
  }
  f32x4 acc[NB][MB] = {};
  for (int b = wv; b < g.KB; b += WAVES) {
    BOperand<OT == DT_F32> wf[NB], af[MB];
    float sc[MB];
#pragma unroll
    for (int i = 0; i < NB; ++i) wf[i] = load_block<OT == DT_F32>(wrow[i], b, grp, g.K, true);
#pragma unroll
    for (int j = 0; j < MB; ++j) {
      af[j] = load_block<OT == DT_F32>(arow[j], b, grp, g.K, real[j]);
      sc[j] = asr[j][(long long)b * g.as_b] * ws[b];
    }
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int j = 0; j < MB; ++j) {
        const f32x4 t = block_sums(wf[i], af[j]);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(t[r], sc[j], acc[i][j][r]);
      }
  }
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
    if (source_row(g, s.row0 + r) < 0) t = f32x4{};
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

template <int NB, int MB, int WAVES>
static int block_rows_launch(const BlockGemmArgs& g, int ot, hipStream_t st) {
  BlockGemmArgs c = g;
  int ntn = (g.N + 16 * NB - 1) / (16 * NB);
  const long long tiles = row_spans(g, 16 * MB) * ntn;
  if (tiles * WAVES * 64 > kMaxThreads) return kTooManyTiles;
  void* args[] = {&c, &ntn};
  return (int)hipLaunchKernel(
      ot == DT_BF16 ? (void*)block_rows_kernel<NB, MB, WAVES, DT_BF16> : (void*)block_rows_kernel<NB, MB, WAVES, DT_F32>,
      dim3((unsigned)tiles), dim3(WAVES * 64), args, 0, st);
}

int launch_block_rows(const BlockGemmArgs& g, int ot, int rows, hipStream_t st) {
  if (rows <= 16) return block_rows_launch<1, 1, 16>(g, ot, st);
  if (rows <= 32) return block_rows_launch<2, 2, 8>(g, ot, st);
  return block_rows_launch<2, 4, 4>(g, ot, st);
}

}  // namespace moe
