// block_gemm.hip -- block-scaled E4M3 product for many rows, of a whole batch
// or of the rows of each expert:
//   out[m, n] = sum_b as[m, b] ws[n / 128, b] sum_{k in block b} a[m, k] w[n, k]
//
// A workgroup computes TN columns of out (weight rows) x TM rows of a; its
// WN x WM waves own (TN / WN) x (TM / WM) each, weights on the MFMA row
// operand.  One 16x16x128 MFMA starts from zero and holds a whole block of
// 128 along K, so its four results a lane are added to the accumulators with
// one fused multiply-add each, the scale of the token (a lane's column) times
// that of the weight block (the same for all of a wave).
//
// Operands come through a two-stage LDS ring by direct-to-LDS loads, 128
// bytes of each row a stage, both scales with them.  Row r's 16-byte column
// c lies at physical column (c + (r >> 1)) mod 8.
#include "block_gemm.hpp"
#include "common.hpp"
#include "launch.hpp"

namespace moe {

template <int TN, int TM, int WN, int WM>
struct BTile {
  static constexpr int kWaves = WN * WM;
  static constexpr int NI = TN / WN / 16, MJ = TM / WM / 16;  // blocks of 16 of a wave
  static constexpr int WLoads = TN / 8 / kWaves, ALoads = TM / 8 / kWaves;  // ring loads of a wave (8 rows each)
  static constexpr int kCodes = (TN + TM) * 128;
  static constexpr int kStage = kCodes + (TM + 64) * 4;  // codes, scales of the rows of a, of the weight blocks
  static_assert(TN % (8 * kWaves) == 0 && TM % (8 * kWaves) == 0, "whole loads");
  static_assert(128 % (TN / WN) == 0, "a wave's weight rows share their scale");
  static_assert(TM % 64 == 0 && TM / 64 <= kWaves, "whole loads of the rows' scales");
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t b_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ void b_dma16(__amdgpu_buffer_rsrc_t r, char* dst, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)dst, 16, voff, soff, 0, 0);
}
__device__ __forceinline__ void b_dma4(__amdgpu_buffer_rsrc_t r, char* dst, uint32_t voff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)dst, 4, voff, 0, 0, 0);
}

constexpr uint32_t kNowhere = 0x80000000u;  // past every buffer here: such a load gives zeros

template <int TN, int TM, int WN, int WM, int OT>
__global__ __launch_bounds__(WN * WM * 64) void block_gemm_kernel(BlockGemmArgs g, int ntn) {
  using B = BTile<TN, TM, WN, WM>;
  constexpr int NI = B::NI, MJ = B::MJ;
  __shared__ __attribute__((aligned(16))) char stage0[B::kStage];
  __shared__ __attribute__((aligned(16))) char stage1[B::kStage];
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wv % WN, wm = wv / WN;
  const int l16 = lane & 15, grp = lane >> 4;

  const RowSpan s = row_span<TM>(g, blockIdx.x / ntn);
  if (s.rows <= 0) return;
  const int n0 = (int)(blockIdx.x % ntn) * TN;

  // sources.  Weight rows past N and rows of a past the span lie past their
  // buffers; the columns past K of a last, partial block are sent there
  const int nrows = min(TN, g.N - n0);
  const auto wres = b_rsrc(g.w + ((size_t)s.e * g.N + n0) * g.K, (uint32_t)nrows * g.K);
  const bool moved = g.ids && g.topk;  // rows of a come from anywhere
  const uint8_t* abase = moved ? g.a : g.a + (size_t)s.row0 * g.a_stride;
  const float* asbase = moved ? g.as : g.as + (size_t)s.row0 * g.as_m;
  const int arows = moved ? g.M : s.rows;
  const uint32_t abytes = (uint32_t)((size_t)(arows - 1) * g.a_stride + g.K);
  const auto ares = b_rsrc(abase, abytes);
  const float* wsbase = g.ws + (size_t)s.e * g.NB * g.KB;

  // this wave's loads: lane l takes row l / 8 of eight, physical column l mod 8
  uint32_t woff[B::WLoads], aoff[B::ALoads];
#pragma unroll
  for (int q = 0; q < B::WLoads; ++q) {
    const int r = (wv * B::WLoads + q) * 8 + (lane >> 3);
    woff[q] = r < nrows ? (uint32_t)r * g.K + (((lane & 7) - (r >> 1)) & 7) * 16 : kNowhere;
  }
#pragma unroll
  for (int q = 0; q < B::ALoads; ++q) {
    const int r = (wv * B::ALoads + q) * 8 + (lane >> 3);
    int at = r < s.rows ? source_row(g, s.row0 + r) : -1;
    if (at >= 0 && !moved) at = r;
    aoff[q] = at >= 0 ? (uint32_t)(at * g.a_stride) + (((lane & 7) - (r >> 1)) & 7) * 16 : kNowhere;
  }
  // scales: wave q takes rows 64 q .. of the tile (any row's where there is
  // none: its products are not kept), the last wave the weight blocks'
  uint32_t soff = 0;
  if (wv * 64 < TM) {
    const int r = min(wv * 64 + lane, s.rows - 1);
    int at = max(source_row(g, s.row0 + r), 0);
    if (!moved) at = r;
    soff = (uint32_t)(at * g.as_m) * 4;
  }
  const uint32_t wsoff = (uint32_t)min(n0 / 128 + lane, g.NB - 1) * g.KB * 4;

  auto fetch = [&](int b, char* stage) {
    const uint32_t k = (uint32_t)b * 128;
    const bool cut = (int)k + 128 > g.K;
#pragma unroll
    for (int q = 0; q < B::WLoads; ++q) {
      const int r = (wv * B::WLoads + q) * 8 + (lane >> 3);
      const bool past = cut && (int)k + (int)((((lane & 7) - (r >> 1)) & 7) * 16) >= g.K;
      b_dma16(wres, stage + (wv * B::WLoads + q) * 1024, past ? kNowhere : woff[q], k);
    }
#pragma unroll
    for (int q = 0; q < B::ALoads; ++q) {
      const int r = (wv * B::ALoads + q) * 8 + (lane >> 3);
      const bool past = cut && (int)k + (int)((((lane & 7) - (r >> 1)) & 7) * 16) >= g.K;
      b_dma16(ares, stage + TN * 128 + (wv * B::ALoads + q) * 1024, past ? kNowhere : aoff[q], k);
    }
    if (wv * 64 < TM) b_dma4(b_rsrc(asbase + (long long)b * g.as_b, 0xffffffffu), stage + B::kCodes + wv * 256, soff);
    if (wv == B::kWaves - 1) b_dma4(b_rsrc(wsbase + b, 0xffffffffu), stage + B::kCodes + TM * 4, wsoff);
  };

  f32x4 acc[NI][MJ] = {};
  const int nb = (TN / WN) * wn, mb = (TM / WM) * wm;  // this wave's first rows
  auto multiply = [&](const char* stage) {
    const float* as = reinterpret_cast<const float*>(stage + B::kCodes);
    const float ws = as[TM + (n0 % 128 + nb) / 128];
    BOperand<OT == DT_F32> bf[MJ];
    float sc[MJ];
#pragma unroll
    for (int j = 0; j < MJ; ++j) {
      const int r = mb + 16 * j + l16;
      const char* p = stage + TN * 128 + r * 128;
      const i32x4 lo = ld16(p + ((grp + (r >> 1)) & 7) * 16), hi = ld16(p + ((grp + 4 + (r >> 1)) & 7) * 16);
      bf[j].set(lo, hi);
      sc[j] = as[r] * ws;
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int r = nb + 16 * i + l16;
      const char* p = stage + r * 128;
      const i32x4 lo = ld16(p + ((grp + (r >> 1)) & 7) * 16), hi = ld16(p + ((grp + 4 + (r >> 1)) & 7) * 16);
      BOperand<OT == DT_F32> af;
      af.set(lo, hi);
#pragma unroll
      for (int j = 0; j < MJ; ++j) {
        const f32x4 t = block_sums(af, bf[j]);
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][j][v] = __builtin_fmaf(t[v], sc[j], acc[i][j][v]);
      }
    }
  };

  fetch(0, stage0);
  for (int b = 0; b < g.KB; b += 2) {
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (b + 1 < g.KB) fetch(b + 1, stage1);
    multiply(stage0);
    if (b + 1 >= g.KB) break;
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (b + 2 < g.KB) fetch(b + 2, stage0);
    multiply(stage1);
  }

  // value v of lane l of block (i, j): column 16 i + 4 (l / 16) + v of row
  // 16 j + l mod 16
#pragma unroll
  for (int j = 0; j < MJ; ++j) {
    const int r = mb + 16 * j + l16;
    if (r >= s.rows) continue;
    const bool real = source_row(g, s.row0 + r) >= 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const f32x4 t = real ? acc[i][j] : f32x4{};
      const int n = n0 + nb + 16 * i + 4 * grp;
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
}

template <int TN, int TM, int WN, int WM>
static int block_gemm_launch(const BlockGemmArgs& g, int ot, hipStream_t st) {
  BlockGemmArgs c = g;
  int ntn = (g.N + TN - 1) / TN;
  const long long tiles = row_spans(g, TM) * ntn;
  if (tiles * WN * WM * 64 > kMaxThreads) return kTooManyTiles;
  void* args[] = {&c, &ntn};
  return (int)hipLaunchKernel(ot == DT_BF16 ? (void*)block_gemm_kernel<TN, TM, WN, WM, DT_BF16>
                                            : (void*)block_gemm_kernel<TN, TM, WN, WM, DT_F32>,
                              dim3((unsigned)tiles), dim3(WN * WM * 64), args, 0, st);
}

int launch_block_product(const BlockGemmArgs& g, int ot, hipStream_t st) {
  const int rows = g.ids ? g.bm : g.M;
  if (rows <= 64) return launch_block_rows(g, ot, rows, st);
  return block_gemm_launch<128, 128, 2, 2>(g, ot, st);
}

}  // namespace moe
