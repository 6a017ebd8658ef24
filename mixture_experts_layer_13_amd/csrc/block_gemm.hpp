// block_gemm.hpp -- arguments of the block quantisation (quant_blocks.hip) and
// of the block-scaled E4M3 products (block_gemm.hip, block_rows.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

namespace moe {

struct QuantArgs {
  const void* x;
  long long x_stride;
  int M, K;                 // K: values of a row of codes (gated: half a row of x)
  const int32_t* num_rows;  // device, or NULL: rows from there on are left alone
  uint8_t* codes;           // [M, K]
  float* scales;
  long long s_row, s_block;
};

int launch_quant_blocks(const QuantArgs& a, int dt, bool gated, int block_rows, hipStream_t st);

// A gathered call's rows times the stride of their scales, and of their codes, at
// most: a lane's byte offsets into them stay below 2^31.
constexpr long long kMostScales = (1LL << 29) - 1, kMostCodes = (1LL << 31) - 1;

// out[m, n] = sum_b as[m, b] ws[n / 128, b] sum_{k in block b} a[m, k] w[n, k]
struct BlockGemmArgs {
  const uint8_t* a;
  const float* as;
  long long a_stride, as_m, as_b;
  const uint8_t* w;
  const float* ws;
  int M, N, K;  // M: rows of a
  int KB, NB;   // blocks of 128 along K and N
  void* out;
  long long out_stride;
  int vec;      // rows of out can be written 16 bytes at a time
  // grouped (ids != NULL): out rows in the alignment's order, w [E] of these
  const int32_t* ids;
  const int32_t* block_expert;
  const int32_t* offsets;
  const int32_t* num_padded;
  int E, bm, R, pairs, topk;  // topk 0: a is in the alignment's order too
};

// Rows row0 .. row0 + rows - 1 of out, those of one expert; the `empty` rows behind
// them are padding that no other span has.
struct RowSpan {
  int row0, rows, e, empty;
};

#ifdef __HIPCC__
typedef float b_f32x4 __attribute__((ext_vector_type(4)));
typedef int b_i32x4 __attribute__((ext_vector_type(4)));
typedef int b_i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 b_bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 b_bf16x8 __attribute__((ext_vector_type(8)));

// One lane's 32 codes of a block of 128 along K as an MFMA operand.  E4M3
// instructions add products by groups of eight, aligned to the group's largest
// and cut below 2^-13 of its power of two (measured): of random values far inside a
// bf16 result's rounding (2.7e-5 against 1.7e-3), but not an fp32 result's, and where
// large products cancel the small ones of their group are lost.  For fp32 results
// (WIDE) the codes become bf16, exactly, whose products are added in fp32, at half
// the rate (7.7e-8).
template <bool WIDE>
struct BOperand16;
template <>
struct BOperand16<false> {
  b_i32x8 v;
  __device__ __forceinline__ void set(b_i32x4 lo, b_i32x4 hi) {
    v = b_i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  }
};
__device__ __forceinline__ void b_widen(b_i32x4 c, b_bf16x8& lo, b_bf16x8& hi) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const b_bf16x2 x = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[q], 1.0f, false);
    const b_bf16x2 y = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[q], 1.0f, true);
    b_bf16x8& o = q < 2 ? lo : hi;
    o[4 * (q % 2)] = x[0];
    o[4 * (q % 2) + 1] = x[1];
    o[4 * (q % 2) + 2] = y[0];
    o[4 * (q % 2) + 3] = y[1];
  }
}
template <>
struct BOperand16<true> {
  b_bf16x8 v[4];
  __device__ __forceinline__ void set(b_i32x4 lo, b_i32x4 hi) {
    b_widen(lo, v[0], v[1]);
    b_widen(hi, v[2], v[3]);
  }
  __device__ __forceinline__ void set(const BOperand16<false>& c) {
    set(__builtin_shufflevector(c.v, c.v, 0, 1, 2, 3), __builtin_shufflevector(c.v, c.v, 4, 5, 6, 7));
  }
};
// The sums of one block, of 16 weight rows and 16 rows of a.
__device__ __forceinline__ b_f32x4 block_sums16(const BOperand16<false>& w, const BOperand16<false>& a) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w.v, a.v, b_f32x4{}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ b_f32x4 block_sums16(const BOperand16<true>& w, const BOperand16<true>& a) {
  b_f32x4 t = {};
#pragma unroll
  for (int q = 0; q < 4; ++q) t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[q], a.v[q], t, 0, 0, 0);
  return t;
}
// Sum over the lanes up to this one.
__device__ __forceinline__ int b_sum_to(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // the lane 1 below, in rows of 16
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // lane 15 of the row below, to rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // lane 31, to the upper half
  return v;
}

// The spans of up to TM rows that the rows fall into, none of two experts, in order.
// An expert's begin with its first row; those of padding alone, which blocks longer
// than a span can end in, are left to the last one with rows (`empty`).  They are
// counted by 64 experts at a time, a lane each; to the few-row kernel, whose blocks are
// mostly as long as its spans, span i is block i then.
// (One span for every TM rows, or for every block, cost the workgroups that only
// found out that there is nothing to do their slots on the chip, and worse where they
// came in a pattern: every second one means half of the shader engines, to which
// workgroups are dealt in turn.  64 experts of 1024 rows x 2048 x 4096 in blocks of
// 128 907 us, of 16 1956, now both 587 as in blocks of 256; 49 experts of 149 rows x
// 680 x 3872 in blocks of 256 78 -> 47.)
template <int TM>
struct RowSpans {
  int from, to, count, before;  // this lane's expert of the 64 looked at
  // Looks at the experts e0 .. e0 + 63, `ahead` spans being those of the experts
  // before; returns the spans with these.
  __device__ __forceinline__ int look(const BlockGemmArgs& g, int e0, int ahead) {
    const int e = e0 + (threadIdx.x & 63);
    from = min(g.offsets[min(e, g.E)], g.R);
    to = min(g.offsets[min(e + 1, g.E)], g.R);
    count = (to - from + TM - 1) / TM;
    if (g.bm > TM && count > 0) {
      // the spans of its last block up to the last one whose first row is a pair's
      const int parts = g.bm / TM;
      int last = (count - 1) / parts * parts, end = min(count, last + parts);
      for (int step = parts > 4 ? parts / 4 : 1;; step = 1) {
        int more = 0;
#pragma unroll
        for (int k = 1; k <= 3; ++k) {
          const int c = last + k * step, f = g.ids[from + min(c, count - 1) * TM];
          more += c < end && f >= 0 && f < g.pairs;
        }
        last += more * step;
        end = min(end, last + step);
        if (step == 1) break;
      }
      count = last + 1;
    }
    const int upto = ahead + b_sum_to(count);
    before = upto - count;
    return __builtin_amdgcn_readlane(upto, 63);
  }
  // How many there are (of experts).
  __device__ __forceinline__ int total(const BlockGemmArgs& g) {
    int n = 0;
    for (int e0 = 0; e0 < g.E; e0 += 64) n = look(g, e0, n);
    return n;
  }
  // The expert e of span i, its rows [first, end) and spans [span, span + spans);
  // known: total() has just been asked.  e < 0: there is none.
  struct Expert {
    int e, first, end, span, spans;
  };
  __device__ __forceinline__ Expert expert_of(const BlockGemmArgs& g, int i, bool known) {
    for (int e0 = 0, n = 0; e0 < g.E; e0 += 64) {
      if (!known || g.E > 64) {
        n = look(g, e0, n);
        if (i >= n) continue;
      }
      const int own = __builtin_ctzll(__ballot(i >= before && i < before + count));
      return {e0 + own, __builtin_amdgcn_readlane(from, own), __builtin_amdgcn_readlane(to, own),
              __builtin_amdgcn_readlane(before, own), __builtin_amdgcn_readlane(count, own)};
    }
    return {-1, 0, 0, 0, 0};
  }
  // An expert's span number k.
  static __device__ __forceinline__ RowSpan span(const Expert& x, int k) {
    const int row0 = x.first + k * TM, left = x.end - row0;
    return {row0, min(TM, left), x.e, k == x.spans - 1 ? max(left - TM, 0) : 0};
  }
  // Span number i, less than the grid's; rows = 0: none.
  __device__ __forceinline__ RowSpan at(const BlockGemmArgs& g, int i) {
    if (g.ids && g.bm != TM) {
      const Expert x = expert_of(g, i, false);
      return x.e < 0 ? RowSpan{0, 0, 0, 0} : span(x, i - x.span);
    }
    RowSpan s{i * TM, 0, 0, 0};
    if (g.ids) s.e = g.block_expert[i];  // (asked for along with the number of rows)
    s.rows = max(min(TM, (g.ids ? min(*g.num_padded, g.R) : g.M) - s.row0), 0);
    if (s.e < 0 || (g.ids && s.e >= g.E)) s.rows = 0;
    return s;
  }
};

// The row of a that out row `row`, of pair f, comes from, -1: none (the row is zero).
__device__ __forceinline__ int source_row(const BlockGemmArgs& g, int row, int f) {
  if (!g.ids) return row;
  if (f < 0 || f >= g.pairs) return -1;
  const int at = g.topk ? f / g.topk : row;
  return at < g.M ? at : -1;
}

// Zeros for a span's rows of padding, in a tile of COLS columns from n0 on: pieces of
// at least 256 bytes, by the workgroup of a piece's first tile (tiles side by side
// are on different XCDs, whose half lines do not meet before memory).
template <int OT, int COLS>
__device__ __forceinline__ void zero_rows(const BlockGemmArgs& g, const RowSpan& s, int n0, int threads) {
  constexpr int V = OT == 1 ? 8 : 4;  // values in 16 bytes
  constexpr int kPiece = COLS > 16 * V ? COLS : 16 * V;
  if (s.empty <= 0 || n0 % kPiece) return;
  const int row0 = s.row0 + s.rows;
  const int n1 = min(n0 + kPiece, g.N), w = g.vec ? (n1 - n0) / V : 0, rest = n1 - n0 - w * V;
  if (w) {  // a thread keeps its column: one division
    const int step = threads / w, c = (int)threadIdx.x % w;
    for (int r = (int)threadIdx.x / w; r < s.empty; r += step) {
      if ((int)threadIdx.x >= step * w) break;
      const size_t at = (size_t)(row0 + r) * g.out_stride + n0 + c * V;
      *reinterpret_cast<b_i32x4*>(reinterpret_cast<char*>(g.out) + at * (16 / V)) = b_i32x4{};
    }
  }
  for (int q = threadIdx.x; q < s.empty * rest; q += threads) {
    const size_t at = (size_t)(row0 + q / rest) * g.out_stride + n0 + w * V + q % rest;
    if constexpr (OT == 1)
      reinterpret_cast<uint16_t*>(g.out)[at] = 0;
    else
      reinterpret_cast<float*>(g.out)[at] = 0.0f;
  }
}
#endif

// At most so many spans of up to tm rows.
inline long long row_spans(const BlockGemmArgs& g, int tm) {
  if (!g.ids) return ((long long)g.M + tm - 1) / tm;
  const long long n = ((long long)g.R + tm - 1) / tm;
  // the experts' pairs, and their rows
  const long long of_pairs = (g.pairs + (long long)std::min(g.E, g.pairs) * (tm - 1)) / tm;
  const long long experts = std::min<long long>(g.E, ((long long)g.R + g.bm - 1) / g.bm);
  return std::min(of_pairs, g.bm >= tm ? n : (g.R + experts * (tm - 1)) / tm);
}

// About how many of these have real rows: an expert's pairs end in one that is half
// empty on the average.
inline long long spans_estimate(const BlockGemmArgs& g, int tm) {
  if (!g.ids) return row_spans(g, tm);
  const long long pairs = g.pairs < g.R ? g.pairs : g.R, most = row_spans(g, tm);
  const long long n = pairs / tm + (g.E < pairs ? g.E : pairs) / 2 + 1;
  return n < most ? n : most;
}

// Whether weights that are read about once go past the caches: 64 MiB and more would
// only push others out (of the MALL's 256 MiB).  The few-row kernel, us: 537 MB 101.7
// -> 99.7, 67 MB 15.9 -> 15.2; 134 MB 27.5 -> 28.8 where the MALL holds them, 57 -> 33
// where it is full of another kernel's writes; 8 MB that it holds 5.6 -> 6.9.
inline bool weights_past_caches(const BlockGemmArgs& g) {
  return (long long)(g.ids ? g.E : 1) * g.N * g.K >= 64LL << 20;
}

// What a launcher returns, launching nothing, for more tiles than a grid has.
constexpr int kTooManyTiles = -1;
constexpr long long kMaxThreads = (1LL << 32) - 1;  // of a grid

// The product, by the kernel that fits (block_gemm.hip); rows: of a span.
int launch_block_product(const BlockGemmArgs& g, int out_type, hipStream_t st);
int launch_block_rows(const BlockGemmArgs& g, int out_type, int rows, hipStream_t st);

}  // namespace moe
