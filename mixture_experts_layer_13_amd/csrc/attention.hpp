// attention.hpp -- what the paged-attention kernels share.
//
// Both compute, for a query row r (one head of one token) and the tokens t it
// sees, with kc, vc the E4M3 codes and ks, vs their page's scales,
//   s_t = sm_scale ks q.kc_t,  out = sum_t softmax(s)_t vs vc_t
// in one pass over the tokens with, in base 2 and fp32, a running maximum m of
// s + log2 vs and sums l of exp2(s - m) and o of exp2(s + log2 vs - m) vc:
// out = o / l, lse = m + log2 l.  Taking vs into the maximum is what lets the
// second product's operands, x = exp2(s + log2 vs - m) and the codes, be fp16
// whatever the scales: x is at most 2^15, a row's largest at least 2^7 (kMaxLow,
// kMaxSlack), so x has 11 bits down to 2^-21 of the largest and an error of
// 2^-32 of it below; as bf16 it would have 8 bits.  Codes are exact in both, and
// bf16 queries go into bf16 MFMA as they are; both accumulate in fp32.  fp32
// queries, and their x, are the sum of three bf16 terms: 24 bits, three MFMAs
// in place of one.
//
// Operand layout.  The first product is computed transposed, S^T = K Q^T, and
// the tokens of a 64-token tile are dealt to the rows of its MFMA tiles so
// that the result leaves every lane with runs of 16 consecutive tokens of one
// query row: they are exactly the lane's contraction indices as the B operand
// of O^T = V^T P^T when A is a 16-byte load of value codes (paged.hpp).  So
// probabilities never leave their lane, and neither operand of either product
// needs a transposition.
//   16x16x32 (few rows): tile j of four has as its row m the token
//   16 (m / 4) + 4 j + m % 4; lane l gets tokens 16 (l / 16) + 4 j + i
//   (i = 0..3) of query l % 16.
//   32x32x16 (many rows): tile j of two has as its row m the token
//   32 (m / 4 % 2) + 16 j + 4 (m / 8) + m % 4; lane l gets tokens
//   32 (l / 32) + 16 j + i (i = 0..15) of query l % 32.
// The D values of a key are dealt to the lane groups in turn, 16 at a time, as
// they are loaded.
#pragma once

#include "paged.hpp"

namespace moe {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kAttnTile = 64;  // tokens of a tile
// Workgroups of the few-row kernel: one per CU, or two where a tile is half as
// large (64 sequences of 8192 tokens, D 128: 169 us with one, 173 with two;
// D 64: 113 and 93).
constexpr int kAttnGroups = 512;  // at most
constexpr int attn_groups(int D) { return D <= 64 ? 512 : 256; }

struct AttnArgs {
  PagedArgs c;
  BatchArgs b;
  const void* q;
  long long qs_t, qs_h;  // strides in elements
  int nH, G;             // query heads, query heads per KV head
  float scale2;          // |sm_scale| log2(e)
  int neg;               // sm_scale < 0: the queries change sign
  int causal, window;
  void* out;             // [T][nH][D]
  float* lse;            // [T][nH] or NULL
  float* part_o;         // partial results of sequences that several workgroups share
  float* part_ml;
  int2* part_seq;        // [H][W]: sequence that begins in the workgroup's run and goes on after it, and its parts
  int W;                 // workgroups per KV head
  int rows;              // rows of a sequence, at most
};

// Tiles [t0, t0 + n) of tokens that some row of [row0, row0 + rows) of the
// sequence sees (rows count query tokens here), and the tokens [lo, hi) they see.
struct View {
  int lo, hi, t0, n;
};

__device__ __forceinline__ View view_of(const AttnArgs& a, const Seq& s, int i0, int i1) {
  View v;
  const int p0 = s.kv - s.q + i0, p1 = s.kv - s.q + i1 - 1;  // tokens of the first and last query
  int hi = a.causal && p1 + 1 < s.lim ? p1 + 1 : s.lim;
  int lo = a.window > 0 && p0 - a.window + 1 > 0 ? p0 - a.window + 1 : 0;
  if (hi < 0) hi = 0;
  if (lo > hi) lo = hi;
  v.lo = lo;
  v.hi = hi;
  v.t0 = lo / kAttnTile;
  v.n = hi > lo ? (hi + kAttnTile - 1) / kAttnTile - v.t0 : 0;
  return v;
}

// Two E4M3 codes (byte pair `hi` of w) as packed bf16: exact.
template <bool HI>
__device__ __forceinline__ uint32_t codes_bf16x2(int w) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)w, 1.0f, HI));
}

// Eight codes (two dwords) as a bf16 MFMA operand.
__device__ __forceinline__ bf16x8 codes_op(int w0, int w1) {
  const i32x4 r = {(int)codes_bf16x2<false>(w0), (int)codes_bf16x2<true>(w0), (int)codes_bf16x2<false>(w1),
                   (int)codes_bf16x2<true>(w1)};
  return as_bf16x8(r);
}

// The second product's operands, as bits: fp16 for bf16 queries (NS 1), bf16
// terms for fp32 ones.
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

template <int NS>
__device__ __forceinline__ bf16x8 value_op(int w0, int w1) {
  if (NS > 1) return codes_op(w0, w1);
  const i32x4 r = {
      __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((unsigned)w0, 1.0f, false)),
      __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((unsigned)w0, 1.0f, true)),
      __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((unsigned)w1, 1.0f, false)),
      __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((unsigned)w1, 1.0f, true))};
  return as_bf16x8(r);
}

// x as NS bf16 terms whose sum is x to 8 NS bits: term k of the eight values.
template <int NS>
__device__ __forceinline__ void split_bf16(const float x[8], bf16x8 out[NS]) {
  float rest[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) rest[i] = x[i];
#pragma unroll
  for (int k = 0; k < NS; ++k) {
    i32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = pack_bf16x2(rest[2 * i], rest[2 * i + 1]);
      w[i] = (int)v;
      if (k + 1 < NS) {
        rest[2 * i] -= bf16_bits_to_f32(v & 0xffffu);
        rest[2 * i + 1] -= bf16_bits_to_f32(v >> 16);
      }
    }
    out[k] = as_bf16x8(w);
  }
}

template <int NS>
__device__ __forceinline__ f32x4 mfma_split(const bf16x8 a, const bf16x8 b[NS], f32x4 c) {
#pragma unroll
  for (int k = NS - 1; k >= 0; --k) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b[k], c, 0, 0, 0);
  return c;
}
template <int NS>
__device__ __forceinline__ f32x16 mfma_split(const bf16x8 a, const bf16x8 b[NS], f32x16 c) {
#pragma unroll
  for (int k = NS - 1; k >= 0; --k) c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b[k], c, 0, 0, 0);
  return c;
}

// The second product: a value fragment and x, operands of value_op and
// attn_probs.
template <int NS>
__device__ __forceinline__ f32x4 mfma_value(const bf16x8 a, const bf16x8 b[NS], f32x4 c) {
  if (NS > 1) return mfma_split<NS>(a, b, c);
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b[0]), c, 0, 0, 0);
}
template <int NS>
__device__ __forceinline__ f32x16 mfma_value(const bf16x8 a, const bf16x8 b[NS], f32x16 c) {
  if (NS > 1) return mfma_split<NS>(a, b, c);
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b[0]), c, 0, 0, 0);
}

// A page's scale, within the bounds that an append keeps (a scale of zero, or
// none at all, then makes no infinity or NaN of its own).
__device__ __forceinline__ float page_scale_of(float s) {
  return __builtin_fminf(__builtin_fmaxf(s, kMinPageScale), kMaxPageScale);
}

// Scale of a page's scores; at least the smallest normal number, so that a
// hidden score, -infinity, stays that.  Where that is above the product (a scale
// of 0 among them) it takes sums of queries times codes of 2^100 to show.
__device__ __forceinline__ float score_scale(const AttnArgs& a, float ks) {
  return __builtin_fmaxf(page_scale_of(ks) * a.scale2, 0x1p-126f);
}

// Over lanes l and l ^ 16, and l and l ^ 32 (gfx950 swaps rows and halves of
// two registers in one instruction each, without LDS).
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u32x2 swap16(float v) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false));
}
__device__ __forceinline__ u32x2 swap32(float v) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false));
}
__device__ __forceinline__ float max16(float v) {
  const u32x2 w = swap16(v);
  return __builtin_fmaxf(__uint_as_float(w[0]), __uint_as_float(w[1]));
}
__device__ __forceinline__ float max32(float v) {
  const u32x2 w = swap32(v);
  return __builtin_fmaxf(__uint_as_float(w[0]), __uint_as_float(w[1]));
}
__device__ __forceinline__ float sum16(float v) {
  const u32x2 w = swap16(v);
  return __uint_as_float(w[0]) + __uint_as_float(w[1]);
}
__device__ __forceinline__ float sum32(float v) {
  const u32x2 w = swap32(v);
  return __uint_as_float(w[0]) + __uint_as_float(w[1]);
}

// The running m is put kMaxLow (in powers of two) below the maximum, and
// replaced only when a score passes it by kMaxSlack: until then neither the
// maximum over lanes nor the accumulators' scaling is needed, and x stays below
// fp16's largest value.
constexpr float kMaxLow = 7.0f, kMaxSlack = 15.0f;

// w with its bytes before `skip` and from n on zeroed.
__device__ __forceinline__ i32x4 keep_bytes(i32x4 w, int skip, int n) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int a = skip - 4 * j, b = n - 4 * j;
    const uint32_t lo = a <= 0 ? 0xffffffffu : (a >= 4 ? 0u : ~((1u << (8 * a)) - 1u));
    const uint32_t hi = b >= 4 ? 0xffffffffu : (b <= 0 ? 0u : (1u << (8 * b)) - 1u);
    w[j] &= (int)(lo & hi);
  }
  return w;
}

// The lane's values of a query row as KC B operands of 8 values and NS bf16
// terms each (zeros where the row is not live, or past the head): first every
// load, then, once other loads are on their way too, the operands.  Values come
// in 16s, STEP apart, from d0 on.
template <int STEP>
constexpr int q_place(int d0, int c) {
  return d0 + STEP * (c >> 1) + 8 * (c & 1);
}
template <int KC, int NS>
struct QueryRaw {
  i32x4 w[KC][NS == 1 ? 1 : 2];
};

template <int STEP, int KC, int NS>
__device__ __forceinline__ void load_q(const AttnArgs& a, size_t row, int d0, QueryRaw<KC, NS>& raw) {
#pragma unroll
  for (int c = 0; c < KC; ++c) {
    const int d = q_place<STEP>(d0, c);
    const size_t at = row + (d < a.c.D ? d : 0);
#pragma unroll
    for (int k = 0; k < (NS == 1 ? 1 : 2); ++k)
      raw.w[c][k] = NS == 1 ? ld16(reinterpret_cast<const uint16_t*>(a.q) + at)
                            : ld16(reinterpret_cast<const float*>(a.q) + at + 4 * k);
  }
}

template <int STEP, int KC, int NS>
__device__ __forceinline__ void make_q(const AttnArgs& a, const QueryRaw<KC, NS>& raw, int d0, bool live,
                                       bf16x8 out[KC][NS]) {
  const int sign = a.neg ? (NS == 1 ? (int)0x80008000 : (int)0x80000000) : 0;
#pragma unroll
  for (int c = 0; c < KC; ++c) {
    const bool use = live && q_place<STEP>(d0, c) < a.c.D;
    if (NS == 1) {
      i32x4 w = raw.w[c][0];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = use ? w[j] ^ sign : 0;
      out[c][0] = as_bf16x8(w);
    } else {
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = use ? __int_as_float(raw.w[c][j >> 2][j & 3] ^ sign) : 0.0f;
      split_bf16<NS>(x, out[c]);
    }
  }
}

// Scores of a lane's 16 tokens t.. of one row: -infinity where the row does
// not see the token (outside [lo, hi), or all if gone).
__device__ __forceinline__ void attn_hide(f32x16& sc, bool gone, int t, int lo, int hi) {
  const int off = t - lo;
  const unsigned n = gone || hi <= lo ? 0u : (unsigned)(hi - lo);
#pragma unroll
  for (int k = 0; k < 16; ++k) sc[k] = (unsigned)(off + k) < n ? sc[k] : -__builtin_inff();
}

__device__ __forceinline__ float attn_top(const f32x16& sc) {
  float v = sc[0];
#pragma unroll
  for (int k = 1; k < 16; ++k) v = __builtin_fmaxf(v, sc[k]);
  return v;
}

// x = exp2(s f + c), c = log2 vs - m, of a lane's 16 tokens, as operands;
// returns their sum.  The lane's tokens lie in one page, so f and vs are the
// lane's, and dividing the sum by vs once gives that of exp2(s f - m).
template <int NS>
__device__ __forceinline__ float attn_probs(const f32x16& sc, float f, float c, bf16x8 p[2][NS]) {
  float x[16], sum = 0.0f;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    x[k] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[k], f, c));
    sum += x[k];
  }
  if (NS > 1) {
    split_bf16<NS>(x, p[0]);
    split_bf16<NS>(x + 8, p[1]);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      i32x4 w;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = __builtin_bit_cast(
            int, __builtin_convertvector((f32x2_t{x[8 * h + 2 * k], x[8 * h + 2 * k + 1]}), f16x2_t));
      p[h][0] = as_bf16x8(w);
    }
  }
  return sum;
}

// Sum of exp2(s f - m) of a lane's 16 tokens by itself, for tiles with values of
// a scale below 2^kLowScale (an append of zeros leaves 2^-64): beside values of
// a scale of 2^48, m is up to 2^41 of the largest weight, and such a token's x
// is under fp32's smallest number from a weight of 2^-21 of it on.  From
// kLowScale on that takes a weight of 2^-45.
constexpr float kLowScale = -40.0f;
__device__ __forceinline__ float attn_weights(const f32x16& sc, float f, float m) {
  float sum = 0.0f;
#pragma unroll
  for (int k = 0; k < 16; ++k) sum += __builtin_amdgcn_exp2f(__builtin_fmaf(sc[k], f, -m));
  return sum;
}

// l 2^-below, in two steps: where m rises from values of the smallest scale to
// some of the largest, 2^-below is no fp32 number but l 2^-below is.
__device__ __forceinline__ float attn_lower(float l, float below) {
  const float half = __builtin_amdgcn_exp2f(-0.5f * below);
  return l * half * half;
}

// Four values of a row's output from its sums o and l.
template <int NS>
__device__ __forceinline__ void attn_store4(const AttnArgs& a, size_t row, int d, const float o[4], float l) {
  const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
  if (NS == 1) {
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) + row * a.c.D + d) =
        make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
  } else {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + row * a.c.D + d) =
        make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
  }
}

__device__ __forceinline__ float attn_lse(float m, float l) {
  return l == 0.0f ? -__builtin_inff() : kLn2 * (m + __builtin_log2f(l));
}

}  // namespace moe
