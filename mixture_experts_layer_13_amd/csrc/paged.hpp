// paged.hpp -- the paged E4M3 key/value cache and the batch description that
// kv_append.hip and the attention kernels share, and the search that turns a
// workgroup's place in the flattened work of a ragged batch into a sequence.
#pragma once

#include "common.hpp"

namespace moe {

// Codes of keys [pages][H][S][D] and of values [pages][H][S/16][D][16]: a
// value block holds 16 tokens channel by channel, so that a lane reads the 16
// tokens of a channel, the contraction of the second attention product, as
// one 16-byte load; the append transposes once what every later step reads.
// One fp32 scale per page and head each.
struct PagedArgs {
  uint8_t *kc, *vc;
  float *ks, *vs;
  int pages, lS, H, D;  // page size S = 1 << lS
};

// Bounds of a page's scale.
constexpr float kMinPageScale = 0x1p-64f, kMaxPageScale = 0x1p+48f;

struct BatchArgs {
  const int32_t* cu_q;     // [B + 1] first query row of each sequence, or NULL (row b)
  const int32_t* kv_lens;  // [B] cached tokens, the queries' own among them
  const int32_t* table;    // [B][max_pages]
  int B, max_pages, T;
};

// Sequence b: rows [q0, q0 + q) of the packed batch; row i stands at token
// kv - q + i; tokens [0, lim) lie in the table.  Row offsets are clamped to
// [0, T] and lim to what the table can hold, so no value read here leads
// outside the caller's buffers.
struct Seq {
  int q0, q, kv, lim;
};

__device__ __forceinline__ Seq load_seq(const BatchArgs& a, int lS, int b) {
  Seq s;
  if (a.cu_q) {
    int lo = a.cu_q[b], hi = a.cu_q[b + 1];
    lo = lo < 0 ? 0 : (lo > a.T ? a.T : lo);
    hi = hi < lo ? lo : (hi > a.T ? a.T : hi);
    s.q0 = lo;
    s.q = hi - lo;
  } else {
    s.q0 = b;
    s.q = 1;
  }
  const int cap = a.max_pages << lS;  // at most 2^30
  const int kv = a.kv_lens[b];
  s.kv = kv < 0 ? 0 : kv;
  s.lim = s.kv < cap ? s.kv : cap;
  return s;
}

// Inclusive prefix sum over the workgroup's threads (WAVES waves; 0: as many
// as the launch has); *total the whole sum.  scratch: one int per wave in LDS.
// Ends with a barrier, so that it can be called again at once.
template <int WAVES>
__device__ __forceinline__ int block_scan(int v, int* scratch, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = WAVES ? WAVES : (int)blockDim.x >> 6;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int up = __shfl_up(v, o, 64);
    if (lane >= o) v += up;
  }
  if (lane == 63) scratch[wave] = v;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < waves; ++w) {
    const int x = scratch[w];
    before += w < wave ? x : 0;
    all += x;
  }
  __syncthreads();
  *total = all;
  return v + before;
}

}  // namespace moe
