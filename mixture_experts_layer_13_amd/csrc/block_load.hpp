// block_load.hpp -- direct-to-LDS loads and waits of the block-scaled products.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "block_gemm.hpp"

namespace moe {

// f(0), f(1), .. f(B - 1), as constants.
template <int A, int B, class F>
__device__ __forceinline__ void b_for(F&& f) {
  if constexpr (A < B) {
    f(std::integral_constant<int, A>{});
    b_for<A + 1, B>(f);
  }
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t b_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}
constexpr int kPastCaches = 2;  // non-temporal
template <int AUX = 0>
__device__ __forceinline__ void b_dma16(__amdgpu_buffer_rsrc_t r, char* dst, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)dst, 16, voff, soff, 0, AUX);
}
__device__ __forceinline__ void b_dma4(__amdgpu_buffer_rsrc_t r, char* dst, uint32_t voff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)dst, 4, voff, 0, 0, 0);
}

constexpr uint32_t kNowhere = 0x80000000u;  // past every buffer here: such a load gives zeros
// A buffer whose loads are all inside what it stands for (not all ones: a choice
// between those and nothing is made lane by lane, and the load looped over).  The
// farthest are a gathered call's scales: a_rows times their stride is below 2^29.
constexpr uint32_t kMost = 0x7ffffffcu;
static_assert(4 * kMostScales <= kMost && kMost < kNowhere, "a row's scale may lie that far");

template <int N>
__device__ __forceinline__ void b_wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt is six bits");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}
// Barrier behind this wave's own LDS reads.
__device__ __forceinline__ void b_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4) | (0 << 8));  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

}  // namespace moe
