// permute.hpp -- arguments of the dispatch and combine kernels (permute.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// Strides in elements.  Scatter reads tok_in and writes rows_out; gather reads
// rows_in and writes tok_out; with dw (the weights' gradient) scatter reads
// rows_in too, and gather tok_in.
struct PermuteArgs {
  const int32_t* sorted_ids;
  const int32_t* pair_pos;
  const int32_t* num_padded;
  int M, topk, P, rows, K;
  const void* tok_in;
  const void* rows_in;
  void* tok_out;
  void* rows_out;
  long long tok_in_stride, rows_in_stride, tok_out_stride, rows_out_stride;
  const float* weights;  // or NULL: 1
  float* dw;             // or NULL
};

int launch_scatter(const PermuteArgs& a, int tok_type, int rows_type, hipStream_t st);
int launch_gather(const PermuteArgs& a, int tok_type, int rows_type, hipStream_t st);

}  // namespace moe
