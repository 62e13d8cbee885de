// Launchers of the row movement by a schedule table outside the layer, and of the E4M3 quantisers and
// products with a scale for each block of 128 (include/mok.h).
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

namespace mok {

constexpr int ROWS_MAX_K = 16;

struct RowsArgs {
  int64_t T, R, H, token_stride, row_stride;  // strides in elements
  int k;
  const int32_t* index;  // src_of [R] or row_of [T k]
  const float* gates;    // [T][k] or null
  const void* tokens;    // x or dy
  const void* rows;      // o
  void* out;             // x_g, y or do
  float* dgates;
  int* status;
};

cudaError_t launch_expert_gather(const RowsArgs& a, bool bf16, cudaStream_t st);
cudaError_t launch_expert_merge(const RowsArgs& a, bool bf16, cudaStream_t st);
cudaError_t launch_expert_merge_backward(const RowsArgs& a, bool bf16, int n_sm, cudaStream_t st);

}  // namespace mok
