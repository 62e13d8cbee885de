// Launchers of the E4M3 operators with a scale for each block of 128 (include/mok.h): quantisers, the grouped
// product and its weight gradient.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

namespace mok {

constexpr int FP8_BLOCK = 128;
constexpr int FP8_MAX_E = 1024;
// The least that a block's largest magnitude counts as, 2^-110, and the scale that comes of it: of a block of zeros.
constexpr float FP8_LEAST = 7.703719777548943e-34f, FP8_LEAST_SCALE = (float)(7.703719777548943e-34 / 448);

enum Fp8Source { FP8_PLAIN = 0, FP8_SWIGLU = 1, FP8_SWIGLU_GRAD = 2 };

struct Fp8QuantizeArgs {
  int64_t R, C, T;                 // rows, width of the quantised rows, tokens (gathered source)
  int64_t x_stride, grad_stride;   // elements
  int64_t q_stride, scale_stride;  // bytes, floats
  int64_t qt_stride;               // bytes
  int E, k;
  const void* x;
  const void* grad;
  const int32_t* src_of;
  const float* gates;
  const int32_t* offsets;  // [E+1] (columns)
  uint8_t* q;
  float* scale;
  uint8_t* qt;
  float* qt_scale;
  int* status;
};

struct Fp8WeightsArgs {
  int64_t N, K, q_stride, qt_stride;
  int E;
  const void* w;
  uint8_t* q;
  float* scale;
  uint8_t* qt;
  float* qt_scale;
};

struct Fp8MatmulArgs {
  int64_t R, N, K;
  int64_t x_stride, w_stride, x_scale_stride, out_stride;  // bytes, bytes, floats, elements
  int E;
  const uint8_t* x;
  const float* x_scale;
  const uint8_t* w;
  const float* w_scale;
  const int32_t* offsets;  // [E+1], or null: one group of all rows
  void* out;
  int* status;
};

struct Fp8WeightGradArgs {
  int64_t R, N, H;
  int64_t dy_stride, x_stride;  // bytes
  int E;
  const uint8_t* dy;  // [N][P]
  const float* dy_scale;
  const uint8_t* x;   // [H][P]
  const float* x_scale;
  const int32_t* offsets;
  void* out;  // [E][N][H]
  int* status;
};

cudaError_t launch_fp8_quantize(const Fp8QuantizeArgs& a, int source, bool bf16, int n_sm, cudaStream_t st);
cudaError_t launch_fp8_weights(const Fp8WeightsArgs& a, bool bf16, cudaStream_t st);
cudaError_t launch_fp8_matmul(const Fp8MatmulArgs& a, bool bf16_out, int n_sm, cudaStream_t st);
cudaError_t launch_fp8_weight_grad(const Fp8WeightGradArgs& a, bool bf16_out, int n_sm, cudaStream_t st);

// An end of a group's rows as the kernels take it: in [least, R], with least 0 for the first row and the first row for
// the end, so that a table that is wrong reads and writes nothing outside the tensors.
__device__ __forceinline__ int fp8_offset(int32_t v, int least, int64_t R) {
  const int r = v < least ? least : v;
  return r > R ? (int)R : r;
}

}  // namespace mok
