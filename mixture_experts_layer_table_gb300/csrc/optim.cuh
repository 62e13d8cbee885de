// Tensor tables of the optimizer kernels (internal to the library).  A launch takes its tensors in
// its kernel parameters, so that a step reads no table from device memory and needs no copy before it.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace mok {

struct AdamTensor {
  void* param;
  float* master;
  const void* grad;
  void* m;
  void* v;
  uint8_t* m_scale;
  uint8_t* v_scale;
  int64_t n;
  uint64_t counter;  // element counter of the rounding bits, of element 0 (a multiple of 8)
  float lr, weight_decay;
};

struct AdamHyper {
  float beta1, one_minus_beta1, beta2, one_minus_beta2, eps;
  float beta2_sqrt, one_minus_beta2_sqrt;  // square roots of beta2 and 1 - beta2
  float inv_bc1;       // 1 / (1 - beta1^t)
  float inv_bc2_sqrt;  // 1 / sqrt(1 - beta2^t)
  uint32_t seed;
};

struct GradTensor {
  const void* grad;
  int64_t n;
  int32_t bf16;
};

// Kinds of one launch: every tensor of it has the same three.
enum ParamKind { PARAM_F32 = 0, PARAM_BF16_MASTER = 1, PARAM_BF16 = 2 };
enum GradKind { GRAD_F32 = 0, GRAD_BF16 = 1 };
enum StateKind { STATE_F32 = 0, STATE_MX8 = 1 };

// Most tensors of one launch: the table and its chunk starts fit the kernel's parameters (32,764 bytes).
constexpr int OPTIM_TABLE = 256;
// grad_norm's workspace: a ticket (zero between calls), then one f32 sum per block of the call.
constexpr int NORM_MAX_PARTIALS = 4096;
constexpr int NORM_PARTIALS_OFFSET = 256;
constexpr int NORM_WS_BYTES = NORM_PARTIALS_OFFSET + NORM_MAX_PARTIALS * 4;

cudaError_t launch_adamw(const AdamTensor* tensors, int count, int param, int grad, int state, const AdamHyper& h,
                         const float* grad_scale, int n_sm, cudaStream_t st);
// One launch of a call: blocks first_block .. first_block + blocks - 1 of total_blocks; the last block of
// the call writes out = {norm, scale}.
cudaError_t launch_grad_norm(const GradTensor* tensors, int count, int blocks, int first_block, int total_blocks,
                             float max_norm, float* out, void* ws, cudaStream_t st);
int64_t grad_norm_chunks(int64_t n);

}  // namespace mok
