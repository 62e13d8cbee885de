// C ABI of the training step around the layer (include/mok.h): argument checks and launches of the
// gradient norm and the AdamW step.  As for the layer: no allocation, no host synchronisation, every
// kernel enqueued on the caller's stream.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "api_common.h"
#include "mok.h"
#include "optim.cuh"

using namespace mok_api;

namespace {

bool elem_type(int32_t t) { return t == MOK_ELEM_F32 || t == MOK_ELEM_BF16; }
bool aligned_elem(const void* p, int32_t type) {
  return (reinterpret_cast<uintptr_t>(p) & (type == MOK_ELEM_F32 ? 3u : 1u)) == 0;
}

mok_status check_adamw(const mok_adamw_tensor& t) {
  if (t.n < 0 || !elem_type(t.param_type) || !elem_type(t.grad_type) || t.reserved != 0) return MOK_ERR_INVALID_ARG;
  if (t.state_type != MOK_STATE_F32 && t.state_type != MOK_STATE_MX8) return MOK_ERR_INVALID_ARG;
  if (!std::isfinite(t.lr) || !std::isfinite(t.weight_decay)) return MOK_ERR_INVALID_ARG;
  if (t.counter % 8 != 0) return MOK_ERR_INVALID_ARG;
  if (t.master != nullptr && t.param_type != MOK_ELEM_BF16) return MOK_ERR_INVALID_ARG;
  const bool mx8 = t.state_type == MOK_STATE_MX8;
  if (!mx8 && (t.m_scale != nullptr || t.v_scale != nullptr)) return MOK_ERR_INVALID_ARG;
  if (t.n == 0) return MOK_OK;
  if (!t.param || !t.grad || !t.m || !t.v || (mx8 && (!t.m_scale || !t.v_scale))) return MOK_ERR_INVALID_ARG;
  if (!aligned_elem(t.param, t.param_type) || !aligned_elem(t.grad, t.grad_type) ||
      !aligned_elem(t.master, MOK_ELEM_F32))
    return MOK_ERR_INVALID_ARG;
  if (!mx8 && (!aligned_elem(t.m, MOK_ELEM_F32) || !aligned_elem(t.v, MOK_ELEM_F32))) return MOK_ERR_INVALID_ARG;
  return MOK_OK;
}

int param_kind(const mok_adamw_tensor& t) {
  if (t.param_type == MOK_ELEM_F32) return mok::PARAM_F32;
  return t.master != nullptr ? mok::PARAM_BF16_MASTER : mok::PARAM_BF16;
}

}  // namespace

extern "C" {

mok_status mok_grad_norm(const mok_grad_tensor* tensors, int32_t count, float max_norm, float* out, void* ws,
                         size_t ws_bytes, void* stream) {
  static_assert(MOK_GRAD_NORM_WS_BYTES >= mok::NORM_WS_BYTES, "workspace of mok_grad_norm");
  if (count < 0 || (count > 0 && tensors == nullptr) || out == nullptr || ws == nullptr) return MOK_ERR_INVALID_ARG;
  if (!(max_norm > 0.0f) || !aligned16(ws) || !aligned_elem(out, MOK_ELEM_F32)) return MOK_ERR_INVALID_ARG;
  for (int32_t i = 0; i < count; ++i) {
    const mok_grad_tensor& t = tensors[i];
    if (t.n < 0 || !elem_type(t.grad_type) || t.reserved != 0) return MOK_ERR_INVALID_ARG;
    if (t.n > 0 && (t.grad == nullptr || !aligned_elem(t.grad, t.grad_type))) return MOK_ERR_INVALID_ARG;
  }
  if (ws_bytes < (size_t)MOK_GRAD_NORM_WS_BYTES) return MOK_ERR_WORKSPACE_TOO_SMALL;
  const int n_sm = sm_count();
  if (n_sm <= 0) return MOK_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // one launch for each OPTIM_TABLE tensors; each adds its blocks to the call's ticket
  const int launches = std::max(1, (count + mok::OPTIM_TABLE - 1) / mok::OPTIM_TABLE);
  if (launches > mok::NORM_MAX_PARTIALS) return MOK_ERR_UNSUPPORTED;
  const int64_t most = std::min<int64_t>(4 * n_sm, mok::NORM_MAX_PARTIALS / launches);
  auto blocks_of = [&](int l) {
    int64_t chunks = 0;
    for (int i = l * mok::OPTIM_TABLE; i < std::min(count, (l + 1) * mok::OPTIM_TABLE); ++i)
      chunks += mok::grad_norm_chunks(tensors[i].n);
    return (int)std::max<int64_t>(1, std::min(chunks, most));
  };
  int total = 0, first = 0;
  for (int l = 0; l < launches; ++l) total += blocks_of(l);
  for (int l = 0; l < launches; ++l) {
    mok::GradTensor part[mok::OPTIM_TABLE];
    int n = 0;
    for (int i = l * mok::OPTIM_TABLE; i < std::min(count, (l + 1) * mok::OPTIM_TABLE); ++i)
      part[n++] = {tensors[i].grad, tensors[i].n, tensors[i].grad_type == MOK_ELEM_BF16};
    const int blocks = blocks_of(l);
    MOK_LAUNCH("grad_norm", st, mok::launch_grad_norm(part, n, blocks, first, total, max_norm, out, ws, st));
    first += blocks;
  }
  return MOK_OK;
}

mok_status mok_adamw_step(const mok_adamw_tensor* tensors, int32_t count, const mok_adamw_hyper* hyper,
                          const float* grad_scale, void* stream) {
  if (count < 0 || (count > 0 && tensors == nullptr) || hyper == nullptr) return MOK_ERR_INVALID_ARG;
  if (!(hyper->beta1 >= 0.0 && hyper->beta1 < 1.0) || !(hyper->beta2 >= 0.0 && hyper->beta2 < 1.0) ||
      !(hyper->eps >= 0.0) || !std::isfinite(hyper->eps) || hyper->step < 1 || hyper->reserved != 0)
    return MOK_ERR_INVALID_ARG;
  if (!aligned_elem(grad_scale, MOK_ELEM_F32)) return MOK_ERR_INVALID_ARG;
  for (int32_t i = 0; i < count; ++i) {
    const mok_status s = check_adamw(tensors[i]);
    if (s != MOK_OK) return s;
  }
  const int n_sm = sm_count();
  if (n_sm <= 0) return MOK_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  mok::AdamHyper h;
  h.beta1 = (float)hyper->beta1;
  h.one_minus_beta1 = (float)(1.0 - hyper->beta1);
  h.beta2 = (float)hyper->beta2;
  h.one_minus_beta2 = (float)(1.0 - hyper->beta2);
  h.eps = (float)hyper->eps;
  h.inv_bc1 = (float)(1.0 / (1.0 - std::pow(hyper->beta1, (double)hyper->step)));
  h.inv_bc2_sqrt = (float)(1.0 / std::sqrt(1.0 - std::pow(hyper->beta2, (double)hyper->step)));
  h.seed = hyper->seed ^ ((uint32_t)hyper->step * 0x9E3779B1u);
  // tensors of the same kinds share a launch
  for (int param = 0; param < 3; ++param) {
    for (int grad = 0; grad < 2; ++grad) {
      for (int state = 0; state < 2; ++state) {
        mok::AdamTensor part[mok::OPTIM_TABLE];
        int n = 0;
        auto flush = [&]() -> mok_status {
          if (n > 0) MOK_LAUNCH("adamw", st, mok::launch_adamw(part, n, param, grad, state, h, grad_scale, n_sm, st));
          n = 0;
          return MOK_OK;
        };
        for (int32_t i = 0; i < count; ++i) {
          const mok_adamw_tensor& t = tensors[i];
          if (t.n == 0 || param_kind(t) != param || t.grad_type != grad || t.state_type != state) continue;
          part[n++] = {t.param, t.master, t.grad, t.m, t.v, t.m_scale, t.v_scale, t.n, t.counter, t.lr, t.weight_decay};
          if (n == mok::OPTIM_TABLE) {
            const mok_status s = flush();
            if (s != MOK_OK) return s;
          }
        }
        const mok_status s = flush();
        if (s != MOK_OK) return s;
      }
    }
  }
  return MOK_OK;
}

}  // extern "C"
