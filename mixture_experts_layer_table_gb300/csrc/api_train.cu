// C ABI of the training step around the layer (include/mok.h): argument checks and launches of the
// group-limited routing and its backward, the gradient norm and the AdamW step.  As for the layer: no allocation, no host synchronisation, every
// kernel enqueued on the caller's stream.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "api_common.h"
#include "mok.h"
#include "optim.cuh"
#include "router.cuh"

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

mok_status check_route(const mok_route_desc* d) {
  if (d == nullptr || d->T < 0 || d->E < 1 || d->k < 1 || d->reserved != 0) return MOK_ERR_INVALID_ARG;
  if (d->router != MOK_ROUTER_SOFTMAX && d->router != MOK_ROUTER_SIGMOID) return MOK_ERR_INVALID_ARG;
  if (d->group_score != MOK_GROUP_MAX && d->group_score != MOK_GROUP_TOP2) return MOK_ERR_INVALID_ARG;
  if (!elem_type(d->logits_type)) return MOK_ERR_INVALID_ARG;
  if (!std::isfinite(d->route_scale) || !std::isfinite(d->balance_coef) || !std::isfinite(d->bias_rate))
    return MOK_ERR_INVALID_ARG;
  if (d->logits_stride != 0 && d->logits_stride < d->E) return MOK_ERR_INVALID_ARG;
  if (d->n_group < 1 || d->E % d->n_group != 0 || d->topk_group < 1 || d->topk_group > d->n_group)
    return MOK_ERR_INVALID_ARG;
  if (d->k > (int64_t)d->topk_group * (d->E / d->n_group)) return MOK_ERR_INVALID_ARG;
  if (d->E > mok::ROUTE_MAX_E || d->k > mok::ROUTE_MAX_K || d->n_group > mok::ROUTE_MAX_GROUPS)
    return MOK_ERR_UNSUPPORTED;
  return MOK_OK;
}

int param_kind(const mok_adamw_tensor& t) {
  if (t.param_type == MOK_ELEM_F32) return mok::PARAM_F32;
  return t.master != nullptr ? mok::PARAM_BF16_MASTER : mok::PARAM_BF16;
}

}  // namespace

extern "C" {

mok_status mok_route(const mok_route_desc* d, const void* logits, const float* bias, int32_t* topk_idx, float* gates,
                     float* scores, int32_t* counts, float* prob_sum, float* loss, float* dprob, float* bias_next,
                     void* ws, size_t ws_bytes, void* stream) {
  static_assert(MOK_ROUTE_WS_BYTES >= mok::ROUTE_WS_BYTES, "workspace of mok_route");
  mok_status s = check_route(d);
  if (s != MOK_OK) return s;
  if (d->T > 0 && (!logits || !topk_idx)) return MOK_ERR_INVALID_ARG;
  if (!aligned_elem(logits, d->logits_type)) return MOK_ERR_INVALID_ARG;
  const void* words[] = {bias, topk_idx, gates, scores, counts, prob_sum, loss, dprob, bias_next};
  for (const void* p : words)
    if (!aligned_elem(p, MOK_ELEM_F32)) return MOK_ERR_INVALID_ARG;
  if (bias_next != nullptr && bias == nullptr) return MOK_ERR_INVALID_ARG;
  mok::RouteArgs a = {};
  a.counts = counts;
  a.prob_sum = prob_sum;
  a.loss = loss;
  a.dprob = dprob;
  a.bias_next = bias_next;
  if (mok::route_balances(a)) {
    if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return MOK_ERR_INVALID_ARG;
    if (ws_bytes < (size_t)MOK_ROUTE_WS_BYTES) return MOK_ERR_WORKSPACE_TOO_SMALL;
    if (d->T >= (int64_t(1) << 31)) return MOK_ERR_UNSUPPORTED;
    char* base = static_cast<char*>(ws);
    a.ticket = reinterpret_cast<unsigned*>(base);
    a.not_finite = a.ticket + 1;
    a.acc_prob = reinterpret_cast<unsigned long long*>(base + mok::ROUTE_WS_SUMS);
    a.acc_counts = reinterpret_cast<int32_t*>(base + mok::ROUTE_WS_COUNTS);
  } else if (d->T == 0) {
    return MOK_OK;
  }
  a.logits = logits;
  a.bias = bias;
  a.T = d->T;
  a.stride = d->logits_stride != 0 ? d->logits_stride : d->E;
  a.E = d->E;
  a.k = d->k;
  a.router = d->router;
  a.renorm = d->renorm;
  a.scale = d->route_scale;
  a.n_group = d->n_group;
  a.topk_group = d->topk_group;
  a.group_top2 = d->group_score == MOK_GROUP_TOP2;
  a.topk_idx = topk_idx;
  a.gates = gates;
  a.scores = scores;
  a.dprob_unit = d->T == 0 ? 0.0f : (float)(d->balance_coef * (double)d->E / ((double)d->k * (double)d->T * (double)d->T));
  a.bias_rate = d->bias_rate;
  // a sum of T probabilities of at most 1 stays below 2^62 units
  int bits = 0;
  while ((d->T >> bits) != 0) ++bits;
  a.sum_shift = std::min(52, 62 - bits);
  const int n_sm = sm_count();
  if (n_sm <= 0) return MOK_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  MOK_LAUNCH("route", st, mok::launch_route(a, d->logits_type == MOK_ELEM_BF16, n_sm, st));
  return MOK_OK;
}

mok_status mok_route_backward(const mok_route_desc* d, const void* logits, const int32_t* topk_idx, const float* dgates,
                              const float* dprob, void* dlogits, int64_t dlogits_stride, int32_t* device_status,
                              void* stream) {
  mok_status s = check_route(d);
  if (s != MOK_OK) return s;
  if (dlogits_stride != 0 && dlogits_stride < d->E) return MOK_ERR_INVALID_ARG;
  if (!aligned_elem(logits, d->logits_type) || !aligned_elem(dlogits, d->logits_type)) return MOK_ERR_INVALID_ARG;
  const void* words[] = {topk_idx, dgates, dprob, device_status};
  for (const void* p : words)
    if (!aligned_elem(p, MOK_ELEM_F32)) return MOK_ERR_INVALID_ARG;
  if (d->T == 0) return MOK_OK;
  if ((dgates == nullptr && dprob == nullptr) || (dgates != nullptr && topk_idx == nullptr)) return MOK_ERR_INVALID_ARG;
  if (!logits || !dlogits) return MOK_ERR_INVALID_ARG;
  mok::RouteBackwardArgs a = {};
  a.logits = logits;
  a.T = d->T;
  a.stride = d->logits_stride != 0 ? d->logits_stride : d->E;
  a.out_stride = dlogits_stride != 0 ? dlogits_stride : d->E;
  a.E = d->E;
  a.k = d->k;
  a.router = d->router;
  a.renorm = d->renorm;
  a.scale = d->route_scale;
  a.topk_idx = topk_idx;
  a.dgates = dgates;
  a.dprob = dprob;
  a.dlogits = dlogits;
  a.status = device_status;
  const int n_sm = sm_count();
  if (n_sm <= 0) return MOK_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  MOK_LAUNCH("route_backward", st, mok::launch_route_backward(a, d->logits_type == MOK_ELEM_BF16, n_sm, st));
  return MOK_OK;
}

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
  unsigned kinds = 0;  // bit kind_of(t) of every kind of tensor there is
  auto kind_of = [](const mok_adamw_tensor& t) { return (param_kind(t) * 2 + t.grad_type) * 2 + t.state_type; };
  for (int32_t i = 0; i < count; ++i) {
    const mok_status s = check_adamw(tensors[i]);
    if (s != MOK_OK) return s;
    if (tensors[i].n > 0) kinds |= 1u << kind_of(tensors[i]);
  }
  const int n_sm = sm_count();
  if (n_sm <= 0) return MOK_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  mok::AdamHyper h;
  h.beta1 = (float)hyper->beta1;
  h.one_minus_beta1 = (float)(1.0 - hyper->beta1);
  h.beta2 = (float)hyper->beta2;
  h.one_minus_beta2 = (float)(1.0 - hyper->beta2);
  h.beta2_sqrt = (float)std::sqrt(hyper->beta2);
  h.one_minus_beta2_sqrt = (float)std::sqrt(1.0 - hyper->beta2);
  h.eps = (float)hyper->eps;
  h.inv_bc1 = (float)(1.0 / (1.0 - std::pow(hyper->beta1, (double)hyper->step)));
  h.inv_bc2_sqrt = (float)(1.0 / std::sqrt(1.0 - std::pow(hyper->beta2, (double)hyper->step)));
  h.seed = hyper->seed ^ ((uint32_t)hyper->step * 0x9E3779B1u);
  // tensors of one kind share a launch
  for (int kind = 0; kind < 12; ++kind) {
    if (!(kinds >> kind & 1u)) continue;
    mok::AdamTensor part[mok::OPTIM_TABLE];
    int n = 0;
    for (int32_t i = 0; i < count; ++i) {
      const mok_adamw_tensor& t = tensors[i];
      if (t.n > 0 && kind_of(t) == kind)
        part[n++] = {t.param, t.master, t.grad, t.m, t.v, t.m_scale, t.v_scale, t.n, t.counter, t.lr, t.weight_decay};
      if (n == mok::OPTIM_TABLE || (n > 0 && i == count - 1)) {
        MOK_LAUNCH("adamw", st,
                   mok::launch_adamw(part, n, kind / 4, kind / 2 % 2, kind % 2, h, grad_scale, n_sm, st));
        n = 0;
      }
    }
  }
  return MOK_OK;
}

}  // extern "C"
