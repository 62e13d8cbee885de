// C ABI of the operators for experts outside the layer (include/mok.h): argument checks and launches of the row
// movement by a schedule table, and of the E4M3 quantisers and products with a scale for each block of 128.  As for
// the layer: no allocation, no host synchronisation, every kernel enqueued on the caller's stream.
#include <cuda_runtime.h>

#include <initializer_list>

#include "api_common.h"
#include "expert_rows.cuh"
#include "fp8.cuh"
#include "mok.h"

using namespace mok_api;

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 31;  // rows, widths and assignments stay below
constexpr int64_t kMaxWidth = int64_t(1) << 28;

bool elem_type(int32_t t) { return t == MOK_ELEM_F32 || t == MOK_ELEM_BF16; }
bool aligned_to(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool aligned_elem(const void* p, int32_t type) { return aligned_to(p, type == MOK_ELEM_F32 ? 4 : 2); }
// 0 stands for `packed`, any other stride holds at least `width`
bool stride_ok(int64_t stride, int64_t width) { return stride == 0 || stride >= width; }
bool byte_stride_ok(int64_t stride, int64_t width) { return stride_ok(stride, width) && stride % 16 == 0; }
int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }

mok_status check_rows(const mok_rows_desc* d) {
  if (d == nullptr || d->T < 0 || d->R < 0 || d->H < 1 || d->k < 1 || !elem_type(d->type)) return MOK_ERR_INVALID_ARG;
  if (!stride_ok(d->token_stride, d->H) || !stride_ok(d->row_stride, d->H)) return MOK_ERR_INVALID_ARG;
  if (d->k > mok::ROWS_MAX_K || d->R >= kMaxRows || d->T >= kMaxRows / d->k || d->H >= kMaxWidth)
    return MOK_ERR_UNSUPPORTED;
  return MOK_OK;
}

mok::RowsArgs rows_args(const mok_rows_desc* d, const int32_t* index, const float* gates, int32_t* device_status) {
  mok::RowsArgs a = {};
  a.T = d->T;
  a.R = d->R;
  a.H = d->H;
  a.token_stride = d->token_stride != 0 ? d->token_stride : d->H;
  a.row_stride = d->row_stride != 0 ? d->row_stride : d->H;
  a.k = d->k;
  a.index = index;
  a.gates = gates;
  a.status = device_status;
  return a;
}

bool words_aligned(std::initializer_list<const void*> words) {
  for (const void* p : words)
    if (!aligned_to(p, 4)) return false;
  return true;
}

}  // namespace

extern "C" {

mok_status mok_gather_rows(const mok_rows_desc* d, const void* x, const int32_t* src_of, const float* gates, void* x_g,
                           int32_t* device_status, void* stream) {
  const mok_status s = check_rows(d);
  if (s != MOK_OK) return s;
  if (!aligned_elem(x, d->type) || !aligned_elem(x_g, d->type) || !words_aligned({src_of, gates, device_status}))
    return MOK_ERR_INVALID_ARG;
  if (d->R == 0) return MOK_OK;
  if (!src_of || !x_g || (d->T > 0 && !x)) return MOK_ERR_INVALID_ARG;
  mok::RowsArgs a = rows_args(d, src_of, gates, device_status);
  a.tokens = x;
  a.out = x_g;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  MOK_LAUNCH("expert_gather", st, mok::launch_expert_gather(a, d->type == MOK_ELEM_BF16, st));
  return MOK_OK;
}

mok_status mok_merge_rows(const mok_rows_desc* d, const void* o, const int32_t* row_of, const float* gates, void* y,
                          int32_t* device_status, void* stream) {
  const mok_status s = check_rows(d);
  if (s != MOK_OK) return s;
  if (!aligned_elem(o, d->type) || !aligned_elem(y, d->type) || !words_aligned({row_of, gates, device_status}))
    return MOK_ERR_INVALID_ARG;
  if (d->T == 0) return MOK_OK;
  if (!row_of || !y || (d->R > 0 && !o)) return MOK_ERR_INVALID_ARG;
  mok::RowsArgs a = rows_args(d, row_of, gates, device_status);
  a.rows = o;
  a.out = y;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  MOK_LAUNCH("expert_merge", st, mok::launch_expert_merge(a, d->type == MOK_ELEM_BF16, st));
  return MOK_OK;
}

mok_status mok_merge_rows_backward(const mok_rows_desc* d, const void* dy, const void* o, const int32_t* row_of,
                                   const float* gates, void* d_o, float* dgates, int32_t* device_status, void* stream) {
  const mok_status s = check_rows(d);
  if (s != MOK_OK) return s;
  if (!aligned_elem(dy, d->type) || !aligned_elem(o, d->type) || !aligned_elem(d_o, d->type) ||
      !words_aligned({row_of, gates, dgates, device_status}))
    return MOK_ERR_INVALID_ARG;
  if (d->T == 0) return MOK_OK;
  if (!dy || !row_of || (d->R > 0 && (!o || !d_o))) return MOK_ERR_INVALID_ARG;
  mok::RowsArgs a = rows_args(d, row_of, gates, device_status);
  a.tokens = dy;
  a.rows = o;
  a.out = d_o;
  a.dgates = dgates;
  const int n_sm = sm_count();
  if (n_sm <= 0) return MOK_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  MOK_LAUNCH("expert_merge_backward", st, mok::launch_expert_merge_backward(a, d->type == MOK_ELEM_BF16, n_sm, st));
  return MOK_OK;
}

mok_status mok_fp8_quantize(const mok_fp8_quantize_desc* d, const void* x, const void* grad, const int32_t* src_of,
                            const float* gates, const int32_t* offsets, uint8_t* q, float* scale, uint8_t* qt,
                            float* qt_scale, int32_t* device_status, void* stream) {
  if (d == nullptr || d->R < 0 || d->C < 1 || d->T < 0 || !elem_type(d->type)) return MOK_ERR_INVALID_ARG;
  if (d->source < MOK_FP8_PLAIN || d->source > MOK_FP8_SWIGLU_GRAD) return MOK_ERR_INVALID_ARG;
  const bool gathered = d->source == MOK_FP8_PLAIN && src_of != nullptr;
  if (d->source != MOK_FP8_PLAIN && (src_of != nullptr || gates != nullptr)) return MOK_ERR_INVALID_ARG;
  if (gates != nullptr && !gathered) return MOK_ERR_INVALID_ARG;
  if ((d->source == MOK_FP8_SWIGLU_GRAD) != (grad != nullptr)) return MOK_ERR_INVALID_ARG;
  if (d->source == MOK_FP8_SWIGLU_GRAD && d->C % 2 != 0) return MOK_ERR_INVALID_ARG;
  if (gathered && d->k < 1) return MOK_ERR_INVALID_ARG;
  if (d->R == 0) return MOK_OK;  // nothing to read or write: no pointer is looked at
  if ((q == nullptr) != (scale == nullptr) || (qt == nullptr) != (qt_scale == nullptr)) return MOK_ERR_INVALID_ARG;
  if (q == nullptr && qt == nullptr) return MOK_ERR_INVALID_ARG;
  if (qt != nullptr && (offsets == nullptr || d->E < 1)) return MOK_ERR_INVALID_ARG;
  const int64_t x_width = d->source == MOK_FP8_SWIGLU ? 2 * d->C : d->C;
  const int64_t blocks = d->R / 128 + (qt != nullptr ? d->E : 0), P = 128 * blocks;
  if (!stride_ok(d->x_stride, x_width) || !stride_ok(d->grad_stride, d->C / 2) || !stride_ok(d->scale_stride, d->R) ||
      !byte_stride_ok(d->q_stride, d->C) || !byte_stride_ok(d->qt_stride, P))
    return MOK_ERR_INVALID_ARG;
  if (!aligned_elem(x, d->type) || !aligned_elem(grad, d->type) || !aligned16(q) || !aligned16(qt) ||
      !words_aligned({src_of, gates, offsets, scale, qt_scale, device_status}))
    return MOK_ERR_INVALID_ARG;
  if (d->R >= kMaxRows - 128 || d->C >= kMaxWidth || (qt != nullptr && d->E > mok::FP8_MAX_E) ||
      (gathered && (d->k > mok::ROWS_MAX_K || d->T >= kMaxRows / d->k)))
    return MOK_ERR_UNSUPPORTED;
  if (x == nullptr && !(gathered && d->T == 0)) return MOK_ERR_INVALID_ARG;
  mok::Fp8QuantizeArgs a = {};
  a.R = d->R;
  a.C = d->C;
  a.T = d->T;
  a.x_stride = d->x_stride != 0 ? d->x_stride : x_width;
  a.grad_stride = d->grad_stride != 0 ? d->grad_stride : d->C / 2;
  a.q_stride = d->q_stride != 0 ? d->q_stride : up16(d->C);
  a.scale_stride = d->scale_stride != 0 ? d->scale_stride : d->R;
  a.qt_stride = d->qt_stride != 0 ? d->qt_stride : P;
  a.E = d->E;
  a.k = d->k;
  a.x = x;
  a.grad = grad;
  a.src_of = src_of;
  a.gates = gates;
  a.offsets = offsets;
  a.q = q;
  a.scale = scale;
  a.qt = qt;
  a.qt_scale = qt_scale;
  a.status = device_status;
  const int n_sm = sm_count();
  if (n_sm <= 0) return MOK_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  MOK_LAUNCH("fp8_quantize", st, mok::launch_fp8_quantize(a, d->source, d->type == MOK_ELEM_BF16, n_sm, st));
  return MOK_OK;
}

mok_status mok_fp8_quantize_weights(const mok_fp8_weights_desc* d, const void* w, uint8_t* q, float* scale, uint8_t* qt,
                                    float* qt_scale, void* stream) {
  if (d == nullptr || d->E < 1 || d->N < 1 || d->K < 1 || !elem_type(d->type)) return MOK_ERR_INVALID_ARG;
  if (!byte_stride_ok(d->q_stride, d->K) || !byte_stride_ok(d->qt_stride, d->N)) return MOK_ERR_INVALID_ARG;
  if ((q == nullptr) != (scale == nullptr) || (qt == nullptr) != (qt_scale == nullptr)) return MOK_ERR_INVALID_ARG;
  if ((q == nullptr && qt == nullptr) || w == nullptr) return MOK_ERR_INVALID_ARG;
  if (!aligned_elem(w, d->type) || !aligned16(q) || !aligned16(qt) || !words_aligned({scale, qt_scale}))
    return MOK_ERR_INVALID_ARG;
  if (d->E > mok::FP8_MAX_E || d->N >= kMaxWidth || d->K >= kMaxWidth) return MOK_ERR_UNSUPPORTED;
  mok::Fp8WeightsArgs a = {};
  a.N = d->N;
  a.K = d->K;
  a.q_stride = d->q_stride != 0 ? d->q_stride : up16(d->K);
  a.qt_stride = d->qt_stride != 0 ? d->qt_stride : up16(d->N);
  a.E = d->E;
  a.w = w;
  a.q = q;
  a.scale = scale;
  a.qt = qt;
  a.qt_scale = qt_scale;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  MOK_LAUNCH("fp8_weights", st, mok::launch_fp8_weights(a, d->type == MOK_ELEM_BF16, st));
  return MOK_OK;
}

mok_status mok_fp8_matmul(const mok_fp8_matmul_desc* d, const uint8_t* x, const float* x_scale, const uint8_t* w,
                          const float* w_scale, const int32_t* offsets, void* out, int32_t* device_status,
                          void* stream) {
  if (d == nullptr || d->R < 0 || d->N < 1 || d->K < 1 || d->E < 1 || !elem_type(d->out_type)) return MOK_ERR_INVALID_ARG;
  if (offsets == nullptr && d->E != 1) return MOK_ERR_INVALID_ARG;
  if (!byte_stride_ok(d->x_stride, d->K) || !byte_stride_ok(d->w_stride, d->K) || !stride_ok(d->x_scale_stride, d->R) ||
      !stride_ok(d->out_stride, d->N))
    return MOK_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w) || !aligned_elem(out, d->out_type) ||
      !words_aligned({x_scale, w_scale, offsets, device_status}))
    return MOK_ERR_INVALID_ARG;
  if (d->E > mok::FP8_MAX_E || d->R >= kMaxRows - 256 || d->N >= kMaxWidth || d->K >= kMaxWidth)
    return MOK_ERR_UNSUPPORTED;
  if (d->R == 0) return MOK_OK;
  if (!x || !x_scale || !w || !w_scale || !out) return MOK_ERR_INVALID_ARG;
  mok::Fp8MatmulArgs a = {};
  a.R = d->R;
  a.N = d->N;
  a.K = d->K;
  a.x_stride = d->x_stride != 0 ? d->x_stride : up16(d->K);
  a.w_stride = d->w_stride != 0 ? d->w_stride : up16(d->K);
  a.x_scale_stride = d->x_scale_stride != 0 ? d->x_scale_stride : d->R;
  a.out_stride = d->out_stride != 0 ? d->out_stride : d->N;
  a.E = d->E;
  a.x = x;
  a.x_scale = x_scale;
  a.w = w;
  a.w_scale = w_scale;
  a.offsets = offsets;
  a.out = out;
  a.status = device_status;
  const int n_sm = sm_count();
  if (n_sm <= 0) return MOK_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  MOK_LAUNCH("fp8_matmul", st, mok::launch_fp8_matmul(a, d->out_type == MOK_ELEM_BF16, n_sm, st));
  return MOK_OK;
}

mok_status mok_fp8_weight_grad(const mok_fp8_weight_grad_desc* d, const uint8_t* dy, const float* dy_scale,
                               const uint8_t* x, const float* x_scale, const int32_t* offsets, void* out,
                               int32_t* device_status, void* stream) {
  if (d == nullptr || d->R < 0 || d->N < 1 || d->H < 1 || d->E < 1 || !elem_type(d->out_type)) return MOK_ERR_INVALID_ARG;
  const int64_t P = 128 * (d->R / 128 + d->E);
  if (!byte_stride_ok(d->dy_stride, P) || !byte_stride_ok(d->x_stride, P)) return MOK_ERR_INVALID_ARG;
  if (!aligned16(dy) || !aligned16(x) || !aligned_elem(out, d->out_type) ||
      !words_aligned({dy_scale, x_scale, offsets, device_status}))
    return MOK_ERR_INVALID_ARG;
  if (d->E > mok::FP8_MAX_E || d->R >= kMaxRows - 128 * (mok::FP8_MAX_E + 1) || d->N >= kMaxWidth || d->H >= kMaxWidth)
    return MOK_ERR_UNSUPPORTED;
  if (!dy || !dy_scale || !x || !x_scale || !offsets || !out) return MOK_ERR_INVALID_ARG;
  mok::Fp8WeightGradArgs a = {};
  a.R = d->R;
  a.N = d->N;
  a.H = d->H;
  a.dy_stride = d->dy_stride != 0 ? d->dy_stride : P;
  a.x_stride = d->x_stride != 0 ? d->x_stride : P;
  a.E = d->E;
  a.dy = dy;
  a.dy_scale = dy_scale;
  a.x = x;
  a.x_scale = x_scale;
  a.offsets = offsets;
  a.out = out;
  a.status = device_status;
  const int n_sm = sm_count();
  if (n_sm <= 0) return MOK_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  MOK_LAUNCH("fp8_weight_grad", st, mok::launch_fp8_weight_grad(a, d->out_type == MOK_ELEM_BF16, n_sm, st));
  return MOK_OK;
}

}  // extern "C"
