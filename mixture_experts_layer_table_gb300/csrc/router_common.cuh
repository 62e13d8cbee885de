// What the routing kernels share: scores, orders and the end of the load-balancing sums.
#pragma once
#include <cuda_bf16.h>

#include <cmath>
#include <cstdint>

#include "f32x2.cuh"
#include "router.cuh"

namespace mok {
namespace {

constexpr unsigned ALL = 0xffffffffu;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float x, float* p) { *p = x; }
__device__ __forceinline__ void from_f32(float x, __nv_bfloat16* p) { *p = __float2bfloat16_rn(x); }

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(ALL, x, o);
  return x;
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(ALL, x, o));
  return x;
}

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// The hardware's exponential and reciprocal, off by about 2^-22.
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float inverse_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
constexpr float LOG2E = 1.442695041f;
// e^(a - shift) and e^(b - shift) by it.  The shift is taken off first: as a rounded product of its own in the exponent it
// would skew all terms of a softmax's sum alike (4e-5 at a shift of 1000), but not a score that is formed apart from them.
__device__ __forceinline__ void exp_pair(float a, float b, float shift, float& ea, float& eb) {
  split(mul2(add2(f2(a, b), f2(-shift)), f2(LOG2E)), ea, eb);
  ea = exp2_fast(ea), eb = exp2_fast(eb);
}

// Unsigned integers in the order of the floats (-inf is the least, above 0); -0 equals +0.
__device__ __forceinline__ uint32_t ordered(float r) {
  const int b = __float_as_int(r + 0.0f);
  return (uint32_t)b ^ ((uint32_t)(b >> 31) | 0x80000000u);
}

// a's two largest and b's two largest to the two largest of all
__device__ __forceinline__ void merge_top2(float& a1, float& a2, float b1, float b2) {
  a2 = fmaxf(fminf(a1, b1), fmaxf(a2, b2));
  a1 = fmaxf(a1, b1);
}

// The end of a kernel with load-balancing outputs: every block adds its counts and probability sums (sum_of(expert))
// to the workspace, as integers (the probabilities in units of 2^-sum_shift), whose sum does not depend on the order
// of the blocks; the block that comes last writes the results and leaves the workspace as it was.  Called by all
// threads of every block, after a barrier behind the last sum.
template <typename Sum>
__device__ __forceinline__ void finish_balance(const RouteArgs& a, const int* counts, Sum sum_of) {
  __shared__ bool last;
  __shared__ float part[32];
  const float units_of = __int_as_float((127 + a.sum_shift) << 23);
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
    const float p = sum_of(e);
    const int at = (blockIdx.x % ROUTE_COPIES) * ROUTE_MAX_E + e;
    if (isfinite(p)) atomicAdd(&a.acc_prob[at], (unsigned long long)__float2ll_rn(p * units_of));
    else atomicOr(a.not_finite, 1u);
    if (counts[e] != 0) atomicAdd(&a.acc_counts[at], counts[e]);
  }
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  const bool bad = __ldcg(a.not_finite) != 0u;
  const float unit = __int_as_float((127 - a.sum_shift) << 23);
  float loss = 0.0f;
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
    long long units = 0;
    int n = 0;
#pragma unroll
    for (int c = 0; c < ROUTE_COPIES; ++c) {
      units += (long long)__ldcg(&a.acc_prob[c * ROUTE_MAX_E + e]);
      n += __ldcg(&a.acc_counts[c * ROUTE_MAX_E + e]);
    }
#pragma unroll
    for (int c = 0; c < ROUTE_COPIES; ++c) a.acc_prob[c * ROUTE_MAX_E + e] = 0ull, a.acc_counts[c * ROUTE_MAX_E + e] = 0;
    const float p = bad ? __int_as_float(0x7fffffff) : __ll2float_rn(units) * unit;
    const float d = (float)n * a.dprob_unit;
    if (a.counts != nullptr) a.counts[e] = n;
    if (a.prob_sum != nullptr) a.prob_sum[e] = p;
    if (a.dprob != nullptr) a.dprob[e] = d;
    if (a.bias_next != nullptr) {
      const long long lack = a.T * a.k - (long long)a.E * n;
      a.bias_next[e] = a.bias[e] + (lack > 0 ? a.bias_rate : lack < 0 ? -a.bias_rate : 0.0f);
    }
    loss = fmaf(d, p, loss);
  }
  if (a.loss != nullptr) {
    loss = warp_sum(loss);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = loss;
    __syncthreads();
    if (threadIdx.x < 32) {
      loss = warp_sum(threadIdx.x < blockDim.x / 32 ? part[threadIdx.x] : 0.0f);
      if (threadIdx.x == 0) *a.loss = loss;
    }
  }
  if (threadIdx.x == 0) {
    *a.ticket = 0u;
    *a.not_finite = 0u;
  }
}

}  // namespace
}  // namespace mok
