// Optimizer kernels: the global 2-norm of many gradients with the clip factor, and an AdamW step
// over many tensors with f32 or 8-bit states.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "optim.cuh"

namespace mok {

namespace {

constexpr int VEC = 8;                      // elements of one thread: a quarter of a 32-element scale block
constexpr int ADAM_THREADS = 256;
constexpr int CHUNK = ADAM_THREADS * VEC;   // elements of one block
constexpr int NORM_THREADS = 512;
constexpr int NORM_CHUNK = NORM_THREADS * VEC * 4;

// Two sizes: a launch with 21 KB of parameters costs its caller about 0.7 us more than one with 1.4 KB.
constexpr int SMALL_TABLE = 16;
template <typename Tensor, int CAP>
struct Table {
  Tensor t[CAP];
  int32_t first[CAP + 1];  // first chunk of each tensor; first[count] = chunks in all
  int32_t count;
};

// The tensor that holds chunk c: the last one whose first chunk is <= c (empty tensors have none).
template <typename Tensor, int CAP>
__device__ __forceinline__ int tensor_of(const Table<Tensor, CAP>& tab, int c) {
  int lo = 0, hi = tab.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tab.first[mid] <= c) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ bool aligned_to(const void* p, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

// 8 elements from p + i, `left` of them in range; `wide`: all 8, and p is 16-byte aligned.
__device__ __forceinline__ void load8(const float* p, int64_t i, int left, bool wide, float (&x)[VEC]) {
  if (wide) {
    const float4 a = *reinterpret_cast<const float4*>(p + i), b = *reinterpret_cast<const float4*>(p + i + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) x[j] = j < left ? p[i + j] : 0.0f;
  }
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, int64_t i, int left, bool wide, float (&x)[VEC]) {
  if (wide) {
    const uint4 a = *reinterpret_cast<const uint4*>(p + i);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = __uint_as_float(w[j] << 16);
      x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) x[j] = j < left ? __bfloat162float(p[i + j]) : 0.0f;
  }
}
__device__ __forceinline__ void store8(float* p, int64_t i, int left, bool wide, const float (&x)[VEC]) {
  if (wide) {
    *reinterpret_cast<float4*>(p + i) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + i + 4) = make_float4(x[4], x[5], x[6], x[7]);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (j < left) p[i + j] = x[j];
  }
}
// 8 bf16 bit patterns, the low half of each word
__device__ __forceinline__ void store8(__nv_bfloat16* p, int64_t i, int left, bool wide, const uint32_t (&b)[VEC]) {
  if (wide) {
    *reinterpret_cast<uint4*>(p + i) = make_uint4(b[0] | b[1] << 16, b[2] | b[3] << 16, b[4] | b[5] << 16, b[6] | b[7] << 16);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (j < left) p[i + j] = __ushort_as_bfloat16((unsigned short)b[j]);
  }
}

// 32 bits for each of the 8 elements of a counter group: MurmurHash3's 32-bit finaliser (A. Appleby) of the
// group's number and the step's seed, times one odd number each.
__device__ __forceinline__ void rounding_bits(uint64_t group, uint32_t seed, uint32_t (&z)[VEC]) {
  uint32_t x = (uint32_t)group ^ ((uint32_t)(group >> 32) * 0x9E3779B1u) ^ seed;
  x = (x ^ (x >> 16)) * 0x85EBCA6Bu;
  x = (x ^ (x >> 13)) * 0xC2B2AE35u;
  x ^= x >> 16;
  const uint32_t odd[VEC] = {0x9E3779B1u, 0x85EBCA77u, 0xC2B2AE3Du, 0x27D4EB2Fu,
                             0x165667B1u, 0xD3A2646Du, 0xFD7046C5u, 0xB55A4F09u};
#pragma unroll
  for (int j = 0; j < VEC; ++j) z[j] = x * odd[j];
}

// ----------------------------------------------------------------------------- 8-bit states
// A block of 32 elements is held as E4M3 elements and one power of two 2^(b - 127) (an E8M0 byte b): the least
// one with amax <= 448 * 2^(b - 127), so that the largest element is not cut off.  b is kept in [1, 254], where
// the power and its inverse are normal f32 numbers.
__device__ __forceinline__ int scale_byte(float amax) {
  const int b = ((__float_as_int(amax) + 0x1fffff) >> 23) - 8;  // mantissas above 1.75 carry to the next power
  return min(max(b, 1), 254);
}
__device__ __forceinline__ float power_of_two(int biased) { return __int_as_float(biased << 23); }

// y (|y| <= 448) to the E4M3 grid: floor(y / ulp + u) * ulp, exactly; u uniform in [0, 1) makes the mean y.
// t = y's power of two, at least 2^-6 (below it the grid is 2^-9); 1.5 * 2^20 * t has an ulp of t / 8, the grid's.
__device__ __forceinline__ float to_grid(float y, float u) {
  const float t = fmaxf(__int_as_float(__float_as_int(y) & 0x7f800000), 0.015625f);
  const float f = fmaf(t, u * 0.125f, y);
  const float a = __fmaf_rd(t, 1572864.0f, f);
  return fmaf(t, -1572864.0f, a);
}

__device__ __forceinline__ float block_max(const float (&x)[VEC]) {
  float a = 0.0f;
#pragma unroll
  for (int j = 0; j < VEC; ++j) a = fmaxf(a, fabsf(x[j]));
  a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
  return fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
}

__device__ __forceinline__ void load_state8(const uint8_t* q, const uint8_t* scale, int64_t i, int left, bool wide,
                                            float (&x)[VEC]) {
  uint32_t w[2] = {0u, 0u};
  if (wide) {
    const uint2 a = *reinterpret_cast<const uint2*>(q + i);
    w[0] = a.x, w[1] = a.y;
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (j < left) w[j >> 2] |= (uint32_t)q[i + j] << (8 * (j & 3));
  }
  const float s = left > 0 ? power_of_two(scale[i >> 5]) : 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[j >> 1] >> (16 * (j & 1))), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    x[2 * j] = f.x * s;
    x[2 * j + 1] = f.y * s;
  }
}
__device__ __forceinline__ void store_state8(uint8_t* q, uint8_t* scale, int64_t i, int left, bool wide, int b,
                                             const float (&y)[VEC]) {
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_fp8x2_storage_t c =
        __nv_cvt_float2_to_fp8x2(make_float2(y[2 * j], y[2 * j + 1]), __NV_SATFINITE, __NV_E4M3);
    w[j >> 1] |= (uint32_t)c << (16 * (j & 1));
  }
  if (wide) {
    *reinterpret_cast<uint2*>(q + i) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (j < left) q[i + j] = (uint8_t)(w[j >> 2] >> (8 * (j & 3)));
  }
  if (left > 0 && (i & 31) == 0) scale[i >> 5] = (uint8_t)b;
}

// ----------------------------------------------------------------------------- AdamW
//   g' = c g;  m = b1 m + (1 - b1) g';  v = b2 v + (1 - b2) g'^2
//   p -= lr ( (m / bc1) / (sqrt(v / bc2) + eps) + wd p )
// 8-bit states hold m and sqrt(v).  A step moves sqrt(v) by (1 - b2) / 2 of itself, 0.05% to 2.5%, and E4M3's
// grid is 6% to 12% wide: rounded to nearest, a state would never move again, so both are rounded up or down
// at random with the mean unchanged.  sqrt(v) > 0 never becomes 0, so that no step divides by eps alone.
// bf16 parameters without an f32 master are rounded the same way (their updates are below half a spacing too).
// A clip factor c that is NaN leaves the tensor as it is (grad_norm gives one for gradients that are not finite).
template <int PK, int GK, int SK, int CAP>
__global__ void __launch_bounds__(ADAM_THREADS)
    adamw_kernel(const __grid_constant__ Table<AdamTensor, CAP> tab, const AdamHyper h, const float* __restrict__ grad_scale) {
  const float c = grad_scale != nullptr ? *grad_scale : 1.0f;
  if (isnan(c)) return;
  const int chunk = blockIdx.x;
  const int k = tensor_of(tab, chunk);
  const AdamTensor& T = tab.t[k];
  const int64_t i = (int64_t)(chunk - tab.first[k]) * CHUNK + threadIdx.x * VEC;
  const int left = (int)min((int64_t)VEC, max((int64_t)0, T.n - i));
  bool wide = left == VEC && aligned_to(T.param, 16) && aligned_to(T.grad, 16) && aligned_to(T.m, 16) && aligned_to(T.v, 16);
  if (PK == PARAM_BF16_MASTER) wide = wide && aligned_to(T.master, 16);

  float p[VEC], g[VEC], m[VEC], v[VEC];
  if constexpr (PK == PARAM_F32) load8(static_cast<const float*>(T.param), i, left, wide, p);
  else if constexpr (PK == PARAM_BF16_MASTER) load8(T.master, i, left, wide, p);
  else load8(static_cast<const __nv_bfloat16*>(T.param), i, left, wide, p);
  if constexpr (GK == GRAD_F32) load8(static_cast<const float*>(T.grad), i, left, wide, g);
  else load8(static_cast<const __nv_bfloat16*>(T.grad), i, left, wide, g);
  if constexpr (SK == STATE_F32) {
    load8(static_cast<const float*>(T.m), i, left, wide, m);
    load8(static_cast<const float*>(T.v), i, left, wide, v);
  } else {
    load_state8(static_cast<const uint8_t*>(T.m), T.m_scale, i, left, wide, m);
    load_state8(static_cast<const uint8_t*>(T.v), T.v_scale, i, left, wide, v);
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] *= v[j];
  }

  float r[VEC];  // sqrt(v)
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    const float gj = c * g[j];
    m[j] = fmaf(h.beta1, m[j], h.one_minus_beta1 * gj);
    v[j] = fmaf(h.beta2, v[j], h.one_minus_beta2 * gj * gj);
    r[j] = sqrtf(v[j]);
    const float update = (m[j] * h.inv_bc1) / fmaf(r[j], h.inv_bc2_sqrt, h.eps) + T.weight_decay * p[j];
    p[j] = fmaf(-T.lr, update, p[j]);
  }

  uint32_t z[VEC];
  if constexpr (SK == STATE_MX8 || PK == PARAM_BF16) rounding_bits((T.counter + (uint64_t)i) >> 3, h.seed, z);
  if constexpr (PK == PARAM_F32) {
    store8(static_cast<float*>(T.param), i, left, wide, p);
  } else {
    uint32_t b[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      if constexpr (PK == PARAM_BF16) b[j] = (__float_as_uint(p[j]) + (z[j] & 0xffffu)) >> 16;
      else b[j] = __bfloat16_as_ushort(__float2bfloat16_rn(p[j]));
    }
    store8(static_cast<__nv_bfloat16*>(T.param), i, left, wide, b);
    if constexpr (PK == PARAM_BF16_MASTER) store8(T.master, i, left, wide, p);
  }
  if constexpr (SK == STATE_F32) {
    store8(static_cast<float*>(T.m), i, left, wide, m);
    store8(static_cast<float*>(T.v), i, left, wide, v);
  } else {
    const int bm = scale_byte(block_max(m)), bv = scale_byte(block_max(r));
    const float im = power_of_two(254 - bm), iv = power_of_two(254 - bv);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      m[j] = to_grid(m[j] * im, (float)(z[j] >> 9) * 0x1p-23f);
      const float y = r[j] * iv;
      r[j] = to_grid(y, (float)(z[j] & 0x7fffffu) * 0x1p-23f);
      if (y > 0.0f) r[j] = fmaxf(r[j], 0.001953125f);
    }
    store_state8(static_cast<uint8_t*>(T.m), T.m_scale, i, left, wide, bm, m);
    store_state8(static_cast<uint8_t*>(T.v), T.v_scale, i, left, wide, bv, r);
  }
}

// ----------------------------------------------------------------------------- gradient norm
// Each block sums its chunks' squares in f32 per thread and in f64 from there on; the block that comes last in
// the call adds the blocks' sums in their order, so that the result does not depend on the order of arrival.
template <int CAP>
__global__ void __launch_bounds__(NORM_THREADS)
    grad_norm_kernel(const __grid_constant__ Table<GradTensor, CAP> tab, int first_block, int total_blocks, float max_norm,
                     float* __restrict__ out, unsigned* __restrict__ ticket, double* __restrict__ partials) {
  __shared__ double warp_sum[NORM_THREADS / 32];
  __shared__ bool last;
  float acc[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) acc[j] = 0.0f;
  for (int chunk = blockIdx.x; chunk < tab.first[tab.count]; chunk += gridDim.x) {
    const int k = tensor_of(tab, chunk);
    const GradTensor& T = tab.t[k];
    const int64_t base = (int64_t)(chunk - tab.first[k]) * NORM_CHUNK + threadIdx.x * VEC;
    const bool aligned = aligned_to(T.grad, 16);
#pragma unroll
    for (int q = 0; q < NORM_CHUNK / (NORM_THREADS * VEC); ++q) {
      const int64_t i = base + (int64_t)q * NORM_THREADS * VEC;
      const int left = (int)min((int64_t)VEC, max((int64_t)0, T.n - i));
      float g[VEC];
      if (T.bf16) load8(static_cast<const __nv_bfloat16*>(T.grad), i, left, left == VEC && aligned, g);
      else load8(static_cast<const float*>(T.grad), i, left, left == VEC && aligned, g);
#pragma unroll
      for (int j = 0; j < VEC; ++j) acc[j] = fmaf(g[j], g[j], acc[j]);
    }
  }
  double s = 0.0;
#pragma unroll
  for (int j = 0; j < VEC; ++j) s += (double)acc[j];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) warp_sum[warp] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    double b = 0.0;
    for (int w = 0; w < NORM_THREADS / 32; ++w) b += warp_sum[w];
    partials[first_block + blockIdx.x] = b;
    __threadfence();
    last = atomicAdd(ticket, 1u) == (unsigned)(total_blocks - 1);
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  s = 0.0;
  for (int b = threadIdx.x; b < total_blocks; b += NORM_THREADS) s += __ldcg(&partials[b]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) warp_sum[warp] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    double b = 0.0;
    for (int w = 0; w < NORM_THREADS / 32; ++w) b += warp_sum[w];
    const double norm = sqrt(b);
    out[0] = (float)norm;
    out[1] = isfinite(norm) ? (float)fmin(1.0, (double)max_norm / (norm + 1e-6)) : __int_as_float(0x7fffffff);
    *ticket = 0u;
  }
}

// The table of `count` tensors; returns their chunks, or -1 if there are more than a grid has blocks.
template <typename Tensor, int CAP, typename Chunks>
int64_t fill_table(Table<Tensor, CAP>& tab, const Tensor* tensors, int count, Chunks chunks_of) {
  int64_t chunks = 0;
  for (int i = 0; i < count; ++i) {
    tab.t[i] = tensors[i];
    tab.first[i] = (int32_t)chunks;
    chunks += chunks_of(tensors[i].n);
    if (chunks > INT32_MAX) return -1;
  }
  tab.first[count] = (int32_t)chunks;
  tab.count = count;
  return chunks;
}

template <int PK, int GK, int SK, int CAP>
cudaError_t launch_table(const AdamTensor* tensors, int count, const AdamHyper& h, const float* scale, cudaStream_t st) {
  Table<AdamTensor, CAP> tab;
  const int64_t chunks = fill_table(tab, tensors, count, [](int64_t n) { return (n + CHUNK - 1) / CHUNK; });
  if (chunks < 0) return cudaErrorInvalidValue;
  if (chunks == 0) return cudaSuccess;
  adamw_kernel<PK, GK, SK, CAP><<<(int)chunks, ADAM_THREADS, 0, st>>>(tab, h, scale);
  return cudaGetLastError();
}

template <int PK, int GK>
cudaError_t launch_kind(const AdamTensor* t, int count, int state, const AdamHyper& h, const float* scale,
                        cudaStream_t st) {
  const bool small = count <= SMALL_TABLE;
  if (state == STATE_F32)
    return small ? launch_table<PK, GK, STATE_F32, SMALL_TABLE>(t, count, h, scale, st)
                 : launch_table<PK, GK, STATE_F32, OPTIM_TABLE>(t, count, h, scale, st);
  return small ? launch_table<PK, GK, STATE_MX8, SMALL_TABLE>(t, count, h, scale, st)
               : launch_table<PK, GK, STATE_MX8, OPTIM_TABLE>(t, count, h, scale, st);
}

template <int CAP>
cudaError_t launch_norm(const GradTensor* tensors, int count, int blocks, int first_block, int total_blocks,
                        float max_norm, float* out, void* ws, cudaStream_t st) {
  Table<GradTensor, CAP> tab;
  if (fill_table(tab, tensors, count, grad_norm_chunks) < 0) return cudaErrorInvalidValue;
  grad_norm_kernel<CAP><<<blocks, NORM_THREADS, 0, st>>>(
      tab, first_block, total_blocks, max_norm, out, static_cast<unsigned*>(ws),
      reinterpret_cast<double*>(static_cast<char*>(ws) + NORM_PARTIALS_OFFSET));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_adamw(const AdamTensor* t, int count, int param, int grad, int state, const AdamHyper& h,
                         const float* grad_scale, int n_sm, cudaStream_t st) {
  switch (param * 2 + grad) {
    case PARAM_F32 * 2 + GRAD_F32: return launch_kind<PARAM_F32, GRAD_F32>(t, count, state, h, grad_scale, st);
    case PARAM_F32 * 2 + GRAD_BF16: return launch_kind<PARAM_F32, GRAD_BF16>(t, count, state, h, grad_scale, st);
    case PARAM_BF16_MASTER * 2 + GRAD_F32: return launch_kind<PARAM_BF16_MASTER, GRAD_F32>(t, count, state, h, grad_scale, st);
    case PARAM_BF16_MASTER * 2 + GRAD_BF16: return launch_kind<PARAM_BF16_MASTER, GRAD_BF16>(t, count, state, h, grad_scale, st);
    case PARAM_BF16 * 2 + GRAD_F32: return launch_kind<PARAM_BF16, GRAD_F32>(t, count, state, h, grad_scale, st);
    default: return launch_kind<PARAM_BF16, GRAD_BF16>(t, count, state, h, grad_scale, st);
  }
}

int64_t grad_norm_chunks(int64_t n) { return (n + NORM_CHUNK - 1) / NORM_CHUNK; }

cudaError_t launch_grad_norm(const GradTensor* tensors, int count, int blocks, int first_block, int total_blocks,
                             float max_norm, float* out, void* ws, cudaStream_t st) {
  if (count <= SMALL_TABLE)
    return launch_norm<SMALL_TABLE>(tensors, count, blocks, first_block, total_blocks, max_norm, out, ws, st);
  return launch_norm<OPTIM_TABLE>(tensors, count, blocks, first_block, total_blocks, max_norm, out, ws, st);
}

}  // namespace mok
