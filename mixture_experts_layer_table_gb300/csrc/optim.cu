// Optimizer kernels: the global 2-norm of many gradients with the clip factor, and an AdamW step
// over many tensors with f32 or 8-bit states.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "f32x2.cuh"
#include "optim.cuh"

namespace mok {

namespace {

constexpr int VEC = 8;                      // elements of one thread: a quarter of a 32-element scale block
constexpr int ADAM_THREADS = 256;
constexpr int PASS = ADAM_THREADS * VEC;    // elements of one pass of a block
constexpr int NORM_THREADS = 512;
constexpr int NORM_CHUNK = NORM_THREADS * VEC * 4;

// Two sizes: a launch with 24 KB of parameters costs its caller about 0.7 us more than one with 1.4 KB.
constexpr int SMALL_TABLE = 16;
template <typename Tensor, int CAP>
struct Table {
  Tensor t[CAP];
  int32_t first[CAP + 1];  // first chunk of each tensor; first[count] = chunks in all
  int32_t count;
  static constexpr int MAPPED = CAP > SMALL_TABLE ? 2048 : 4;
  uint8_t of_chunk[MAPPED];  // the tensor of each chunk, where there are at most so many (0.3 us less than a search)
};

// The tensor that holds chunk c: the last one whose first chunk is <= c (empty tensors have none).
template <typename Tensor, int CAP>
__device__ __forceinline__ int tensor_of(const Table<Tensor, CAP>& tab, int c) {
  if (CAP > SMALL_TABLE && tab.first[tab.count] <= tab.MAPPED) return tab.of_chunk[c];
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

// 8 elements from p + i, `left` of them in range; WIDE: all 8, and p is 16-byte aligned.
template <bool WIDE>
__device__ __forceinline__ void load8(const float* p, uint32_t i, int left, float (&x)[VEC]) {
  if constexpr (WIDE) {
    const float4 a = *reinterpret_cast<const float4*>(p + i), b = *reinterpret_cast<const float4*>(p + i + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) x[j] = j < left ? p[i + j] : 0.0f;
  }
}
template <bool WIDE>
__device__ __forceinline__ void load8(const __nv_bfloat16* p, uint32_t i, int left, float (&x)[VEC]) {
  if constexpr (WIDE) {
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
template <bool WIDE>
__device__ __forceinline__ void store8(float* p, uint32_t i, int left, const float (&x)[VEC]) {
  if constexpr (WIDE) {
    *reinterpret_cast<float4*>(p + i) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + i + 4) = make_float4(x[4], x[5], x[6], x[7]);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (j < left) p[i + j] = x[j];
  }
}
// 8 bf16, two to a word
template <bool WIDE>
__device__ __forceinline__ void store8(__nv_bfloat16* p, uint32_t i, int left, const uint32_t (&w)[VEC / 2]) {
  if constexpr (WIDE) {
    *reinterpret_cast<uint4*>(p + i) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (j < left) p[i + j] = __ushort_as_bfloat16((unsigned short)(w[j >> 1] >> (16 * (j & 1))));
  }
}

// 32 bits for each of the 8 elements of a counter group: MurmurHash3's 32-bit finaliser (A. Appleby) of the
// group's number and the step's seed, times one odd number each (the first five are the primes of XXH32, Y. Collet).
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

// ----------------------------------------------------------------------------- packed f32
// (the 8-bit step is bound by issued instructions)
__device__ __forceinline__ F2 fma2_down(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rm.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// one unit in the last place or so; subnormal arguments count as 0
__device__ __forceinline__ float fast_sqrt(float x) {
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float fast_inverse(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
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

// y's power of two, at least 2^-6 (below it E4M3's grid is 2^-9): 8 spacings of the grid at y
__device__ __forceinline__ float eight_spacings(float y) {
  return fmaxf(__int_as_float(__float_as_int(y) & 0x7f800000), 0.015625f);
}
// y (|y| <= 448) to the E4M3 grid: floor(y / spacing + u) * spacing, exactly, u uniform in [0, 1), so that the
// mean is y.  With t the eight spacings, 1.5 * 2^20 * t has a spacing of t / 8: the sum rounded down to it is
// 1.5 * 2^20 * t plus the floor.  w holds (1 + u) / 8, from 23 random bits behind an exponent; the added spacing
// is taken off at the end.
__device__ __forceinline__ F2 to_grid(F2 y, F2 w) {
  float y0, y1;
  split(y, y0, y1);
  const F2 t = f2(eight_spacings(y0), eight_spacings(y1));
  const F2 a = fma2_down(t, f2(1572864.0f), fma2(t, w, y));
  return fma2(t, f2(-1572864.125f), a);
}
__device__ __forceinline__ float high_bits(uint32_t z) { return __uint_as_float(__funnelshift_r(z, 0x7cu, 9)); }
__device__ __forceinline__ float low_bits(uint32_t z) { return __uint_as_float((z & 0x7fffffu) | 0x3e000000u); }

// Infinities to NaN: E4M3 has none, and the least power of two that reaches one would leave nothing of the block's other
// elements.
__device__ __forceinline__ void infinities_to_nan(F2 (&x)[VEC / 2]) {
#pragma unroll
  for (int j = 0; j < VEC / 2; ++j) x[j] = fma2(x[j], f2(0.0f), x[j]);
}
// Largest magnitude, NaN aside, of this thread's 8 elements, and of a block: those of the three threads next to it too.
__device__ __forceinline__ float thread_max(const F2 (&x)[VEC / 2]) {
  float a = 0.0f;
#pragma unroll
  for (int j = 0; j < VEC / 2; ++j) {
    float lo, hi;
    split(x[j], lo, hi);
    a = fmaxf(a, fmaxf(fabsf(lo), fabsf(hi)));
  }
  return a;
}
__device__ __forceinline__ float block_max(float a) {
  a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
  return fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
}

__device__ __forceinline__ uint2 load_e4m3(const uint8_t* q, uint32_t i, int left) {
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < VEC; ++j)
    if (j < left) w[j >> 2] |= (uint32_t)q[i + j] << (8 * (j & 3));
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void from_e4m3(uint2 q, F2 (&x)[VEC / 2]) {
#pragma unroll
  for (int j = 0; j < VEC / 2; ++j) {
    const uint32_t w = j < 2 ? q.x : q.y;
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * (j & 1))), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    x[j] = f2(f.x, f.y);
  }
}
template <bool WIDE>
__device__ __forceinline__ void store_e4m3(uint8_t* q, uint32_t i, int left, const F2 (&y)[VEC / 2]) {
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < VEC / 2; ++j) {
    float lo, hi;
    split(y[j], lo, hi);
    const __nv_fp8x2_storage_t c = __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
    w[j >> 1] |= (uint32_t)c << (16 * (j & 1));
  }
  if constexpr (WIDE) {
    *reinterpret_cast<uint2*>(q + i) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (j < left) q[i + j] = (uint8_t)(w[j >> 2] >> (8 * (j & 3)));
  }
}

// ----------------------------------------------------------------------------- AdamW
//   g' = c g;  m = b1 m + (1 - b1) g';  v = b2 v + (1 - b2) g'^2
//   p -= lr ( (m / bc1) / (sqrt(v / bc2) + eps) + wd p )
// 8-bit states hold m and sqrt(v).  A step moves sqrt(v) by (1 - b2) / 2 of itself, 0.05% to 2.5%, and E4M3's
// grid is 6% to 12% wide: rounded to nearest, a state would never move again, so both are rounded up or down
// at random with the mean unchanged.  sqrt(v) > 0 never becomes 0, so that no step divides by eps alone.
// bf16 parameters without an f32 master are rounded the same way (their updates are below half a spacing too).
// What is not finite shows in its own element: NaN stays NaN in a bf16 parameter, and an m or sqrt(v) that is not finite
// is an E4M3 NaN that its block's scale does not see.
// A clip factor c that is NaN leaves the tensor as it is (grad_norm gives one for gradients that are not finite).
//
// 8 consecutive elements to a thread (16 bytes of bf16, 32 of f32; four threads hold a block of 32), 2048 to a
// pass of the block.  With f32 states the step is bound by DRAM and keeps IEEE roots and divisions: bf16 parameters
// with masters and f32 gradients, 30 bytes an element, 354 million elements in 1.48 ms, 7.16 TB/s, issue slots 28%
// full; 96 tensors of 1 to 30,011 elements (8 MB, from L2) 5.7 us.  With 8-bit states it moves 10 to 18 bytes an
// element and issue decides (plain f32: 92 instructions an element, 0.98 ms for those 354 million elements at 10.1
// bytes), so it runs on packed f32 pairs with approximate roots and reciprocals (2^-22; v below 2^-126 counts as 0)
// and rounds without conversions to and from integers: 53 instructions an element, 83% of the issue slots, 0.567 ms,
// 6.32 TB/s; with masters or f32 gradients 6.9 to 7.1 TB/s.
struct AdamConstants {
  float c, beta1, one_minus_beta1, beta2, one_minus_beta2, eps, inv_bc1, inv_bc2_sqrt, lr, weight_decay;
  uint32_t seed;
};

// The part of a tensor from element `begin` (a multiple of 32) on, so that the elements of a block have 32-bit
// offsets.
template <int PK, int GK, int SK>
__device__ __forceinline__ AdamTensor from_element(const AdamTensor& T, int64_t begin) {
  AdamTensor t = T;
  t.param = static_cast<char*>(T.param) + begin * (PK == PARAM_F32 ? 4 : 2);
  t.master = PK == PARAM_BF16_MASTER ? T.master + begin : nullptr;
  t.grad = static_cast<const char*>(T.grad) + begin * (GK == GRAD_F32 ? 4 : 2);
  t.m = static_cast<char*>(T.m) + begin * (SK == STATE_F32 ? 4 : 1);
  t.v = static_cast<char*>(T.v) + begin * (SK == STATE_F32 ? 4 : 1);
  t.m_scale = T.m_scale + (begin >> 5);
  t.v_scale = T.v_scale + (begin >> 5);
  t.n = T.n - begin;
  t.counter = T.counter + (uint64_t)begin;
  return t;
}

template <int PK, bool WIDE>
__device__ __forceinline__ void load_param(const AdamTensor& T, uint32_t i, int left, float (&p)[VEC]) {
  if constexpr (PK == PARAM_F32) load8<WIDE>(static_cast<const float*>(T.param), i, left, p);
  else if constexpr (PK == PARAM_BF16_MASTER) load8<WIDE>(T.master, i, left, p);
  else load8<WIDE>(static_cast<const __nv_bfloat16*>(T.param), i, left, p);
}
template <int GK, bool WIDE>
__device__ __forceinline__ void load_grad(const AdamTensor& T, uint32_t i, int left, float (&g)[VEC]) {
  if constexpr (GK == GRAD_F32) load8<WIDE>(static_cast<const float*>(T.grad), i, left, g);
  else load8<WIDE>(static_cast<const __nv_bfloat16*>(T.grad), i, left, g);
}
// Two values to bf16, each up or down by 16 random bits (z's low half) added to its own bits and what lies below bf16
// cut off.  The conversion keeps infinities and NaN, which the sum itself would carry over (0x7fffffff to -0).
__device__ __forceinline__ uint32_t to_bf16_random(float lo, float hi, uint32_t z_lo, uint32_t z_hi) {
  uint32_t r;
  asm("cvt.rs.bf16x2.f32 %0, %1, %2, %3;" : "=r"(r) : "f"(hi), "f"(lo), "r"(__byte_perm(z_lo, z_hi, 0x5410)));
  return r;
}
__device__ __forceinline__ uint32_t to_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
template <int PK, bool WIDE>
__device__ __forceinline__ void store_param(const AdamTensor& T, uint32_t i, int left, const float (&p)[VEC],
                                            const uint32_t (&z)[VEC]) {
  if constexpr (PK == PARAM_F32) {
    store8<WIDE>(static_cast<float*>(T.param), i, left, p);
  } else {
    uint32_t w[VEC / 2];
#pragma unroll
    for (int j = 0; j < VEC; j += 2) {
      if constexpr (PK == PARAM_BF16) w[j / 2] = to_bf16_random(p[j], p[j + 1], z[j], z[j + 1]);
      else w[j / 2] = to_bf16(p[j], p[j + 1]);
    }
    store8<WIDE>(static_cast<__nv_bfloat16*>(T.param), i, left, w);
    if constexpr (PK == PARAM_BF16_MASTER) store8<WIDE>(T.master, i, left, p);
  }
}

// The f32-state step of elements i .. i + 7 of a tensor, `left` of them in range.
template <int PK, int GK, bool WIDE>
__device__ __forceinline__ void step8_f32(const AdamTensor& T, const AdamConstants& h, uint32_t i, int left) {
  float p[VEC], g[VEC], m[VEC], v[VEC];
  load_param<PK, WIDE>(T, i, left, p);
  load_grad<GK, WIDE>(T, i, left, g);
  load8<WIDE>(static_cast<const float*>(T.m), i, left, m);
  load8<WIDE>(static_cast<const float*>(T.v), i, left, v);
  uint32_t z[VEC];
  if constexpr (PK == PARAM_BF16) rounding_bits((T.counter + (uint64_t)i) >> 3, h.seed, z);
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    const float gj = h.c * g[j];
    m[j] = fmaf(h.beta1, m[j], h.one_minus_beta1 * gj);
    v[j] = fmaf(h.beta2, v[j], h.one_minus_beta2 * gj * gj);
    const float update = (m[j] * h.inv_bc1) / fmaf(sqrtf(v[j]), h.inv_bc2_sqrt, h.eps) + h.weight_decay * p[j];
    p[j] = fmaf(-h.lr, update, p[j]);
  }
  store_param<PK, WIDE>(T, i, left, p, z);
  store8<WIDE>(static_cast<float*>(T.m), i, left, m);
  store8<WIDE>(static_cast<float*>(T.v), i, left, v);
}

struct Mx8Constants {
  float beta1, beta2_sqrt, k1, k2, root_factor, root_offset, decay;
  uint32_t seed;
};
__device__ __forceinline__ Mx8Constants mx8_constants_of(const AdamHyper& h, const AdamTensor& T, float c) {
  // without a rate, or with one that f32 cannot divide by, the divisor is as large as can be, and the quotient 0 (an
  // infinite one would make NaN of a root that is 0)
  const float rate = -T.lr * h.inv_bc1;
  const bool none = rate == 0.0f;
  auto over_rate = [&](float x) { return none ? FLT_MAX : fminf(fmaxf(x / rate, -FLT_MAX), FLT_MAX); };
  return {h.beta1, h.beta2_sqrt, c * h.one_minus_beta1, c * h.one_minus_beta2_sqrt, over_rate(h.inv_bc2_sqrt),
          over_rate(h.eps), -T.lr * T.weight_decay, h.seed};
}

// The 8-bit-state step of elements i .. i + 7 (`left` of them in range) on values that were loaded: parameters,
// gradients, E4M3 bytes and scale bytes.  All threads of a warp come here together.
template <int PK, bool WIDE>
__device__ __forceinline__ void step8_mx8(const AdamTensor& T, const Mx8Constants& h, uint32_t i, int left,
                                          float (&p)[VEC], const float (&g)[VEC], uint2 mq, uint2 rq, int mb, int rb) {
  F2 m[VEC / 2], r[VEC / 2];
  from_e4m3(mq, m);
  from_e4m3(rq, r);
  uint32_t z[VEC];
  rounding_bits((T.counter + (uint64_t)i) >> 3, h.seed, z);
  // m = b1 m + k1 g;  v = (sqrt(b2) r)^2 + (k2 g)^2;  p = p + decay p + m / (a sqrt(v) + b), the rate in a and b
  const F2 ms = f2(h.beta1 * power_of_two(mb)), rs = f2(h.beta2_sqrt * power_of_two(rb));
  const F2 k1 = f2(h.k1), k2 = f2(h.k2), a = f2(h.root_factor), b = f2(h.root_offset), decay = f2(h.decay);
#pragma unroll
  for (int j = 0; j < VEC / 2; ++j) {
    const F2 gj = f2(g[2 * j], g[2 * j + 1]);
    m[j] = fma2(m[j], ms, mul2(gj, k1));
    const F2 r0 = mul2(r[j], rs), g2 = mul2(gj, k2);
    float v0, v1, d0, d1;
    split(fma2(r0, r0, mul2(g2, g2)), v0, v1);
    r[j] = f2(fast_sqrt(v0), fast_sqrt(v1));
    split(fma2(r[j], a, b), d0, d1);
    const F2 pj = f2(p[2 * j], p[2 * j + 1]);
    split(fma2(m[j], f2(fast_inverse(d0), fast_inverse(d1)), fma2(pj, decay, pj)), p[2 * j], p[2 * j + 1]);
  }
  store_param<PK, WIDE>(T, i, left, p, z);
  // (looked for once per thread: without the branch, in every element, the step was 4% slower)
  float am = thread_max(m), ar = thread_max(r);
  if (fmaxf(am, ar) == INFINITY) {
    infinities_to_nan(m);
    infinities_to_nan(r);
    am = thread_max(m), ar = thread_max(r);
  }
  const int bm = scale_byte(block_max(am)), br = scale_byte(block_max(ar));
  const F2 im = f2(power_of_two(254 - bm)), ir = f2(power_of_two(254 - br));
#pragma unroll
  for (int j = 0; j < VEC / 2; ++j) {
    m[j] = to_grid(mul2(m[j], im), f2(high_bits(z[2 * j]), high_bits(z[2 * j + 1])));
    const F2 y = mul2(r[j], ir);
    float y0, y1, q0, q1;
    split(y, y0, y1);
    split(to_grid(y, f2(low_bits(z[2 * j]), low_bits(z[2 * j + 1]))), q0, q1);
    // a nonzero root below the least E4M3 value becomes that value (and NaN, of which y > 0 is false, stays)
    if (y0 > 0.0f) q0 = fmaxf(q0, 0.001953125f);
    if (y1 > 0.0f) q1 = fmaxf(q1, 0.001953125f);
    r[j] = f2(q0, q1);
  }
  store_e4m3<WIDE>(static_cast<uint8_t*>(T.m), i, left, m);
  store_e4m3<WIDE>(static_cast<uint8_t*>(T.v), i, left, r);
  if ((WIDE || left > 0) && (i & 31) == 0) {
    T.m_scale[i >> 5] = (uint8_t)bm;
    T.v_scale[i >> 5] = (uint8_t)br;
  }
}

template <int PK>
__device__ __forceinline__ bool aligned_tensor(const AdamTensor& T) {
  return aligned_to(T.param, 16) && aligned_to(T.grad, 16) && aligned_to(T.m, 16) && aligned_to(T.v, 16) &&
         (PK != PARAM_BF16_MASTER || aligned_to(T.master, 16));
}
__device__ __forceinline__ AdamConstants constants_of(const AdamHyper& h, const AdamTensor& T, float c) {
  return {c, h.beta1, h.one_minus_beta1, h.beta2, h.one_minus_beta2, h.eps, h.inv_bc1, h.inv_bc2_sqrt, T.lr,
          T.weight_decay, h.seed};
}

// f32 states: a block takes 2048 elements.
template <int PK, int GK, int CAP>
__global__ void __launch_bounds__(ADAM_THREADS)
    adamw_kernel(const __grid_constant__ Table<AdamTensor, CAP> tab, const AdamHyper h,
                 const float* __restrict__ grad_scale) {
  const float c = grad_scale != nullptr ? *grad_scale : 1.0f;
  if (isnan(c)) return;
  const int k = tensor_of(tab, blockIdx.x);
  const AdamTensor T = from_element<PK, GK, STATE_F32>(tab.t[k], (int64_t)(blockIdx.x - tab.first[k]) * PASS);
  const uint32_t i = threadIdx.x * VEC;
  const int left = min(VEC, max(0, (int)min((int64_t)PASS, T.n) - (int)i));
  const AdamConstants hc = constants_of(h, T, c);
  if (left == VEC && aligned_tensor<PK>(T)) step8_f32<PK, GK, true>(T, hc, i, left);
  else step8_f32<PK, GK, false>(T, hc, i, left);
}

// 8-bit states: a block takes `passes` times 2048 elements, each warp its 256 of every pass.  The lanes of a warp
// copy the elements of the passes ahead into the warp's slots of a ring in shared memory (cp.async, 16 bytes next
// to 16 bytes: copies that leave half a 32-byte sector to a second one cost a fifth of the bandwidth), so that
// loads stay in flight under the arithmetic without registers, and without barriers between warps.  The scale
// bytes of the two passes ahead are held in registers (one ahead was 0.13 ms slower of 0.69).
constexpr int MX8_THREADS = 256;
constexpr int MX8_PASS = MX8_THREADS * VEC;
constexpr int MX8_MAX_PASSES = 8;
constexpr int SCALES_AHEAD = 2;
template <int PK, int GK>
struct Ring {
  static constexpr int P = PK == PARAM_BF16 ? 1 : 2, G = GK == GRAD_BF16 ? 1 : 2;  // 16-byte slots of a lane
  static constexpr int SLOTS = P + G + 1;                                        // the last: m and sqrt(v)
  static constexpr int STAGES = 3;
  static constexpr int STAGE_BYTES = SLOTS * 32 * 16;  // of a warp
  static constexpr int BYTES = STAGES * STAGE_BYTES * (MX8_THREADS / 32);
};
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
}
// 8 elements of a lane from its warp's slots of an array: 1 (bf16) or 2 (f32) pieces of 16 bytes
__device__ __forceinline__ void from_slots(const uint4* slots, int lane, float (&x)[VEC], std::integral_constant<int, 1>) {
  const uint4 a = slots[lane];
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = __uint_as_float(w[j] << 16);
    x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
  }
}
__device__ __forceinline__ void from_slots(const uint4* slots, int lane, float (&x)[VEC], std::integral_constant<int, 2>) {
  const uint4 a = slots[2 * lane], b = slots[2 * lane + 1];
  const uint32_t w[VEC] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int j = 0; j < VEC; ++j) x[j] = __uint_as_float(w[j]);
}

template <int PK, int GK, int CAP>
__global__ void __launch_bounds__(MX8_THREADS, 4)
    adamw_mx8_kernel(const __grid_constant__ Table<AdamTensor, CAP> tab, const AdamHyper h, int passes,
                     const float* __restrict__ grad_scale) {
  using R = Ring<PK, GK>;
  extern __shared__ uint4 ring[];  // [warps][STAGES][SLOTS][32]
  const float c = grad_scale != nullptr ? *grad_scale : 1.0f;
  if (isnan(c)) return;
  const int k = tensor_of(tab, blockIdx.x);
  const AdamTensor T =
      from_element<PK, GK, STATE_MX8>(tab.t[k], (int64_t)(blockIdx.x - tab.first[k]) * passes * MX8_PASS);
  const Mx8Constants hc = mx8_constants_of(h, T, c);
  const int lane = threadIdx.x & 31;
  const int end = (int)min(T.n, (int64_t)passes * MX8_PASS);
  const int warp_begin = (threadIdx.x & ~31) * VEC, first = threadIdx.x * VEC;
  // passes in which all 256 elements of this warp are in range: those go through the ring
  const int room = end - warp_begin - 32 * VEC;
  const int full = aligned_tensor<PK>(T) && room >= 0 ? room / MX8_PASS + 1 : 0;
  const char* p_from = static_cast<const char*>(PK == PARAM_BF16_MASTER ? (const void*)T.master : T.param);
  const char* g_from = static_cast<const char*>(T.grad);
  const uint8_t* m_from = static_cast<const uint8_t*>(T.m);
  const uint8_t* r_from = static_cast<const uint8_t*>(T.v);
  const uint4* my_ring = ring + (threadIdx.x >> 5) * (R::STAGES * R::SLOTS * 32);
  const uint32_t slots = (uint32_t)__cvta_generic_to_shared(my_ring + lane);

  auto fetch = [&](int q, int stage) {
    if (q < full) {
      const uint32_t to = slots + stage * R::STAGE_BYTES;
      const uint32_t i = warp_begin + q * MX8_PASS;
#pragma unroll
      for (int j = 0; j < R::P; ++j) copy16(to + j * 512, p_from + (i * (2 * R::P) + 512 * j + 16 * lane));
#pragma unroll
      for (int j = 0; j < R::G; ++j) copy16(to + (R::P + j) * 512, g_from + (i * (2 * R::G) + 512 * j + 16 * lane));
      copy8(to + (R::SLOTS - 1) * 512, m_from + (i + VEC * lane));
      copy8(to + (R::SLOTS - 1) * 512 + 8, r_from + (i + VEC * lane));
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int q = 0; q < R::STAGES - 1; ++q) fetch(q, q);
  int mb[SCALES_AHEAD] = {}, rb[SCALES_AHEAD] = {};  // scale bytes of the passes ahead
#pragma unroll
  for (int q = 0; q < SCALES_AHEAD; ++q) {
    const uint32_t at = (uint32_t)(first + q * MX8_PASS) >> 5;
    if (q < full) mb[q] = T.m_scale[at], rb[q] = T.v_scale[at];
  }
  int stage = 0;
  for (int q = 0; q < full; ++q) {
    // the stage before this one is free once all lanes have read it
    __syncwarp();
    fetch(q + R::STAGES - 1, stage == 0 ? R::STAGES - 1 : stage - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(R::STAGES - 1) : "memory");
    __syncwarp();
    const uint32_t i = first + q * MX8_PASS;
    const int mb_now = mb[0], rb_now = rb[0];
#pragma unroll
    for (int d = 0; d + 1 < SCALES_AHEAD; ++d) mb[d] = mb[d + 1], rb[d] = rb[d + 1];
    if (q + SCALES_AHEAD < full) {
      const uint32_t at = (i + SCALES_AHEAD * MX8_PASS) >> 5;
      mb[SCALES_AHEAD - 1] = T.m_scale[at], rb[SCALES_AHEAD - 1] = T.v_scale[at];
    }
    const uint4* from = my_ring + stage * (R::SLOTS * 32);
    float p[VEC], g[VEC];
    from_slots(from, lane, p, std::integral_constant<int, R::P>());
    from_slots(from + R::P * 32, lane, g, std::integral_constant<int, R::G>());
    const uint4 mr = from[(R::SLOTS - 1) * 32 + lane];
    step8_mx8<PK, true>(T, hc, i, VEC, p, g, make_uint2(mr.x, mr.y), make_uint2(mr.z, mr.w), mb_now, rb_now);
    stage = stage == R::STAGES - 1 ? 0 : stage + 1;
  }
  // what is left: the tensor's last elements, or a tensor that is not aligned
  for (int base = warp_begin + full * MX8_PASS; base < end; base += MX8_PASS) {
    const uint32_t i = base + lane * VEC;
    const int left = min(VEC, max(0, end - (int)i));
    float p[VEC], g[VEC];
    load_param<PK, false>(T, i, left, p);
    load_grad<GK, false>(T, i, left, g);
    const uint2 mq = load_e4m3(m_from, i, left), rq = load_e4m3(r_from, i, left);
    step8_mx8<PK, false>(T, hc, i, left, p, g, mq, rq, left > 0 ? T.m_scale[i >> 5] : 1, left > 0 ? T.v_scale[i >> 5] : 1);
  }
}

// ----------------------------------------------------------------------------- gradient norm
// Each block sums its chunks' squares in f32, 8 sums to a thread and a tree over the threads; one warp of the
// block that comes last in the call adds the blocks' sums in f64 in a fixed order, so that the result does not
// depend on the order of arrival.  Squares below 2^-149, of gradients below 2.6e-23, count as 0.
// Bound by DRAM reads: 354 million f32 gradients in 0.198 ms, 7.15 TB/s (64 warps an SM in flight, no copy through
// shared memory); small sets by the launch and the last block's turn: 96 tensors of 1 to 30,011 elements 5.7 us (with
// f64 sums within the blocks 8.6).
__device__ __forceinline__ float warp_total(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// A block whose sum of squares leaves f32's range (or has a NaN in it) takes its chunks again, every gradient times
// 2^-80, and hands out the root of that sum, negative, in the sum's place: a norm that f32 can hold is then found whatever
// the squares are.  (A call without such blocks is as fast as before; with f64 in here, or a look at every partial
// sum's sign at the end, it was 0.3 us of 7.9 slower.)
template <int CAP>
__device__ __forceinline__ float scaled_block_norm(const Table<GradTensor, CAP>& tab, float* warp_sum) {
  constexpr float DOWN = 8.27180613e-25f, UP = 1.20892582e24f;  // 2^-80 and 2^80
  float s = 0.0f;
#pragma unroll 1
  for (int chunk = blockIdx.x; chunk < tab.first[tab.count]; chunk += gridDim.x) {
    const int k = tensor_of(tab, chunk);
    const GradTensor& T = tab.t[k];
    const int64_t begin = (int64_t)(chunk - tab.first[k]) * NORM_CHUNK;
    const int end = (int)min((int64_t)NORM_CHUNK, T.n - begin);
    const char* grad = static_cast<const char*>(T.grad) + begin * (T.bf16 ? 2 : 4);
    float of_chunk = 0.0f;
#pragma unroll 1
    for (int i = threadIdx.x; i < end; i += NORM_THREADS) {
      const float g = DOWN * (T.bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(grad)[i])
                                     : reinterpret_cast<const float*>(grad)[i]);
      of_chunk = fmaf(g, g, of_chunk);
    }
    s += of_chunk;
  }
  s = warp_total(s);
  if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = s;
  __syncthreads();
  s = warp_total((threadIdx.x & 31) < NORM_THREADS / 32 ? warp_sum[threadIdx.x & 31] : 0.0f);
  return -sqrtf(s) * UP;
}

template <int CAP>
__global__ void __launch_bounds__(NORM_THREADS)
    grad_norm_kernel(const __grid_constant__ Table<GradTensor, CAP> tab, int first_block, int total_blocks, float max_norm,
                     float* __restrict__ out, unsigned* __restrict__ ticket, float* __restrict__ partials) {
  __shared__ float warp_sum[NORM_THREADS / 32];
  __shared__ unsigned turn;
  float acc[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) acc[j] = 0.0f;
  for (int chunk = blockIdx.x; chunk < tab.first[tab.count]; chunk += gridDim.x) {
    const int k = tensor_of(tab, chunk);
    const GradTensor& T = tab.t[k];
    const int64_t begin = (int64_t)(chunk - tab.first[k]) * NORM_CHUNK;
    const char* grad = static_cast<const char*>(T.grad) + begin * (T.bf16 ? 2 : 4);
    const int end = (int)min((int64_t)NORM_CHUNK, T.n - begin);
    const bool aligned = aligned_to(T.grad, 16);
#pragma unroll
    for (int q = 0; q < NORM_CHUNK / (NORM_THREADS * VEC); ++q) {
      const int i = (q * NORM_THREADS + threadIdx.x) * VEC;
      const int left = min(VEC, max(0, end - i));
      float g[VEC];
      if (left == VEC && aligned) {
        if (T.bf16) load8<true>(reinterpret_cast<const __nv_bfloat16*>(grad), i, left, g);
        else load8<true>(reinterpret_cast<const float*>(grad), i, left, g);
      } else {
        if (T.bf16) load8<false>(reinterpret_cast<const __nv_bfloat16*>(grad), i, left, g);
        else load8<false>(reinterpret_cast<const float*>(grad), i, left, g);
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) acc[j] = fmaf(g[j], g[j], acc[j]);
    }
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < VEC; ++j) s += acc[j];
  s = warp_total(s);
  if (lane == 0) warp_sum[warp] = s;
  __syncthreads();
  // the ticket counts the blocks in its low half, those that hand out a root in its high half
  constexpr unsigned ROOT = 0x10000u, AGAIN = 0xffffffffu;
  static_assert(NORM_MAX_PARTIALS < ROOT, "halves of the ticket");
  auto hand_out = [&](float x, unsigned root) {
    partials[first_block + blockIdx.x] = x;
    __threadfence();
    turn = atomicAdd(ticket, 1u + root) + root;
  };
  if (warp == 0) {
    s = warp_total(lane < NORM_THREADS / 32 ? warp_sum[lane] : 0.0f);
    if (lane == 0) {
      if (s < INFINITY) hand_out(s, 0u);
      else turn = AGAIN;
    }
  }
  __syncthreads();
  if (turn == AGAIN) {
    s = scaled_block_norm(tab, warp_sum);
    if (threadIdx.x == 0) hand_out(s, ROOT);
    __syncthreads();
  }
  if (turn % ROOT != (unsigned)(total_blocks - 1) || warp != 0) return;
  __threadfence();
  double total = 0.0;
  if (turn < ROOT) {
    for (int b = lane; b < total_blocks; b += 32) total += (double)__ldcg(&partials[b]);
  } else {
#pragma unroll 1
    for (int b = lane; b < total_blocks; b += 32) {
      const double x = (double)__ldcg(&partials[b]);
      total += x < 0.0 ? x * x : x;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if (lane == 0) {
    const float norm = (float)sqrt(total);
    out[0] = norm;
    out[1] = isfinite(norm) ? fminf(1.0f, max_norm / (norm + 1e-6f)) : __int_as_float(0x7fffffff);
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
    const int64_t n = chunks_of(tensors[i].n);
    for (int64_t c = chunks; c < std::min<int64_t>(chunks + n, tab.MAPPED); ++c) tab.of_chunk[c] = (uint8_t)i;
    chunks += n;
    if (chunks > INT32_MAX) return -1;
  }
  tab.first[count] = (int32_t)chunks;
  tab.count = count;
  return chunks;
}

template <int PK, int GK, int CAP>
cudaError_t launch_f32(const AdamTensor* tensors, int count, const AdamHyper& h, const float* scale, cudaStream_t st) {
  Table<AdamTensor, CAP> tab;
  const int64_t chunks = fill_table(tab, tensors, count, [](int64_t n) { return (n + PASS - 1) / PASS; });
  if (chunks < 0) return cudaErrorInvalidValue;
  if (chunks == 0) return cudaSuccess;
  adamw_kernel<PK, GK, CAP><<<(int)chunks, ADAM_THREADS, 0, st>>>(tab, h, scale);
  return cudaGetLastError();
}

template <int PK, int GK, int CAP>
cudaError_t launch_mx8(const AdamTensor* tensors, int count, const AdamHyper& h, const float* scale, int n_sm,
                       cudaStream_t st) {
  // as many passes to a block, up to 8, as leave 3 blocks for each of the 4 an SM holds (longer blocks read memory
  // further apart at one time: 32 passes were up to 6% slower than 8, 4 passes 3% slower with bf16 gradients)
  int64_t total = 0;
  for (int i = 0; i < count; ++i) total += (tensors[i].n + MX8_PASS - 1) / MX8_PASS;
  const int passes = (int)std::min<int64_t>(MX8_MAX_PASSES, std::max<int64_t>(1, total / (12 * n_sm)));
  const int64_t chunk = (int64_t)passes * MX8_PASS;
  Table<AdamTensor, CAP> tab;
  const int64_t chunks = fill_table(tab, tensors, count, [chunk](int64_t n) { return (n + chunk - 1) / chunk; });
  if (chunks < 0) return cudaErrorInvalidValue;
  if (chunks == 0) return cudaSuccess;
  auto kernel = adamw_mx8_kernel<PK, GK, CAP>;
  const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Ring<PK, GK>::BYTES);
  if (err != cudaSuccess) return err;
  kernel<<<(int)chunks, MX8_THREADS, Ring<PK, GK>::BYTES, st>>>(tab, h, passes, scale);
  return cudaGetLastError();
}

template <int PK, int GK>
cudaError_t launch_kind(const AdamTensor* t, int count, int state, const AdamHyper& h, const float* scale,
                        int n_sm, cudaStream_t st) {
  const bool small = count <= SMALL_TABLE;
  if (state == STATE_F32)
    return small ? launch_f32<PK, GK, SMALL_TABLE>(t, count, h, scale, st)
                 : launch_f32<PK, GK, OPTIM_TABLE>(t, count, h, scale, st);
  return small ? launch_mx8<PK, GK, SMALL_TABLE>(t, count, h, scale, n_sm, st)
               : launch_mx8<PK, GK, OPTIM_TABLE>(t, count, h, scale, n_sm, st);
}

template <int CAP>
cudaError_t launch_norm(const GradTensor* tensors, int count, int blocks, int first_block, int total_blocks,
                        float max_norm, float* out, void* ws, cudaStream_t st) {
  Table<GradTensor, CAP> tab;
  if (fill_table(tab, tensors, count, grad_norm_chunks) < 0) return cudaErrorInvalidValue;
  grad_norm_kernel<CAP><<<blocks, NORM_THREADS, 0, st>>>(
      tab, first_block, total_blocks, max_norm, out, static_cast<unsigned*>(ws),
      reinterpret_cast<float*>(static_cast<char*>(ws) + NORM_PARTIALS_OFFSET));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_adamw(const AdamTensor* t, int count, int param, int grad, int state, const AdamHyper& h,
                         const float* grad_scale, int n_sm, cudaStream_t st) {
  switch (param * 2 + grad) {
    case PARAM_F32 * 2 + GRAD_F32: return launch_kind<PARAM_F32, GRAD_F32>(t, count, state, h, grad_scale, n_sm, st);
    case PARAM_F32 * 2 + GRAD_BF16: return launch_kind<PARAM_F32, GRAD_BF16>(t, count, state, h, grad_scale, n_sm, st);
    case PARAM_BF16_MASTER * 2 + GRAD_F32: return launch_kind<PARAM_BF16_MASTER, GRAD_F32>(t, count, state, h, grad_scale, n_sm, st);
    case PARAM_BF16_MASTER * 2 + GRAD_BF16: return launch_kind<PARAM_BF16_MASTER, GRAD_BF16>(t, count, state, h, grad_scale, n_sm, st);
    case PARAM_BF16 * 2 + GRAD_F32: return launch_kind<PARAM_BF16, GRAD_F32>(t, count, state, h, grad_scale, n_sm, st);
    default: return launch_kind<PARAM_BF16, GRAD_BF16>(t, count, state, h, grad_scale, n_sm, st);
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
