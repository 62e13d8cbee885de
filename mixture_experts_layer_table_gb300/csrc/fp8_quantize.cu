// Quantisers to E4M3 with an f32 scale for each block of 128 (no counterpart on the pages, whose second precision
// is MXFP8; this is the layout of checkpoints in 8 bits with 128-blocks): scale = max(amax, 2^-110) / 448,
// element = E4M3 nearest to 448 x / amax, ties to even.
//   along the row        q [R][C], scale [C / 128][R]: both operands of x W^T and dy W have their sums along it
//   along the tokens     qt [C][P], qt_scale [P / 128][C]: the weight gradient sums over an expert's rows; each
//                        expert's rows start at a multiple of 128 of P, zeros behind its last
//   128 x 128 (weights)  q [N][K] and qt [K][N] with the same elements
// The source is rows in hand, rows gathered by a schedule table (with their gates), the SwiGLU of [h | u] rows, or
// its gradient.  One read of the source gives both layouts.
//
// A block of 256 threads takes a tile of 16 RPT rows x 128 columns: half-warp w holds rows RPT w .. RPT w + RPT - 1,
// lane l of it columns 8 l .. 8 l + 7, so that a row's maximum is 4 shuffles, a store of a row 128 bytes and, with
// RPT = 8, a lane's 8 rows of a column one 8-byte word of the transposed tile.
#include <cuda_bf16.h>

#include <algorithm>

#include "f32x2.cuh"
#include "fp8.cuh"
#include "mx.cuh"
#include "status.cuh"

namespace mok {
namespace {

constexpr int THREADS = 256;
constexpr float LEAST = 7.703719777548943e-34f;  // 2^-110
constexpr float BIG = 3.4028234663852886e38f;

// What a block's elements are divided by, in the form the quotient is made of.
struct Divisor {
  float a, inv;  // amax / 512 (exact), its reciprocal
};
__device__ __forceinline__ Divisor divisor(float amax) {
  Divisor d;
  d.a = fmaxf(amax, LEAST) * (1.0f / 512);
  d.inv = 1.0f / d.a;
  return d;
}
__device__ __forceinline__ float block_scale(float amax) { return fmaxf(amax, LEAST) / 448.0f; }

// (448 x / 512) / (amax / 512) for two elements: the product with the reciprocal, then one correction by the
// remainder x' - y a, which the FMA forms exactly.  A quotient that is a multiple of few bits (a border between two
// E4M3 values, common with bf16 inputs) comes out as itself, so that ties go to even as they should.  A NaN
// or an infinity gives NaN (inf - inf in the remainder).
__device__ __forceinline__ uint16_t quantize2(float x0, float x1, F2 a0a1, F2 i0i1) {
  const F2 x = mul2(f2(x0, x1), f2(0.875f));
  const F2 y = mul2(x, i0i1);
  float y0, y1, a0, a1;
  split(y, y0, y1);
  split(a0a1, a0, a1);
  const F2 r = fma2(f2(-y0, -y1), a0a1, x);
  split(fma2(r, i0i1, y), y0, y1);
  return e4m3x2_from_f32(y0, y1);
}
__device__ __forceinline__ uint2 quantize8(const float (&v)[8], F2 a, F2 inv) {
  uint2 o;
  o.x = quantize2(v[0], v[1], a, inv) | (uint32_t)quantize2(v[2], v[3], a, inv) << 16;
  o.y = quantize2(v[4], v[5], a, inv) | (uint32_t)quantize2(v[6], v[7], a, inv) << 16;
  return o;
}

// The magnitude that counts for a block: infinities and NaN stay out of it (their elements become NaN, the
// others what they are without them).
__device__ __forceinline__ float magnitude(float v) {
  const float m = fabsf(v);
  return m <= BIG ? m : 0.0f;
}

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }

// Columns c .. c + 7 of a row of `width` elements; zeros behind its end.  VEC: the row is 16-byte aligned and
// width a multiple of 8.
template <bool VEC>
__device__ __forceinline__ void load8(const float* row, int64_t c, int64_t width, float (&v)[8]) {
  if (VEC) {
    if (c < width) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(row + c)), b = __ldg(reinterpret_cast<const float4*>(row + c) + 1);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
      return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.0f;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c + j < width ? __ldg(row + c + j) : 0.0f;
  }
}
template <bool VEC>
__device__ __forceinline__ void load8(const __nv_bfloat16* row, int64_t c, int64_t width, float (&v)[8]) {
  if (VEC) {
    uint4 w = make_uint4(0, 0, 0, 0);
    if (c < width) w = __ldg(reinterpret_cast<const uint4*>(row + c));
    const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(&w);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = __bfloat1622float2(b[j]);
      v[2 * j] = f.x;
      v[2 * j + 1] = f.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c + j < width ? __bfloat162float(row[c + j]) : 0.0f;
  }
}

// silu(h) = h sigmoid(h).  The accurate exponential and quotient: with the approximations (2^-21) a value on the other side of a
// border between two E4M3 values was ten times as frequent, and the kernel is bound by its memory all the same.
__device__ __forceinline__ float sigmoid(float h) { return 1.0f / (1.0f + expf(-h)); }

// Row r (of the sorted order) of the source, columns c .. c + 7.
template <int SRC, typename T, bool VEC>
__device__ __forceinline__ void source8(const Fp8QuantizeArgs& a, int64_t r, int64_t c, float (&v)[8]) {
  const T* x = static_cast<const T*>(a.x);
  if (SRC == FP8_PLAIN) {
    if (a.src_of == nullptr) {
      load8<VEC>(x + r * a.x_stride, c, a.C, v);
      return;
    }
    const int32_t s = __ldg(a.src_of + r);
    const bool ok = s >= 0 && s < a.T * a.k;
    if (!ok) {
      if (s != -1) report_status(a.status, MOK_DEV_INVALID_ROUTING, SITE_FP8_SOURCE);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.0f;
      return;
    }
    load8<VEC>(x + (int64_t)(s / a.k) * a.x_stride, c, a.C, v);
    if (a.gates != nullptr) {
      const float g = __ldg(a.gates + s);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= g;
    }
  } else if (SRC == FP8_SWIGLU) {
    const T* row = x + r * a.x_stride;
    float u[8];
    load8<VEC>(row, c, a.C, v);
    load8<VEC>(row + a.C, c, a.C, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = v[j] * sigmoid(v[j]) * u[j];
  } else {
    const int64_t I = a.C / 2;
    const T* row = x + r * a.x_stride;
    const T* grad = static_cast<const T*>(a.grad) + r * a.grad_stride;
    // VEC: I is a multiple of 8, so that a lane's columns lie in one half
    if (VEC) {
      const bool up = c >= I;
      const int64_t i = up ? c - I : c;
      float h[8], u[8], d[8];
      load8<true>(row, i, I, h);
      load8<true>(grad, i, I, d);
      if (!up) load8<true>(row + I, i, I, u);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float sg = sigmoid(h[j]);
        v[j] = up ? d[j] * h[j] * sg : d[j] * u[j] * sg * (1.0f + h[j] * (1.0f - sg));
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool up = c + j >= I;
        const int64_t i = up ? c + j - I : c + j;
        v[j] = 0.0f;
        if (c + j < a.C) {
          const float h = widen(row[i]), d = widen(grad[i]), sg = sigmoid(h);
          v[j] = up ? d * h * sg : d * widen(row[I + i]) * sg * (1.0f + h * (1.0f - sg));
        }
      }
    }
  }
}

// 8 bytes at p, of which `n` lie in front of the end.
__device__ __forceinline__ void store8(uint8_t* p, uint2 v, int64_t n) {
  if (n >= 8) {
    *reinterpret_cast<uint2*>(p) = v;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = (uint8_t)((j < 4 ? v.x >> (8 * j) : v.y >> (8 * (j - 4))) & 0xff);
  }
}

// The transposed tile in shared memory, 128 columns of 128 bytes: the 8-byte word of half-warp k lies at word
// k ^ (c / 8 mod 16) of column c, so that neither the writes (16 lanes with columns 8 apart) nor the reads (16 words of a
// column) meet in a bank.
__device__ __forceinline__ int tile_word(int c, int k) { return c * 16 + (k ^ ((c >> 3) & 15)); }

// bytes[i] of row i (two words) -> word j: byte i is byte j of row i.
__device__ __forceinline__ uint2 column_word(const uint2 (&rows)[8], int j) {
  const bool high = j >= 4;
  const int s = j & 3;
  const uint32_t sel = s | (s + 4) << 4;
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = __byte_perm(high ? rows[2 * i].y : rows[2 * i].x, high ? rows[2 * i + 1].y : rows[2 * i + 1].x, sel);
  return make_uint2(__byte_perm(h[0], h[1], 0x5410), __byte_perm(h[2], h[3], 0x5410));
}

// Writes the tile's 128 columns to qt rows (128 bytes each, `n` of them in front of the end), of which `cols` exist.
__device__ __forceinline__ void store_tile(const uint2* tile, uint8_t* qt, int64_t stride, int64_t cols, int64_t n) {
  const int k = threadIdx.x & 15;
#pragma unroll
  for (int s = 0; s < 8; ++s) {
    const int c = s * 16 + (threadIdx.x >> 4);
    if (c < cols) store8(qt + c * stride + 8 * k, tile[tile_word(c, k)], n - 8 * k);
  }
}

// ------------------------------------------------------------------ rows
// Tiles of 16 RPT rows along the rows only.
template <int SRC, typename T, bool VEC, int RPT>
__global__ void __launch_bounds__(THREADS) fp8_rows_kernel(const Fp8QuantizeArgs a, int col_blocks) {
  __shared__ float s_scale[16 * RPT];
  const int b = blockIdx.x % col_blocks;
  const int64_t r0 = (int64_t)(blockIdx.x / col_blocks) * (16 * RPT);
  const int w = threadIdx.x >> 4, l = threadIdx.x & 15;
  const int64_t c = (int64_t)b * FP8_BLOCK + 8 * l;
  float v[RPT][8];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int64_t r = r0 + w * RPT + i;
    if (r < a.R) source8<SRC, T, VEC>(a, r, c, v[i]);
    else
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
  }
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int64_t r = r0 + w * RPT + i;
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, magnitude(v[i][j]));
#pragma unroll
    for (int s = 8; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
    const Divisor d = divisor(m);
    const uint2 bytes = quantize8(v[i], f2(d.a), f2(d.inv));
    if (r < a.R && c < a.C) store8(a.q + r * a.q_stride + c, bytes, a.C - c);
    if (l == 0) s_scale[w * RPT + i] = block_scale(m);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * RPT; i += THREADS)
    if (r0 + i < a.R) a.scale[b * a.scale_stride + r0 + i] = s_scale[i];
}

// ------------------------------------------------------------------ rows and columns
// A tile is 128 rows of one expert (of the padded order) x 128 columns.  A block takes `group` column blocks of
// one row tile, after it has found the tile's expert: the offsets are read and scanned by the block itself.
template <int SRC, typename T, bool VEC>
__global__ void __launch_bounds__(THREADS, 2) fp8_columns_kernel(const Fp8QuantizeArgs a, int col_blocks, int group,
                                                                 int groups) {
  __shared__ uint2 tile[128 * 16];
  __shared__ float s_max[8][128];
  __shared__ float2 s_div[128];
  __shared__ float s_scale[128];
  __shared__ int s_warp[8], s_where[2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int p = blockIdx.x / groups;  // row tile
  // the expert whose 128-row blocks hold block p: a scan of the experts' blocks, 256 experts at a time
  if (threadIdx.x == 0) s_where[1] = 0;
  int before = 0;  // blocks of the experts before this round's
  for (int e0 = 0; e0 < a.E; e0 += THREADS) {
    const int e = e0 + threadIdx.x;
    int lo = 0, hi = 0;
    if (e < a.E) {
      lo = fp8_offset(a.offsets[e], 0, a.R);
      hi = fp8_offset(a.offsets[e + 1], lo, a.R);
    }
    const int mine = (hi - lo + 127) >> 7;
    int sum = mine;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, sum, s);
      if (lane >= s) sum += o;
    }
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i < warp) sum += s_warp[i];
      total += s_warp[i];
    }
    const int first = before + sum - mine;
    if (p >= first && p < first + mine) {
      s_where[0] = lo + (p - first) * 128;
      s_where[1] = min(128, hi - lo - (p - first) * 128);
    }
    before += total;
    __syncthreads();
  }
  const int64_t row0 = s_where[0];
  const int rows = s_where[1] == 0 ? 0 : (int)min((int64_t)s_where[1], a.R - row0);  // whatever the table says
  if (rows <= 0) return;  // behind the last expert's blocks
  const int w = threadIdx.x >> 4, l = threadIdx.x & 15;
  const int b_end = min(col_blocks, (int)(blockIdx.x % groups + 1) * group);
  for (int b = (blockIdx.x % groups) * group; b < b_end; ++b) {
    const int64_t c = (int64_t)b * FP8_BLOCK + 8 * l;
    float v[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (w * 8 + i < rows) source8<SRC, T, VEC>(a, row0 + w * 8 + i, c, v[i]);
      else
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    }
    float top[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) top[j] = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float m = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = magnitude(v[i][j]);
        top[j] = fmaxf(top[j], n);
        m = fmaxf(m, n);
      }
      if (a.q != nullptr) {
#pragma unroll
        for (int s = 8; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
        const Divisor d = divisor(m);
        const uint2 bytes = quantize8(v[i], f2(d.a), f2(d.inv));
        if (w * 8 + i < rows && c < a.C) store8(a.q + (row0 + w * 8 + i) * a.q_stride + c, bytes, a.C - c);
        if (l == 0) s_scale[w * 8 + i] = block_scale(m);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], 16));
    if (lane < 16) {
      float4* m = reinterpret_cast<float4*>(&s_max[warp][8 * l]);
      m[0] = make_float4(top[0], top[1], top[2], top[3]);
      m[1] = make_float4(top[4], top[5], top[6], top[7]);
    }
    __syncthreads();
    if (threadIdx.x < 128) {
      float m = s_max[0][threadIdx.x];
#pragma unroll
      for (int i = 1; i < 8; ++i) m = fmaxf(m, s_max[i][threadIdx.x]);
      const Divisor d = divisor(m);
      s_div[threadIdx.x] = make_float2(d.a, d.inv);
      const int64_t col = (int64_t)b * FP8_BLOCK + threadIdx.x;
      if (col < a.C) a.qt_scale[p * a.C + col] = block_scale(m);
    } else if (a.q != nullptr && (int)threadIdx.x - 128 < rows) {
      a.scale[b * a.scale_stride + row0 + threadIdx.x - 128] = s_scale[threadIdx.x - 128];
    }
    __syncthreads();
    uint2 bytes[8];
#pragma unroll
    for (int j = 0; j < 8; j += 2) {  // two columns at a time: their divisors in a pair
      const float2 d0 = s_div[8 * l + j], d1 = s_div[8 * l + j + 1];
      const F2 da = f2(d0.x, d1.x), di = f2(d0.y, d1.y);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t h = quantize2(v[i][j], v[i][j + 1], da, di);
        uint32_t& word = j < 4 ? bytes[i].x : bytes[i].y;
        word = (j & 3) == 0 ? h : word | h << 16;
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) tile[tile_word(8 * l + j, w)] = column_word(bytes, j);
    __syncthreads();
    store_tile(tile, a.qt + (int64_t)b * FP8_BLOCK * a.qt_stride + (int64_t)p * 128, a.qt_stride,
               a.C - (int64_t)b * FP8_BLOCK, 128);
    __syncthreads();  // the tile and the maxima are free again
  }
}

// ------------------------------------------------------------------ weights
template <typename T, bool VEC>
__global__ void __launch_bounds__(THREADS, 2) fp8_weights_kernel(const Fp8WeightsArgs a, int n_blocks, int k_blocks) {
  __shared__ uint2 tile[128 * 16];
  __shared__ float s_max[8];
  const int64_t e = blockIdx.x / ((int64_t)n_blocks * k_blocks);
  const int nb = (int)(blockIdx.x / k_blocks % n_blocks), kb = (int)(blockIdx.x % k_blocks);
  const int w = threadIdx.x >> 4, l = threadIdx.x & 15;
  const int64_t n0 = (int64_t)nb * FP8_BLOCK, k0 = (int64_t)kb * FP8_BLOCK, c = k0 + 8 * l;
  const T* x = static_cast<const T*>(a.w) + e * a.N * a.K;
  float v[8][8], m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t n = n0 + w * 8 + i;
    if (n < a.N) load8<VEC>(x + n * a.K, c, a.K, v[i]);
    else
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, magnitude(v[i][j]));
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, s_max[i]);
  const Divisor d = divisor(m);
  const F2 da = f2(d.a), di = f2(d.inv);
  uint2 bytes[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t n = n0 + w * 8 + i;
    bytes[i] = quantize8(v[i], da, di);
    if (a.q != nullptr && n < a.N && c < a.K) store8(a.q + (e * a.N + n) * a.q_stride + c, bytes[i], a.K - c);
  }
  if (threadIdx.x == 0) {
    if (a.q != nullptr) a.scale[(e * n_blocks + nb) * k_blocks + kb] = block_scale(m);
    if (a.qt != nullptr) a.qt_scale[(e * k_blocks + kb) * n_blocks + nb] = block_scale(m);
  }
  if (a.qt == nullptr) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) tile[tile_word(8 * l + j, w)] = column_word(bytes, j);
  __syncthreads();
  store_tile(tile, a.qt + (e * a.K + k0) * a.qt_stride + n0, a.qt_stride, a.K - k0, a.N - n0);
}

template <int SRC, typename T, bool VEC>
cudaError_t quantize(const Fp8QuantizeArgs& a, int n_sm, cudaStream_t st) {
  const int64_t col_blocks = (a.C + 127) / 128;
  if (a.qt == nullptr) {
    // 64-row tiles once they give every SM two blocks, else 16-row ones
    const bool wide = col_blocks * ((a.R + 63) / 64) >= 2 * n_sm;
    const int64_t blocks = col_blocks * (wide ? (a.R + 63) / 64 : (a.R + 15) / 16);
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    if (wide) fp8_rows_kernel<SRC, T, VEC, 4><<<(unsigned)blocks, THREADS, 0, st>>>(a, (int)col_blocks);
    else fp8_rows_kernel<SRC, T, VEC, 1><<<(unsigned)blocks, THREADS, 0, st>>>(a, (int)col_blocks);
    return cudaGetLastError();
  }
  const int64_t tiles = a.R / 128 + a.E;
  // column blocks of a block: up to 8 while there remain 4 blocks for each SM
  int group = 8;
  while (group > 1 && tiles * ((col_blocks + group - 1) / group) < 4 * n_sm) group /= 2;
  const int64_t groups = (col_blocks + group - 1) / group;
  if (tiles * groups > INT32_MAX) return cudaErrorInvalidValue;
  fp8_columns_kernel<SRC, T, VEC>
      <<<(unsigned)(tiles * groups), THREADS, 0, st>>>(a, (int)col_blocks, group, (int)groups);
  return cudaGetLastError();
}

bool aligned(const void* p, int64_t stride_bytes) {
  return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)stride_bytes) & 15u) == 0;
}

template <int SRC, typename T>
cudaError_t quantize(const Fp8QuantizeArgs& a, int n_sm, cudaStream_t st) {
  const int64_t item = sizeof(T);
  bool vec = aligned(a.x, a.x_stride * item) && (SRC == FP8_SWIGLU_GRAD ? a.C / 2 : a.C) % 8 == 0;
  if (SRC == FP8_SWIGLU_GRAD) vec = vec && aligned(a.grad, a.grad_stride * item);
  return vec ? quantize<SRC, T, true>(a, n_sm, st) : quantize<SRC, T, false>(a, n_sm, st);
}

template <typename T>
cudaError_t weights(const Fp8WeightsArgs& a, cudaStream_t st) {
  const int64_t n = (a.N + 127) / 128, k = (a.K + 127) / 128, blocks = a.E * n * k;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  const bool vec = aligned(a.w, a.K * (int64_t)sizeof(T)) && a.K % 8 == 0;
  if (vec) fp8_weights_kernel<T, true><<<(unsigned)blocks, THREADS, 0, st>>>(a, (int)n, (int)k);
  else fp8_weights_kernel<T, false><<<(unsigned)blocks, THREADS, 0, st>>>(a, (int)n, (int)k);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp8_quantize(const Fp8QuantizeArgs& a, int source, bool bf16, int n_sm, cudaStream_t st) {
  switch (source) {
    case FP8_PLAIN:
      return bf16 ? quantize<FP8_PLAIN, __nv_bfloat16>(a, n_sm, st) : quantize<FP8_PLAIN, float>(a, n_sm, st);
    case FP8_SWIGLU:
      return bf16 ? quantize<FP8_SWIGLU, __nv_bfloat16>(a, n_sm, st) : quantize<FP8_SWIGLU, float>(a, n_sm, st);
    default:
      return bf16 ? quantize<FP8_SWIGLU_GRAD, __nv_bfloat16>(a, n_sm, st)
                  : quantize<FP8_SWIGLU_GRAD, float>(a, n_sm, st);
  }
}

cudaError_t launch_fp8_weights(const Fp8WeightsArgs& a, bool bf16, cudaStream_t st) {
  return bf16 ? weights<__nv_bfloat16>(a, st) : weights<float>(a, st);
}

}  // namespace mok
