// The grouped E4M3 product of few rows a group (include/mok.h, mok_fp8_matmul): out[r][n] = sum_b xs[b][r]
// ws[e][n / 128][b] sum_{k in b} x[r][k] w[e][n][k].  With a few rows the weights are the bytes, each read
// once; so nothing is staged: a warp loads 16 weight rows x 128 k into registers as they lie (4 16-byte loads a lane),
// as the A fragments of mma.m16n8k32, with 8 rows of x the B fragments.  Which k a fragment position holds does not
// matter as long as A and B agree, so a lane takes bytes 16 t .. and 64 + 16 t .. of a row's 128 (t = lane % 4) and the
// fragments are those words in order.
//
// A block is one 16-row piece of one group's weights, its 8 warps every eighth block of 128 along K, each with its
// own f32 sums of scaled blocks; they are added in warp order at the end.  Groups of more than 8 NT rows go round
// again (the weights then come from L2).
#include <cuda_bf16.h>

#include <algorithm>

#include "fp8.cuh"

namespace mok {
namespace {

constexpr int WARPS = 8;

__device__ __forceinline__ void mma_e4m3(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The 32 bytes of block [k0, k0 + 128) of a row that lane quarter t holds; zeros behind K (a row starts at a multiple
// of 16 bytes, so a 16-byte load that starts in front of K stays in the row's stride).
__device__ __forceinline__ void load_words(const uint8_t* row, int64_t k0, int64_t K, int t, uint32_t (&w)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t k = k0 + 64 * h + 16 * t;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (k < K) {
      v = __ldg(reinterpret_cast<const uint4*>(row + k));
      if (k + 16 > K) {
        const int n = (int)(K - k);  // 1 .. 15 bytes stay
        uint32_t* p = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int left = n - 4 * i;
          p[i] = left >= 4 ? p[i] : left <= 0 ? 0u : p[i] & ((1u << (8 * left)) - 1);
        }
      }
    }
    w[4 * h] = v.x;
    w[4 * h + 1] = v.y;
    w[4 * h + 2] = v.z;
    w[4 * h + 3] = v.w;
  }
}

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <int NT, typename OUT>
__global__ void __launch_bounds__(32 * WARPS) fp8_few_kernel(const Fp8MatmulArgs a, int pieces) {
  __shared__ float part[WARPS][8 * NT][17];
  const int e = blockIdx.x / pieces;
  const int64_t n0 = (int64_t)(blockIdx.x % pieces) * 16;
  int64_t lo = 0, hi = a.R;
  if (a.offsets != nullptr) {
    lo = fp8_offset(a.offsets[e], 0, a.R);
    hi = fp8_offset(a.offsets[e + 1], (int)lo, a.R);
  }
  if (lo >= hi) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int nkb = (int)((a.K + 127) / 128);
  // weight rows n0 + g and n0 + g + 8; behind the last one the last one again, whose sums are not stored
  const uint8_t* w0 = a.w + ((int64_t)e * a.N + min(n0 + g, a.N - 1)) * a.w_stride;
  const uint8_t* w1 = a.w + ((int64_t)e * a.N + min(n0 + g + 8, a.N - 1)) * a.w_stride;
  const float* ws = a.w_scale + ((int64_t)e * ((a.N + 127) / 128) + n0 / 128) * nkb;
  OUT* out = static_cast<OUT*>(a.out);
  for (int64_t r0 = lo; r0 < hi; r0 += 8 * NT) {
    float sum[NT][4] = {};
    for (int kb = warp; kb < nkb; kb += WARPS) {
      uint32_t wa[8], wb[8];
      load_words(w0, kb * 128ll, a.K, t, wa);
      load_words(w1, kb * 128ll, a.K, t, wb);
      const float s = __ldg(ws + kb);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if (r0 + 8 * j < hi) {
          uint32_t x[8];
          load_words(a.x + min(r0 + 8 * j + g, hi - 1) * a.x_stride, kb * 128ll, a.K, t, x);
          // columns 2 t and 2 t + 1 of the product are rows r0 + 8 j + 2 t, + 1
          const float* xs = a.x_scale + kb * a.x_scale_stride;
          const float s0 = s * __ldg(xs + min(r0 + 8 * j + 2 * t, hi - 1));
          const float s1 = s * __ldg(xs + min(r0 + 8 * j + 2 * t + 1, hi - 1));
          float d[4] = {};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t f[4] = {wa[2 * i], wb[2 * i], wa[2 * i + 1], wb[2 * i + 1]};
            mma_e4m3(d, f, x[2 * i], x[2 * i + 1]);
          }
          sum[j][0] = fmaf(d[0], s0, sum[j][0]);
          sum[j][1] = fmaf(d[1], s1, sum[j][1]);
          sum[j][2] = fmaf(d[2], s0, sum[j][2]);
          sum[j][3] = fmaf(d[3], s1, sum[j][3]);
        }
      }
    }
    __syncthreads();  // the round before has been read
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[warp][8 * j + 2 * t + (i & 1)][g + 8 * (i >> 1)] = sum[j][i];
    __syncthreads();
    for (int i = threadIdx.x; i < 8 * NT * 16; i += 32 * WARPS) {
      const int r = i >> 4, n = i & 15;
      if (r0 + r < hi && n0 + n < a.N) {
        float v = part[0][r][n];
#pragma unroll
        for (int w = 1; w < WARPS; ++w) v += part[w][r][n];
        put(out + (r0 + r) * a.out_stride + n0 + n, v);
      }
    }
  }
}

template <int NT>
cudaError_t few(const Fp8MatmulArgs& a, bool bf16_out, cudaStream_t st) {
  const int64_t pieces = (a.N + 15) / 16, blocks = pieces * a.E;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  if (bf16_out) fp8_few_kernel<NT, __nv_bfloat16><<<(unsigned)blocks, 32 * WARPS, 0, st>>>(a, (int)pieces);
  else fp8_few_kernel<NT, float><<<(unsigned)blocks, 32 * WARPS, 0, st>>>(a, (int)pieces);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp8_matmul(const Fp8MatmulArgs& a, bool bf16_out, int n_sm, cudaStream_t st) {
  const int64_t each = (a.R + a.E - 1) / a.E;  // rows of a group, about
  if (each > 32) return launch_fp8_product_pairs(a, bf16_out, n_sm, st);
  return each <= 8 ? few<1>(a, bf16_out, st) : each <= 16 ? few<2>(a, bf16_out, st) : few<4>(a, bf16_out, st);
}

}  // namespace mok
