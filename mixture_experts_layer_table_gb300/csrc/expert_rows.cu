// Rows by a schedule table, outside the layer (no counterpart on the pages beyond the layer's own gather and
// merge: "把 MoE 通信延迟从 103μs 压到 18μs：Cursor 开源 GPU 内核 MoK", aientropygate.com, §03 ① and §04):
//   gather          x_g[r] = g[a] x[a / k], a = src_of[r]; a zero row where a = -1
//   merge           y[t] = sum_j g[t][j] o[row_of[t k + j]], j ascending, in f32, rounded once
//   merge backward  do[row_of[t k + j]] = g[t][j] dy[t],  dg[t][j] = <dy[t], o[row_of[t k + j]]>
// All three move rows and compute next to nothing: DRAM bounds them where there are many rows, the
// chain index -> row -> store where there are few.
#include <cuda_bf16.h>

#include <algorithm>

#include "expert_rows.cuh"
#include "ptx.cuh"
#include "status.cuh"

namespace mok {
namespace {

// A piece of a row: BYTES of T's, moved by one instruction.
template <typename T, int BYTES>
struct Piece {
  static constexpr int N = BYTES / (int)sizeof(T);
  T v[N];
};
template <typename T, int BYTES>
struct Raw;
template <typename T>
struct Raw<T, 16> { using type = uint4; };
template <typename T>
struct Raw<T, 4> { using type = uint32_t; };
template <typename T>
struct Raw<T, 2> { using type = uint16_t; };

__device__ __forceinline__ void load_raw(uint4& v, const void* p) {
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
}
// The same for a line that is read again soon: a token's row is read by its k experts, far apart in time.
__device__ __forceinline__ void load_keep(uint4& v, const void* p, uint64_t policy) {
  asm volatile("ld.global.nc.L1::no_allocate.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p), "l"(policy));
}
template <typename W>
__device__ __forceinline__ void load_keep(W& v, const void* p, uint64_t) { v = __ldg(static_cast<const W*>(p)); }
__device__ __forceinline__ void load_raw(uint32_t& v, const void* p) { v = __ldg(static_cast<const uint32_t*>(p)); }
__device__ __forceinline__ void load_raw(uint16_t& v, const void* p) {
  v = __ldg(static_cast<const unsigned short*>(p));
}
template <typename W>
__device__ __forceinline__ void store_raw(void* p, const W& v) {
  __stcs(static_cast<W*>(p), v);
}
__device__ __forceinline__ void store_raw(void* p, const uint16_t& v) {
  __stcs(static_cast<unsigned short*>(p), (unsigned short)v);
}

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void narrow(float& d, float v) { d = v; }
__device__ __forceinline__ void narrow(__nv_bfloat16& d, float v) { d = __float2bfloat16_rn(v); }

template <typename T, int BYTES, typename W>
__device__ __forceinline__ void unpack(const W& w, float (&f)[Piece<T, BYTES>::N]) {
  const Piece<T, BYTES>& p = reinterpret_cast<const Piece<T, BYTES>&>(w);
#pragma unroll
  for (int i = 0; i < Piece<T, BYTES>::N; ++i) f[i] = widen(p.v[i]);
}
template <typename T, int BYTES, typename W>
__device__ __forceinline__ void pack(W& w, const float (&f)[Piece<T, BYTES>::N]) {
  Piece<T, BYTES>& p = reinterpret_cast<Piece<T, BYTES>&>(w);
#pragma unroll
  for (int i = 0; i < Piece<T, BYTES>::N; ++i) narrow(p.v[i], f[i]);
}

// The source of row r, or -1 for a zero row; an index outside [0, n) other than -1 is reported.
__device__ __forceinline__ int64_t checked(int32_t i, int64_t n, int* status, int site) {
  if (i >= 0 && i < n) return i;
  if (i != -1) report_status(status, MOK_DEV_INVALID_ROUTING, site);
  return -1;
}

// V pieces of a row, X apart, from piece i on: all loaded, then all stored.  ALL: they are all there.
template <typename T, int BYTES, int V, int X, bool ALL, typename W>
__device__ __forceinline__ void copy_pieces(const char* s, char* d, int i, int pieces, bool gated, float g, const W*) {
  const uint64_t keep = BYTES == 16 ? l2_policy_evict_last() : 0;
  W v[V] = {};
  s += (int64_t)i * BYTES;
  d += (int64_t)i * BYTES;
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (ALL || i + j * X < pieces) load_keep(v[j], s + j * X * BYTES, keep);
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (ALL || i + j * X < pieces) {
      if (gated) {
        float f[Piece<T, BYTES>::N];
        unpack<T, BYTES>(v[j], f);
#pragma unroll
        for (int q = 0; q < Piece<T, BYTES>::N; ++q) f[q] *= g;
        pack<T, BYTES>(v[j], f);
      }
      store_raw(d + j * X * BYTES, v[j]);
    }
}

// X threads to a row, 128 / X rows to a block, 8 pieces of a thread in flight at once.  Short-lived blocks in row order, as
// the layer's own gather (rows.cu) found best, and the tokens' lines kept in L2 (32,768 rows of 7,168 bf16 133 -> 102 us,
// 5.2 TB/s; 524,288 rows of 64 bf16, 16 of them a block instead of 4, 131 -> 37).
template <typename T, int BYTES, int X>
__global__ void __launch_bounds__(128) expert_gather_kernel(const RowsArgs a, int pieces) {
  using W = typename Raw<T, BYTES>::type;
  const W* kind = nullptr;
  const int64_t r = (int64_t)blockIdx.x * (128 / X) + threadIdx.y;
  if (r >= a.R) return;
  const int64_t src = checked(a.index[r], a.T * a.k, a.status, SITE_ROWS_GATHER);
  char* d = static_cast<char*>(a.out) + r * a.row_stride * (int64_t)sizeof(T);
  int i = threadIdx.x;
  if (src < 0) {
    for (; i < pieces; i += X) store_raw(d + (int64_t)i * BYTES, W{});
    return;
  }
  const bool gated = a.gates != nullptr;
  const float g = gated ? a.gates[src] : 1.0f;
  const char* s = static_cast<const char*>(a.tokens) + (int64_t)((int)src / a.k) * a.token_stride * (int64_t)sizeof(T);
  for (; i + 7 * X < pieces; i += 8 * X) copy_pieces<T, BYTES, 8, X, true>(s, d, i, pieces, gated, g, kind);
  if (i + 2 * X < pieces) {
    copy_pieces<T, BYTES, 8, X, false>(s, d, i, pieces, gated, g, kind);
  } else if (i < pieces) {
    copy_pieces<T, BYTES, 2, X, false>(s, d, i, pieces, gated, g, kind);
  }
}

// One piece of one token to a thread, the token's k rows in flight at once.
template <typename T, int BYTES, int KMAX>
__global__ void __launch_bounds__(128) expert_merge_kernel(const RowsArgs a, int pieces) {
  using W = typename Raw<T, BYTES>::type;
  const int64_t n = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t t = n / pieces;
  if (t >= a.T) return;
  const int i = (int)(n - t * pieces);
  W v[KMAX];
  float g[KMAX];
  bool has[KMAX];
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    has[j] = false;
    if (j < a.k) {
      const int64_t row = checked(a.index[t * a.k + j], a.R, a.status, SITE_ROWS_MERGE);
      has[j] = row >= 0;
      if (has[j]) {
        g[j] = a.gates != nullptr ? a.gates[t * a.k + j] : 1.0f;
        load_raw(v[j], static_cast<const char*>(a.rows) + row * a.row_stride * (int64_t)sizeof(T) + (int64_t)i * BYTES);
      }
    }
  }
  float acc[Piece<T, BYTES>::N] = {};
#pragma unroll
  for (int j = 0; j < KMAX; ++j)
    if (has[j]) {
      float f[Piece<T, BYTES>::N];
      unpack<T, BYTES>(v[j], f);
#pragma unroll
      for (int q = 0; q < Piece<T, BYTES>::N; ++q) acc[q] = fmaf(g[j], f[q], acc[q]);
    }
  W o;
  pack<T, BYTES>(o, acc);
  store_raw(static_cast<char*>(a.out) + t * a.token_stride * (int64_t)sizeof(T) + (int64_t)i * BYTES, o);
}

// The same for pieces of one element, which instructions bound: a block takes one token, whose rows are found once for all
// of its pieces (4,096 tokens of 8 rows of 7,167: f32 305 -> 201 us, bf16 301 -> 274; two bf16 a piece 158 -> 172, so
// those stay with the other).
template <typename T, int BYTES, int KMAX>
__global__ void __launch_bounds__(128) expert_merge_token_kernel(const RowsArgs a, int pieces) {
  using W = typename Raw<T, BYTES>::type;
  const int64_t t = blockIdx.x;
  const char* row[KMAX];
  float g[KMAX];
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    row[j] = nullptr;
    g[j] = 0.0f;
    if (j < a.k) {
      const int64_t r = checked(a.index[t * a.k + j], a.R, a.status, SITE_ROWS_MERGE);
      if (r >= 0) {
        g[j] = a.gates != nullptr ? a.gates[t * a.k + j] : 1.0f;
        row[j] = static_cast<const char*>(a.rows) + r * a.row_stride * (int64_t)sizeof(T);
      }
    }
  }
  char* out = static_cast<char*>(a.out) + t * a.token_stride * (int64_t)sizeof(T);
  for (int i = threadIdx.x; i < pieces; i += blockDim.x) {
    W v[KMAX];
#pragma unroll
    for (int j = 0; j < KMAX; ++j)
      if (row[j] != nullptr) load_raw(v[j], row[j] + (int64_t)i * BYTES);
    float acc[Piece<T, BYTES>::N] = {};
#pragma unroll
    for (int j = 0; j < KMAX; ++j)
      if (row[j] != nullptr) {
        float f[Piece<T, BYTES>::N];
        unpack<T, BYTES>(v[j], f);
#pragma unroll
        for (int q = 0; q < Piece<T, BYTES>::N; ++q) acc[q] = fmaf(g[j], f[q], acc[q]);
      }
    W o;
    pack<T, BYTES>(o, acc);
    store_raw(out + (int64_t)i * BYTES, o);
  }
}

// One token to a block: dy is read once and meets the token's rows four at a time.  The dot products are added
// over a thread's pieces, the lanes and the warps, in that fixed order.
template <typename T, int BYTES, int KMAX>
__global__ void __launch_bounds__(512) expert_merge_backward_kernel(const RowsArgs a, int pieces) {
  using W = typename Raw<T, BYTES>::type;
  constexpr int N = Piece<T, BYTES>::N, G = KMAX < 4 ? KMAX : 4;
  __shared__ float part[16][KMAX];
  const int64_t t = blockIdx.x;
  int32_t row[KMAX];
  float g[KMAX], dot[KMAX];
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    row[j] = -1;
    dot[j] = 0.0f;
    if (j < a.k) {
      row[j] = (int32_t)checked(a.index[t * a.k + j], a.R, a.status, SITE_ROWS_MERGE);
      g[j] = a.gates != nullptr ? a.gates[t * a.k + j] : 1.0f;
    }
  }
  for (int i = threadIdx.x; i < pieces; i += blockDim.x) {
    const int64_t at = (int64_t)i * BYTES;
    W w;
    load_raw(w, static_cast<const char*>(a.tokens) + t * a.token_stride * (int64_t)sizeof(T) + at);
    float dy[N];
    unpack<T, BYTES>(w, dy);
#pragma unroll
    for (int j0 = 0; j0 < KMAX; j0 += G) {
      W v[G];
#pragma unroll
      for (int j = 0; j < G; ++j)
        if (row[j0 + j] >= 0)
          load_raw(v[j], static_cast<const char*>(a.rows) + row[j0 + j] * a.row_stride * (int64_t)sizeof(T) + at);
#pragma unroll
      for (int j = 0; j < G; ++j)
        if (row[j0 + j] >= 0) {
          float o[N], d[N];
          unpack<T, BYTES>(v[j], o);
#pragma unroll
          for (int q = 0; q < N; ++q) {
            dot[j0 + j] = fmaf(dy[q], o[q], dot[j0 + j]);
            d[q] = g[j0 + j] * dy[q];
          }
          W out;
          pack<T, BYTES>(out, d);
          store_raw(static_cast<char*>(a.out) + row[j0 + j] * a.row_stride * (int64_t)sizeof(T) + at, out);
        }
    }
  }
  if (a.dgates == nullptr) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], s);
    if (lane == 0) part[warp][j] = dot[j];
  }
  __syncthreads();
  if (threadIdx.x < a.k) {
    float sum = 0.0f;
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) sum += part[w][threadIdx.x];
    a.dgates[t * a.k + threadIdx.x] = sum;
  }
}

// The widest piece that the rows' starts, strides and width allow.
int piece_bytes(const RowsArgs& a, int item) {
  uint64_t bits = reinterpret_cast<uintptr_t>(a.tokens) | reinterpret_cast<uintptr_t>(a.rows) |
                  reinterpret_cast<uintptr_t>(a.out) | (uint64_t)(a.H * item) | (uint64_t)(a.token_stride * item) |
                  (uint64_t)(a.row_stride * item);
  return bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : item;
}

template <typename T, int BYTES>
cudaError_t gather(const RowsArgs& a, cudaStream_t st) {
  const int pieces = (int)(a.H * (int64_t)sizeof(T) / BYTES);
  // narrow rows share a block: as many threads as the row has pieces, up to a power of two
  int x = 8;
  while (x < 128 && x < pieces) x *= 2;
  const dim3 block(x, 128 / x);
  const int64_t blocks = (a.R + block.y - 1) / block.y;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  switch (x) {
    case 8: expert_gather_kernel<T, BYTES, 8><<<(unsigned)blocks, block, 0, st>>>(a, pieces); break;
    case 16: expert_gather_kernel<T, BYTES, 16><<<(unsigned)blocks, block, 0, st>>>(a, pieces); break;
    case 32: expert_gather_kernel<T, BYTES, 32><<<(unsigned)blocks, block, 0, st>>>(a, pieces); break;
    case 64: expert_gather_kernel<T, BYTES, 64><<<(unsigned)blocks, block, 0, st>>>(a, pieces); break;
    default: expert_gather_kernel<T, BYTES, 128><<<(unsigned)blocks, block, 0, st>>>(a, pieces); break;
  }
  return cudaGetLastError();
}

template <typename T, int BYTES, int KMAX>
cudaError_t merge_k(const RowsArgs& a, cudaStream_t st) {
  const int pieces = (int)(a.H * (int64_t)sizeof(T) / BYTES);
  // A block a token where rows are long enough and tokens enough to fill the SMs (k = 8, f32: 4,096 tokens of 257 elements 11.8 -> 7.5
  // us, of 65 4.6 -> 5.5; of 1,111 elements 1,024 tokens 12.6 -> 5.6, 128 3.2 -> 4.4; bf16 of 1,111: 1,024 12.8 -> 7.8, 500 7.2 both)
  if (BYTES == (int)sizeof(T) && pieces >= 96 && a.T >= 512) {
    if (a.T > INT32_MAX) return cudaErrorInvalidValue;
    expert_merge_token_kernel<T, BYTES, KMAX><<<(unsigned)a.T, 128, 0, st>>>(a, pieces);
    return cudaGetLastError();
  }
  const int64_t blocks = (a.T * pieces + 127) / 128;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  expert_merge_kernel<T, BYTES, KMAX><<<(unsigned)blocks, 128, 0, st>>>(a, pieces);
  return cudaGetLastError();
}

template <typename T, int BYTES>
cudaError_t merge(const RowsArgs& a, cudaStream_t st) {
  if (a.k <= 1) return merge_k<T, BYTES, 1>(a, st);
  if (a.k <= 2) return merge_k<T, BYTES, 2>(a, st);
  if (a.k <= 4) return merge_k<T, BYTES, 4>(a, st);
  if (a.k <= 8) return merge_k<T, BYTES, 8>(a, st);
  return merge_k<T, BYTES, 16>(a, st);
}

template <typename T, int BYTES, int KMAX>
cudaError_t merge_backward_k(const RowsArgs& a, int n_sm, cudaStream_t st) {
  const int pieces = (int)(a.H * (int64_t)sizeof(T) / BYTES);
  // few tokens: a block of as many threads as shorten the row (k = 8 of 7,168 bf16: 64 tokens 8.8 us with 128 threads, 5.3 with 512;
  // 256 11.0 and 9.9; 400 17.3 and 18.7; 1,024 48 and 53)
  const int most = a.T < 2 * n_sm ? 512 : 128;
  const int threads = std::min(most, (pieces + 31) / 32 * 32);
  if (a.T > INT32_MAX) return cudaErrorInvalidValue;
  expert_merge_backward_kernel<T, BYTES, KMAX><<<(unsigned)a.T, threads, 0, st>>>(a, pieces);
  return cudaGetLastError();
}

template <typename T, int BYTES>
cudaError_t merge_backward(const RowsArgs& a, int n_sm, cudaStream_t st) {
  if (a.k <= 1) return merge_backward_k<T, BYTES, 1>(a, n_sm, st);
  if (a.k <= 2) return merge_backward_k<T, BYTES, 2>(a, n_sm, st);
  if (a.k <= 4) return merge_backward_k<T, BYTES, 4>(a, n_sm, st);
  if (a.k <= 8) return merge_backward_k<T, BYTES, 8>(a, n_sm, st);
  return merge_backward_k<T, BYTES, 16>(a, n_sm, st);
}

}  // namespace

cudaError_t launch_expert_gather(const RowsArgs& a, bool bf16, cudaStream_t st) {
  const int bytes = piece_bytes(a, bf16 ? 2 : 4);
  if (!bf16) return bytes == 16 ? gather<float, 16>(a, st) : gather<float, 4>(a, st);
  if (bytes == 16) return gather<__nv_bfloat16, 16>(a, st);
  return bytes == 4 ? gather<__nv_bfloat16, 4>(a, st) : gather<__nv_bfloat16, 2>(a, st);
}

cudaError_t launch_expert_merge(const RowsArgs& a, bool bf16, cudaStream_t st) {
  const int bytes = piece_bytes(a, bf16 ? 2 : 4);
  if (!bf16) return bytes == 16 ? merge<float, 16>(a, st) : merge<float, 4>(a, st);
  if (bytes == 16) return merge<__nv_bfloat16, 16>(a, st);
  return bytes == 4 ? merge<__nv_bfloat16, 4>(a, st) : merge<__nv_bfloat16, 2>(a, st);
}

cudaError_t launch_expert_merge_backward(const RowsArgs& a, bool bf16, int n_sm, cudaStream_t st) {
  const int bytes = piece_bytes(a, bf16 ? 2 : 4);
  if (!bf16) return bytes == 16 ? merge_backward<float, 16>(a, n_sm, st) : merge_backward<float, 4>(a, n_sm, st);
  if (bytes == 16) return merge_backward<__nv_bfloat16, 16>(a, n_sm, st);
  return bytes == 4 ? merge_backward<__nv_bfloat16, 4>(a, n_sm, st) : merge_backward<__nv_bfloat16, 2>(a, n_sm, st);
}

}  // namespace mok
