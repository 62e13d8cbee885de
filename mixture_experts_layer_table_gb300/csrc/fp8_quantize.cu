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
// A half-warp holds whole rows of 128 columns, lane l columns 8 l .. 8 l + 7, so that a row's maximum is 4 shuffles and
// a store of a row 128 bytes.  Rows alone: 256 threads, 1 or 4 rows a half-warp.  128 x 128 tiles: 512 threads, 4 rows a
// half-warp, a lane's 4 rows of a column one word of the transposed tile.
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "fp8.cuh"
#include "mx.cuh"
#include "status.cuh"

namespace mok {
namespace {

// Two f32 in a register pair, one instruction for both.  The compiler's own pairs: those that inline assembly makes of
// two registers cost it moves (16 x 4096 x 7168 weights 402 -> 317 us).
using F2 = float2;
__device__ __forceinline__ F2 f2(float a, float b) { return make_float2(a, b); }
__device__ __forceinline__ F2 f2(float a) { return make_float2(a, a); }
__device__ __forceinline__ void split(F2 x, float& a, float& b) {
  a = x.x;
  b = x.y;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ F2 mul2(F2 a, F2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) { return __ffma2_rn(a, b, c); }

constexpr int THREADS = 256;       // rows alone
constexpr int TILE_THREADS = 512;  // 128 x 128 tiles: 32 half-warps of 4 rows
constexpr float LEAST = FP8_LEAST;
constexpr float BIG = 3.4028234663852886e38f;

// Off by a unit in the last place at most; 0 for what would be below 2^-126.
__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// What a block's elements are divided by, in the form the quotient is made of: -amax / 512 (exact) and about 512 / amax.
struct Divisor {
  F2 minus_a, inv;
};
__device__ __forceinline__ Divisor divisor(float amax0, float amax1) {
  const float a0 = fmaxf(amax0, LEAST) * (1.0f / 512), a1 = fmaxf(amax1, LEAST) * (1.0f / 512);
  return {f2(-a0, -a1), f2(reciprocal(a0), reciprocal(a1))};
}
__device__ __forceinline__ Divisor divisor(float amax) {
  const float a = fmaxf(amax, LEAST) * (1.0f / 512);
  return {f2(-a), f2(reciprocal(a))};
}
// amax / 448, rounded once: the product with 1 / 448, corrected by its remainder.
__device__ __forceinline__ float block_scale(float amax) {
  const float m = fmaxf(amax, LEAST), q = m * (1.0f / 448);
  return fmaf(fmaf(-q, 448.0f, m), 1.0f / 448, q);
}

// (448 x / 512) / (amax / 512) for two elements: the product with the reciprocal, then one correction by the remainder
// x' - y a, which the FMA forms exactly: the quotient as a division rounds it, or in rare cases its neighbour.  One of few bits
// (a border between two E4M3 values, common with bf16 inputs) comes out as itself, so that ties go to even as they should; without the
// correction twice as many elements of computed values lay on the other side of a border.  A NaN gives NaN.
__device__ __forceinline__ uint16_t quantize2(F2 x, F2 minus_a, F2 inv) {
  x = mul2(x, f2(0.875f));
  const F2 y = mul2(x, inv);
  float y0, y1;
  split(fma2(fma2(y, minus_a, x), inv, y), y0, y1);
  return e4m3x2_from_f32(y0, y1);
}

// Eight columns of a row.
struct Row8 {
  F2 v[4];
};
__device__ __forceinline__ uint2 quantize8(const Row8& x, const Divisor& d) {
  uint2 o;
  o.x = quantize2(x.v[0], d.minus_a, d.inv) | (uint32_t)quantize2(x.v[1], d.minus_a, d.inv) << 16;
  o.y = quantize2(x.v[2], d.minus_a, d.inv) | (uint32_t)quantize2(x.v[3], d.minus_a, d.inv) << 16;
  return o;
}

// Infinities become NaN: the conversion keeps a NaN but takes an infinity for 448, and a NaN stays out of maxima.
__device__ __forceinline__ void infinities_to_nan(Row8& x) {
#pragma unroll
  for (int j = 0; j < 4; ++j) x.v[j] = fma2(x.v[j], f2(0.0f), x.v[j]);
}
__device__ __forceinline__ float largest8(const Row8& x) {  // infinities count, NaN do not
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float a, b;
    split(x.v[j], a, b);
    m = fmaxf(fmaxf(m, fabsf(a)), fabsf(b));
  }
  return m;
}
__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ Row8 zero8() { return {{f2(0.0f), f2(0.0f), f2(0.0f), f2(0.0f)}}; }

// Columns c .. c + 7 of a row of `width` elements; zeros behind its end.  VEC: the row is 16-byte aligned and
// width a multiple of 8.
template <bool VEC>
__device__ __forceinline__ Row8 load8(const float* row, int64_t c, int64_t width) {
  Row8 x = zero8();
  if (VEC) {
    if (c < width) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(row + c)), b = __ldg(reinterpret_cast<const float4*>(row + c) + 1);
      x = {{f2(a.x, a.y), f2(a.z, a.w), f2(b.x, b.y), f2(b.z, b.w)}};
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      x.v[j] = f2(c + 2 * j < width ? __ldg(row + c + 2 * j) : 0.0f, c + 2 * j + 1 < width ? __ldg(row + c + 2 * j + 1) : 0.0f);
  }
  return x;
}
template <bool VEC>
__device__ __forceinline__ Row8 load8(const __nv_bfloat16* row, int64_t c, int64_t width) {
  Row8 x;
  if (VEC) {
    uint4 w = make_uint4(0, 0, 0, 0);
    if (c < width) w = __ldg(reinterpret_cast<const uint4*>(row + c));
    const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) x.v[j] = f2(__uint_as_float(words[j] << 16), __uint_as_float(words[j] & 0xffff0000u));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      x.v[j] = f2(c + 2 * j < width ? __bfloat162float(row[c + 2 * j]) : 0.0f,
                  c + 2 * j + 1 < width ? __bfloat162float(row[c + 2 * j + 1]) : 0.0f);
  }
  return x;
}

// 1 / (1 + e^-h), two at a time: the accurate exponential, and a reciprocal corrected once.  With the hardware's 2^x and
// 1 / x alone (2^-21) a value on the other side of a border between two E4M3 values was ten times as frequent.  From h = FAR
// down the value stays at e^FAR: far8 brings the rest.
constexpr float FAR = -40.0f;
__device__ __forceinline__ F2 sigmoid2(F2 h) {
  float a, b;
  split(h, a, b);
  const F2 d = add2(f2(expf(-fmaxf(a, FAR)), expf(-fmaxf(b, FAR))), f2(1.0f));
  split(d, a, b);
  const F2 r = f2(reciprocal(a), reciprocal(b));
  return fma2(fma2(mul2(d, f2(-1.0f)), r, f2(1.0f)), r, r);
}

// Below FAR the sigmoid is e^h = e^FAR e^(h - FAR), soon out of f32's range, while h and what it is multiplied with may be as
// large as the type allows (a mask's lowest value).  So the second part (h - FAR is exact) goes to that other factor, x (a NaN
// for an infinite h), and h itself stops where nothing is left of any product: these then come out to f32's precision, or as 0.
__device__ __forceinline__ void far2(F2& h, F2& x) {
  x = mul2(x, f2(fmaf(h.x, 0.0f, expf(fminf(h.x - FAR, 0.0f))), fmaf(h.y, 0.0f, expf(fminf(h.y - FAR, 0.0f)))));
  h = f2(fmaxf(h.x, -1e4f), fmaxf(h.y, -1e4f));
}
__device__ __forceinline__ void far8(Row8& h, Row8& x) {
  float least = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) least = fminf(fminf(least, h.v[j].x), h.v[j].y);
  if (least < FAR) {
#pragma unroll
    for (int j = 0; j < 4; ++j) far2(h.v[j], x.v[j]);
  }
}
// silu(h) = h s, and its slope s (1 + h (1 - s)); the last product with another factor is the only one that can leave f32's
// range, and only where the result does.
__device__ __forceinline__ F2 silu2(F2 h, F2 s) { return mul2(h, s); }
__device__ __forceinline__ F2 slope2(F2 h, F2 s) { return mul2(s, add2(mul2(h, fma2(s, f2(-1.0f), f2(1.0f))), f2(1.0f))); }

// Where a row of the source lies.
template <typename T>
struct Source {
  const T* x;     // null: a row of zeros
  const T* grad;
  float gate;
};
template <int SRC, typename T>
__device__ __forceinline__ Source<T> source_row(const Fp8QuantizeArgs& a, int64_t r) {
  const T* x = static_cast<const T*>(a.x);
  if (SRC != FP8_PLAIN)
    return {x + r * a.x_stride, SRC == FP8_SWIGLU_GRAD ? static_cast<const T*>(a.grad) + r * a.grad_stride : nullptr, 1.0f};
  if (a.src_of == nullptr) return {x + r * a.x_stride, nullptr, 1.0f};
  const int32_t s = __ldg(a.src_of + r);
  if (s < 0 || s >= a.T * a.k) {
    if (s != -1) report_status(a.status, MOK_DEV_INVALID_ROUTING, SITE_FP8_SOURCE);
    return {nullptr, nullptr, 1.0f};
  }
  return {x + (int64_t)(s / a.k) * a.x_stride, nullptr, a.gates != nullptr ? __ldg(a.gates + s) : 1.0f};
}

// Columns c .. c + 7 of the quantised row that comes of it.
template <int SRC, typename T, bool VEC>
__device__ __forceinline__ Row8 source8(const Fp8QuantizeArgs& a, const Source<T>& s, int64_t c) {
  Row8 o = zero8();
  if (SRC == FP8_PLAIN) {
    if (s.x == nullptr) return o;
    o = load8<VEC>(s.x, c, a.C);
    if (a.gates != nullptr) {
      const F2 g = f2(s.gate);
#pragma unroll
      for (int j = 0; j < 4; ++j) o.v[j] = mul2(o.v[j], g);
    }
  } else if (SRC == FP8_SWIGLU) {
    Row8 h = load8<VEC>(s.x, c, a.C), u = load8<VEC>(s.x + a.C, c, a.C);
    far8(h, u);
#pragma unroll
    for (int j = 0; j < 4; ++j) o.v[j] = mul2(silu2(h.v[j], sigmoid2(h.v[j])), u.v[j]);
  } else {
    const int64_t I = a.C / 2;
    // VEC: I is a multiple of 8, so that a lane's columns lie in one half
    if (VEC) {
      if (c >= I) {
        Row8 h = load8<true>(s.x, c - I, I), d = load8<true>(s.grad, c - I, I);
        far8(h, d);
#pragma unroll
        for (int j = 0; j < 4; ++j) o.v[j] = mul2(silu2(h.v[j], sigmoid2(h.v[j])), d.v[j]);
      } else {
        Row8 h = load8<true>(s.x, c, I), d = load8<true>(s.grad, c, I);
        const Row8 u = load8<true>(s.x + I, c, I);
        far8(h, d);
#pragma unroll
        for (int j = 0; j < 4; ++j) o.v[j] = mul2(mul2(slope2(h.v[j], sigmoid2(h.v[j])), u.v[j]), d.v[j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float h[2], d[2], u[2];
        bool up[2];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const int64_t col = c + 2 * j + z;
          const bool in = col < a.C;
          up[z] = col >= I;
          const int64_t i = up[z] ? col - I : col;
          h[z] = in ? widen(s.x[i]) : 0.0f;
          d[z] = in ? widen(s.grad[i]) : 0.0f;
          u[z] = in && !up[z] ? widen(s.x[I + i]) : 0.0f;
        }
        F2 hh = f2(h[0], h[1]), dd = f2(d[0], d[1]);
        if (fminf(h[0], h[1]) < FAR) far2(hh, dd);
        const F2 sg = sigmoid2(hh);
        const F2 du = mul2(silu2(hh, sg), dd), dh = mul2(mul2(slope2(hh, sg), f2(u[0], u[1])), dd);
        o.v[j] = f2(up[0] ? du.x : dh.x, up[1] ? du.y : dh.y);
      }
    }
  }
  return o;
}

// dh and du of columns i .. i + 7 of h | u: one exponential for both.  (16-byte aligned rows.)
template <typename T>
__device__ __forceinline__ void swiglu_grad8(const Fp8QuantizeArgs& a, const Source<T>& s, int64_t i, Row8& dh, Row8& du) {
  const int64_t I = a.C / 2;
  Row8 h = load8<true>(s.x, i, I), d = load8<true>(s.grad, i, I);
  const Row8 u = load8<true>(s.x + I, i, I);
  far8(h, d);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const F2 sg = sigmoid2(h.v[j]);
    du.v[j] = mul2(silu2(h.v[j], sg), d.v[j]);
    dh.v[j] = mul2(mul2(slope2(h.v[j], sg), u.v[j]), d.v[j]);
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

// The transposed tile in shared memory, 128 columns of 128 bytes: the 4-byte word of half-warp k lies at word k ^ 2 (c / 8 mod
// 16) of column c, so that the writes of a warp (16 lanes with columns 8 apart, two words) do not meet in a bank; the
// words of two neighbouring half-warps stay together, 8 bytes for the way out.
__device__ __forceinline__ int tile_word(int c, int k) { return c * 32 + (k ^ (2 * ((c >> 3) & 15))); }

// Byte j of each of four rows.
__device__ __forceinline__ uint32_t column_word(const uint2 (&rows)[4], int j) {
  const uint32_t sel = (j & 3) | ((j & 3) + 4) << 4;
  const uint32_t lo = j < 4 ? __byte_perm(rows[0].x, rows[1].x, sel) : __byte_perm(rows[0].y, rows[1].y, sel);
  const uint32_t hi = j < 4 ? __byte_perm(rows[2].x, rows[3].x, sel) : __byte_perm(rows[2].y, rows[3].y, sel);
  return __byte_perm(lo, hi, 0x5410);
}

// Writes the tile's 128 columns to qt rows (128 bytes each, `n` of them in front of the end), of which `cols` exist.
__device__ __forceinline__ void store_tile(const uint32_t* tile, uint8_t* qt, int64_t stride, int64_t cols, int64_t n) {
  const int k = threadIdx.x & 15, c0 = threadIdx.x >> 4;
  uint8_t* to = qt + c0 * stride + 8 * k;
  if (cols >= 128 && n >= 128) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
      *reinterpret_cast<uint2*>(to + s * (32 * stride)) = *reinterpret_cast<const uint2*>(tile + tile_word(c0 + 32 * s, 2 * k));
  } else {
#pragma unroll
    for (int s = 0; s < 4; ++s)
      if (c0 + 32 * s < cols)
        store8(to + s * (32 * stride), *reinterpret_cast<const uint2*>(tile + tile_word(c0 + 32 * s, 2 * k)), n - 8 * k);
  }
}

// The largest finite magnitude of each of a half-warp's rows (of the warp's lanes, infinities have become NaN).
__device__ __forceinline__ void row_maxima(const Row8 (&v)[1], float (&m)[1]) {
  m[0] = largest8(v[0]);
#pragma unroll
  for (int s = 8; s > 0; s >>= 1) m[0] = fmaxf(m[0], __shfl_xor_sync(0xffffffffu, m[0], s));
}
// Of four rows: each exchange halves the rows that a lane reduces (9 shuffles, not 16).
__device__ __forceinline__ void row_maxima(const Row8 (&v)[4], float (&m)[4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = largest8(v[i]);
  const bool hi = lane & 8, odd = lane & 4;
  const float x = fmaxf(hi ? m[2] : m[0], __shfl_xor_sync(0xffffffffu, hi ? m[0] : m[2], 8));
  const float y = fmaxf(hi ? m[3] : m[1], __shfl_xor_sync(0xffffffffu, hi ? m[1] : m[3], 8));
  float z = fmaxf(odd ? y : x, __shfl_xor_sync(0xffffffffu, odd ? x : y, 4));
  z = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, 2));
  z = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, 1));
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = __shfl_sync(0xffffffffu, z, (lane & 16) | 4 * i);
}
template <int RPT>
__device__ __forceinline__ void finite_or_nan(Row8 (&v)[RPT]) {
  float all = 0.0f;
#pragma unroll
  for (int i = 0; i < RPT; ++i) all = fmaxf(all, largest8(v[i]));
  if (__any_sync(0xffffffffu, all > BIG)) {
#pragma unroll
    for (int i = 0; i < RPT; ++i) infinities_to_nan(v[i]);
  }
}

// A row's eight columns as they are kept until the scales are known: bf16 rows in their own four words (half the
// registers, so that three blocks share an SM, and maxima of two elements at once).
struct RawRow8 {
  uint32_t w[4];
};
template <typename T, bool VEC>
struct Kept {
  using type = Row8;
};
template <>
struct Kept<__nv_bfloat16, true> {
  using type = RawRow8;
};
template <bool VEC, typename T>
__device__ __forceinline__ void keep(Row8& x, const T* row, int64_t c, int64_t width) { x = load8<VEC>(row, c, width); }
template <bool VEC>
__device__ __forceinline__ void keep(RawRow8& x, const __nv_bfloat16* row, int64_t c, int64_t width) {
  uint4 w = make_uint4(0, 0, 0, 0);
  if (c < width) w = __ldg(reinterpret_cast<const uint4*>(row + c));
  x = {{w.x, w.y, w.z, w.w}};
}
__device__ __forceinline__ Row8 kept(const Row8& x) { return x; }
__device__ __forceinline__ Row8 kept(const RawRow8& x) {
  Row8 o;
#pragma unroll
  for (int j = 0; j < 4; ++j) o.v[j] = f2(__uint_as_float(x.w[j] << 16), __uint_as_float(x.w[j] & 0xffff0000u));
  return o;
}
__device__ __forceinline__ F2 kept_pair(const Row8& x, int j) { return x.v[j]; }
__device__ __forceinline__ F2 kept_pair(const RawRow8& x, int j) {
  return f2(__uint_as_float(x.w[j] << 16), __uint_as_float(x.w[j] & 0xffff0000u));
}
__device__ __forceinline__ float kept_largest(const Row8 (&v)[4]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = fmaxf(m, largest8(v[i]));
  return m;
}
__device__ __forceinline__ float kept_largest(const RawRow8 (&v)[4]) {
  // magnitudes as unsigned 16-bit numbers order like the values, NaN above infinity: they are looked at again then
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) m = __vmaxu2(m, v[i].w[j] & 0x7fff7fffu);
  return __uint_as_float(max(m & 0xffffu, m >> 16) << 16);
}

// Infinities become NaN.  Returns whether an element of the warp's rows is not finite: its magnitude is then left out below.
template <int RPT>
__device__ __forceinline__ bool only_finite_or_nan(Row8 (&v)[RPT]) {
  finite_or_nan(v);
  return false;  // maxima leave NaN out by themselves
}
template <int RPT>
__device__ __forceinline__ bool only_finite_or_nan(RawRow8 (&v)[RPT]) {
  const bool odd = __any_sync(0xffffffffu, !(kept_largest(v) <= BIG));
  if (odd) {
#pragma unroll
    for (int i = 0; i < RPT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i].w[j] |= __vcmpgeu2(v[i].w[j] & 0x7fff7fffu, 0x7f807f80u) & 0x7fff7fffu;
  }
  return odd;
}
template <bool ODD>
__device__ __forceinline__ uint32_t magnitudes(uint32_t w) {
  w &= 0x7fff7fffu;
  return ODD ? w & __vcmpltu2(w, 0x7f807f80u) : w;
}
// The largest magnitudes of columns 2 j and 2 j + 1 of the warp's rows.
template <bool ODD>
__device__ __forceinline__ float2 two_columns(const Row8 (&v)[4], int j) {
  float2 t = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < 4; ++i) t = make_float2(fmaxf(t.x, fabsf(v[i].v[j].x)), fmaxf(t.y, fabsf(v[i].v[j].y)));
  return make_float2(fmaxf(t.x, __shfl_xor_sync(0xffffffffu, t.x, 16)), fmaxf(t.y, __shfl_xor_sync(0xffffffffu, t.y, 16)));
}
template <bool ODD>
__device__ __forceinline__ float2 two_columns(const RawRow8 (&v)[4], int j) {
  uint32_t t = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) t = __vmaxu2(t, magnitudes<ODD>(v[i].w[j]));
  t = __vmaxu2(t, __shfl_xor_sync(0xffffffffu, t, 16));
  return make_float2(__uint_as_float(t << 16), __uint_as_float(t & 0xffff0000u));
}
template <bool ODD, int RPT>
__device__ __forceinline__ void kept_row_maxima(const Row8 (&v)[RPT], float (&m)[RPT]) { row_maxima(v, m); }
// Two rows' maxima in a word: 5 shuffles for four rows.
template <bool ODD>
__device__ __forceinline__ void kept_row_maxima(const RawRow8 (&v)[4], float (&m)[4]) {
  uint32_t t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    t[i] = magnitudes<ODD>(v[i].w[0]);
#pragma unroll
    for (int j = 1; j < 4; ++j) t[i] = __vmaxu2(t[i], magnitudes<ODD>(v[i].w[j]));
  }
  const uint32_t x = __vmaxu2(__byte_perm(t[0], t[1], 0x5410), __byte_perm(t[0], t[1], 0x7632));
  const uint32_t y = __vmaxu2(__byte_perm(t[2], t[3], 0x5410), __byte_perm(t[2], t[3], 0x7632));
  const bool hi = threadIdx.x & 8;
  uint32_t z = __vmaxu2(hi ? y : x, __shfl_xor_sync(0xffffffffu, hi ? x : y, 8));
#pragma unroll
  for (int s = 4; s > 0; s >>= 1) z = __vmaxu2(z, __shfl_xor_sync(0xffffffffu, z, s));
  const uint32_t o = __shfl_xor_sync(0xffffffffu, z, 8), first = hi ? o : z, second = hi ? z : o;
  m[0] = __uint_as_float(first << 16), m[1] = __uint_as_float(first & 0xffff0000u);
  m[2] = __uint_as_float(second << 16), m[3] = __uint_as_float(second & 0xffff0000u);
}

// ------------------------------------------------------------------ rows
// Tiles of 16 RPT rows along the rows only.  RAW: bf16 rows as they are, as below (16,384 x 7,168
// gathered 106 -> 80 us).
template <int SRC, typename T, bool VEC, int RPT, bool RAW>
__global__ void __launch_bounds__(THREADS) fp8_rows_kernel(const Fp8QuantizeArgs a, int col_blocks) {
  __shared__ float s_scale[16 * RPT];
  const int b = blockIdx.x % col_blocks;
  const int64_t r0 = (int64_t)(blockIdx.x / col_blocks) * (16 * RPT);
  const int w = threadIdx.x >> 4, l = threadIdx.x & 15;
  const int64_t c = (int64_t)b * FP8_BLOCK + 8 * l;
  typename std::conditional<RAW, RawRow8, Row8>::type v[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int64_t r = r0 + w * RPT + i;
    if constexpr (RAW) {
      const T* x = r < a.R ? source_row<SRC, T>(a, r).x : nullptr;
      keep<VEC>(v[i], x, c, x == nullptr ? 0 : a.C);
    } else {
      v[i] = r < a.R ? source8<SRC, T, VEC>(a, source_row<SRC, T>(a, r), c) : zero8();
    }
  }
  float m[RPT];
  if (only_finite_or_nan(v)) kept_row_maxima<true>(v, m);
  else kept_row_maxima<false>(v, m);
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int64_t r = r0 + w * RPT + i;
    const uint2 bytes = quantize8(kept(v[i]), divisor(m[i]));
    if (r < a.R && c < a.C) store8(a.q + r * a.q_stride + c, bytes, a.C - c);
    if (l == 0) s_scale[w * RPT + i] = block_scale(m[i]);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * RPT; i += THREADS)
    if (r0 + i < a.R) a.scale[b * a.scale_stride + r0 + i] = s_scale[i];
}

// ------------------------------------------------------------------ rows and columns
// A tile is 128 rows of one expert (of the padded order) x 128 columns.  A block takes `group` column blocks of
// one row tile, after it has found the tile's expert: the offsets are read and scanned by the block itself.
// PAIRED (the SwiGLU's gradient where I is a multiple of 128): a round takes column block b of dh and of du, which come of the
// same h, u and da; du waits in shared memory, each thread's in its own place (169 -> 133 us for 16,384 x 4,096; far8's question after a row's loads has
// since cost 2%).
// RAW (bf16 rows in hand or gathered, without gates): the rows are kept as they are, and three blocks share an SM (16,384 x 7,168
// in both layouts 223 -> 168 us, gathered 225 -> 195; the gates take products in 32 bits, which words of 16 cannot hold).
template <int SRC, typename T, bool VEC, bool PAIRED, bool RAW>
__global__ void __launch_bounds__(TILE_THREADS, RAW ? 3 : 2) fp8_columns_kernel(const Fp8QuantizeArgs a, int col_blocks, int group,
                                                                      int groups) {
  __shared__ __align__(16) uint32_t tile[128 * 32];
  __shared__ __align__(16) int s_max[2][128];  // bits of the columns' maxima, of this turn and the next
  __shared__ float s_scale[2][128];
  __shared__ int s_warp[16], s_where[2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int p = blockIdx.x / groups;  // row tile
  // the expert whose 128-row blocks hold block p: a scan of the experts' blocks, 512 experts at a time
  if (threadIdx.x == 0) s_where[1] = 0;
  int before = 0;  // blocks of the experts before this turn's
  for (int e0 = 0; e0 < a.E; e0 += TILE_THREADS) {
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
    for (int i = 0; i < 16; ++i) {
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
  uint8_t* to = a.q + (row0 + w * 4) * a.q_stride;
  const int b_end = min(col_blocks, (int)(blockIdx.x % groups + 1) * group);
  if (threadIdx.x < 128) s_max[0][threadIdx.x] = s_max[1][threadIdx.x] = 0;
  __syncthreads();
  extern __shared__ __align__(16) float4 waiting[];  // PAIRED: du
  const int first = (blockIdx.x % groups) * group * (PAIRED ? 2 : 1), last = b_end * (PAIRED ? 2 : 1);
  for (int at = first, turn = 0; at < last; ++at, turn ^= 1) {
    const int b = PAIRED ? (at >> 1) + (at & 1) * col_blocks : at;  // dh, then du
    const int64_t c = (int64_t)b * FP8_BLOCK + 8 * l;
    const bool full = rows == 128 && (b + 1) * (int64_t)FP8_BLOCK <= a.C;  // uniform, and most tiles
    typename std::conditional<RAW, RawRow8, Row8>::type v[4];
    if constexpr (RAW) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const T* x = full || w * 4 + i < rows ? source_row<SRC, T>(a, row0 + w * 4 + i).x : nullptr;
        keep<VEC>(v[i], x, c, x == nullptr ? 0 : a.C);
      }
    } else if (PAIRED && (at & 1)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 x = waiting[(2 * i) * TILE_THREADS + threadIdx.x], y = waiting[(2 * i + 1) * TILE_THREADS + threadIdx.x];
        v[i] = {{f2(x.x, x.y), f2(x.z, x.w), f2(y.x, y.y), f2(y.z, y.w)}};
      }
    } else if (PAIRED) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        Row8 du = zero8();
        v[i] = zero8();
        if (full || w * 4 + i < rows) swiglu_grad8<T>(a, source_row<SRC, T>(a, row0 + w * 4 + i), c, v[i], du);
        waiting[(2 * i) * TILE_THREADS + threadIdx.x] = make_float4(du.v[0].x, du.v[0].y, du.v[1].x, du.v[1].y);
        waiting[(2 * i + 1) * TILE_THREADS + threadIdx.x] = make_float4(du.v[2].x, du.v[2].y, du.v[3].x, du.v[3].y);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = full || w * 4 + i < rows ? source8<SRC, T, VEC>(a, source_row<SRC, T>(a, row0 + w * 4 + i), c) : zero8();
    }
    const bool odd = only_finite_or_nan(v);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 t = odd ? two_columns<true>(v, j) : two_columns<false>(v, j);
      // both half-warps hold the maxima: each brings one (as integers, which order like the values they are bits of)
      atomicMax(&s_max[turn][8 * l + 2 * j + (lane >> 4)], __float_as_int(lane < 16 ? t.x : t.y));
    }
    if (a.q != nullptr) {
      float m[4];
      if (odd) kept_row_maxima<true>(v, m);
      else kept_row_maxima<false>(v, m);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint2 bytes = quantize8(kept(v[i]), divisor(m[i]));
        if (full) *reinterpret_cast<uint2*>(to + i * a.q_stride + c) = bytes;
        else if (w * 4 + i < rows && c < a.C) store8(to + i * a.q_stride + c, bytes, a.C - c);
        if (l == 0) s_scale[turn][w * 4 + i] = block_scale(m[i]);
      }
    }
    __syncthreads();
    if (threadIdx.x < 128) {
      const int64_t col = (int64_t)b * FP8_BLOCK + threadIdx.x;
      if (col < a.C) a.qt_scale[p * a.C + col] = block_scale(__int_as_float(s_max[turn][threadIdx.x]));
    } else if (a.q != nullptr && (int)threadIdx.x - 128 < rows) {
      a.scale[b * a.scale_stride + row0 + threadIdx.x - 128] = s_scale[turn][threadIdx.x - 128];
    }
    uint2 bytes[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int4 t = *reinterpret_cast<const int4*>(&s_max[turn][8 * l + 4 * h]);
      const float m[4] = {__int_as_float(t.x), __int_as_float(t.y), __int_as_float(t.z), __int_as_float(t.w)};
      uint32_t q[4][2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {  // two columns at a time: their divisors in a pair
        const Divisor d = divisor(m[2 * j], m[2 * j + 1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i][j] = quantize2(kept_pair(v[i], 2 * h + j), d.minus_a, d.inv);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) (h == 0 ? bytes[i].x : bytes[i].y) = q[i][0] | q[i][1] << 16;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) tile[tile_word(8 * l + j, w)] = column_word(bytes, j);
    // the other turn's maxima have been read: every thread is past the barrier above
    if (threadIdx.x >= 256 && threadIdx.x < 384) s_max[turn ^ 1][threadIdx.x - 256] = 0;
    __syncthreads();
    store_tile(tile, a.qt + (int64_t)b * FP8_BLOCK * a.qt_stride + (int64_t)p * 128, a.qt_stride,
               a.C - (int64_t)b * FP8_BLOCK, 128);
    // the next round writes the tile after its first barrier, which every thread reaches after this
  }
}

// ------------------------------------------------------------------ weights
template <typename T, bool VEC>
__global__ void __launch_bounds__(TILE_THREADS, VEC && sizeof(T) == 2 ? 3 : 2) fp8_weights_kernel(const Fp8WeightsArgs a, int n_blocks, int k_blocks) {
  __shared__ __align__(16) uint32_t tile[128 * 32];
  __shared__ float s_max[16];
  const int row_block = (int)blockIdx.x / k_blocks, kb = (int)blockIdx.x - row_block * k_blocks;
  const int64_t e = row_block / n_blocks;
  const int nb = row_block % n_blocks;
  const int w = threadIdx.x >> 4, l = threadIdx.x & 15;
  const int64_t n0 = (int64_t)nb * FP8_BLOCK, k0 = (int64_t)kb * FP8_BLOCK, c = k0 + 8 * l;
  const bool full = n0 + FP8_BLOCK <= a.N && k0 + FP8_BLOCK <= a.K;  // uniform, and most tiles
  const T* from = static_cast<const T*>(a.w) + (e * a.N + n0 + w * 4) * a.K;
  uint8_t* to = a.q + (e * a.N + n0 + w * 4) * a.q_stride;
  typename Kept<T, VEC>::type v[4] = {};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (full || n0 + w * 4 + i < a.N) keep<VEC>(v[i], from + i * a.K, c, full ? c + 8 : a.K);
  float m = kept_largest(v);
  bool odd = false;  // not all elements of the warp are finite
  if (__any_sync(0xffffffffu, !(m <= BIG))) {
    odd = true;
    m = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      Row8 x = kept(v[i]);
      infinities_to_nan(x);
      m = fmaxf(m, largest8(x));
    }
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 16; ++i) m = fmaxf(m, s_max[i]);
  const Divisor d = divisor(m);
  uint2 bytes[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t n = n0 + w * 4 + i;
    Row8 x = kept(v[i]);
    if (odd) infinities_to_nan(x);
    bytes[i] = quantize8(x, d);
    if (a.q != nullptr) {
      if (full) *reinterpret_cast<uint2*>(to + i * a.q_stride + c) = bytes[i];
      else if (n < a.N && c < a.K) store8(to + i * a.q_stride + c, bytes[i], a.K - c);
    }
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
    // 64-row tiles once they give every SM two blocks, else 16-row ones (256 x 2,048 bf16 rows 2.0 us in 16-row tiles, 2.5 in 64-row
    // ones; 1,024 2.9 both; 2,048 4.3 and 4.0; the SwiGLU's 3.9 and 4.4, 6.2 and 6.6, 4,096 10.7 and 10.3)
    const bool wide = col_blocks * ((a.R + 63) / 64) >= 2 * n_sm;
    const int64_t blocks = col_blocks * (wide ? (a.R + 63) / 64 : (a.R + 15) / 16);
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    if constexpr (SRC == FP8_PLAIN && VEC && sizeof(T) == 2) {
      if (wide && a.gates == nullptr) {
        fp8_rows_kernel<SRC, T, true, 4, true><<<(unsigned)blocks, THREADS, 0, st>>>(a, (int)col_blocks);
        return cudaGetLastError();
      }
    }
    if (wide) fp8_rows_kernel<SRC, T, VEC, 4, false><<<(unsigned)blocks, THREADS, 0, st>>>(a, (int)col_blocks);
    else fp8_rows_kernel<SRC, T, VEC, 1, false><<<(unsigned)blocks, THREADS, 0, st>>>(a, (int)col_blocks);
    return cudaGetLastError();
  }
  const int64_t tiles = a.R / 128 + a.E;
  const bool paired = SRC == FP8_SWIGLU_GRAD && VEC && a.C % 256 == 0;
  const int64_t rounds = paired ? col_blocks / 2 : col_blocks;
  // rounds of a block: up to 8 while there remain 4 blocks for each SM (512 rows of 512 bf16 1 round a block 5.0 us, 4 12.9;
  // 16,384 of 7,168 1 round 134, 4 113, 8 112, 16 132)
  int group = 8;
  while (group > 1 && tiles * ((rounds + group - 1) / group) < 4 * n_sm) group /= 2;
  const int64_t groups = (rounds + group - 1) / group;
  if (tiles * groups > INT32_MAX) return cudaErrorInvalidValue;
  const unsigned blocks = (unsigned)(tiles * groups);
  if constexpr (SRC == FP8_SWIGLU_GRAD && VEC) {
    if (paired) {
      constexpr int bytes = 8 * TILE_THREADS * (int)sizeof(float4);
      auto kern = fp8_columns_kernel<SRC, T, true, true, false>;
      const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
      if (err != cudaSuccess) return err;
      kern<<<blocks, TILE_THREADS, bytes, st>>>(a, (int)rounds, group, (int)groups);
      return cudaGetLastError();
    }
  }
  if constexpr (SRC == FP8_PLAIN && VEC && sizeof(T) == 2) {
    if (a.gates == nullptr) {
      fp8_columns_kernel<SRC, T, true, false, true><<<blocks, TILE_THREADS, 0, st>>>(a, (int)rounds, group, (int)groups);
      return cudaGetLastError();
    }
  }
  fp8_columns_kernel<SRC, T, VEC, false, false><<<blocks, TILE_THREADS, 0, st>>>(a, (int)rounds, group, (int)groups);
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
  if (vec) fp8_weights_kernel<T, true><<<(unsigned)blocks, TILE_THREADS, 0, st>>>(a, (int)n, (int)k);
  else fp8_weights_kernel<T, false><<<(unsigned)blocks, TILE_THREADS, 0, st>>>(a, (int)n, (int)k);
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
