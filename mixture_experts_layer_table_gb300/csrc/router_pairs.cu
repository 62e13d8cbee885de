// Group-limited expert selection for many tokens: two tokens to a warp, 16 lanes to each (or one, where 16 lanes of 16
// experts do not hold the groups: more than 256 experts, groups of 17 that take two lanes each, ...).
//
// With a warp to a token (router.cu) most of the instructions steer lanes: about 1,150 a token at 256 experts, k
// rounds of "the best left" among them.  Here a warp's steps serve two tokens, and each token is selected in a few
// steps (about 400 instructions):
//   1. a group lies on a power of two of lanes, C experts to a lane, the last ones fewer; a lane finds the two largest
//      of its rank values; lanes of a segment, a group or an equal part of one, merge theirs;
//   2. each group's lanes count the groups that are better;
//   3. the least of the chosen segments' second largest values has at least 2 * topk_group * (segments of a group)
//      >= k experts at or above it: a bound from below of the k-th largest value.  The experts that reach it (about
//      11 of 128) are listed in shared memory;
//   4. a lane to each listed expert counts how many are better: its place;
//   5. the gates of the tokens of a few such steps are formed together, a lane to each selected expert.
// A token for which this does not do (more than 64 experts listed, too few unmasked) is selected by the whole warp, one
// expert at a time, by the definition.
//
// The next tokens' logits come to shared memory under the arithmetic of these (cp.async; without, the 37 us below are 39).
//
// A biased sigmoid is ranked on approximate values, and what those leave open is settled exactly where it arises: on
// the listed experts if it is an order among them, from the groups on if it is a group (in the whole warp's way, as
// at first, the code of 10 such tokens in 65,536, cold, was 10 us of a call's 38: a single warp's at the end).
//
// 65,536 tokens of 256 experts (f32, sigmoid with a bias, 8 groups): 37 us, 1.9 TB/s; the row is read once, and the
// bound is instructions (25 million of warps, issued in 64% of the cycles at 24 warps an SM, which wait on one
// another's results: shared memory and shuffles between the steps; the SMs' ends lie 15% apart).  4,096 tokens 6 us,
// with the balance outputs 9.4.  With the scores written, and so formed exactly (as the layer asks for them): 65,536 tokens
// 50 us, 4,096 tokens 7.8.
#include <algorithm>
#include <cfloat>
#include <cstddef>

#include "router_common.cuh"

namespace mok {

namespace {

constexpr int WARPS = 8;
constexpr int THREADS = 32 * WARPS;
constexpr int MAX_EXPERTS = 512;  // 32 lanes of at most 16

// How rank values are formed.  LOGITS: softmax without a bias, ranked by the logits.  FAST: a biased sigmoid by the
// hardware's exponential and reciprocal, 4 instructions instead of about 18, with a check that the order is certain.
enum PairMode { LOGITS = 0, SIGMOID = 1, SIGMOID_FAST = 2 };

// The logits' mode does with 64 registers (12,345 tokens of 160 experts: 4 blocks 11.3 us, 3 12.1), the others with 80
// (65,536 tokens of 256 experts: 3 blocks 37 us, 4 41; more and smaller blocks 38.5 to 41; a grid of twice as many,
// for SMs that are done first, 40).
constexpr int blocks_of_sm(PairMode mode) { return mode == LOGITS ? 4 : 3; }

// One token by the definition, by the whole warp: lane j < k returns the j-th best expert, its score in *score.
// `row` [E] is overwritten with the rank values; lane l holds those of the experts l, l + 32, ... (HELD of them).
template <typename TL, int HELD>
__device__ __noinline__ int select_by_warp(const RouteArgs& a, int64_t t, float* row, int lane, float* score) {
  const TL* from = static_cast<const TL*>(a.logits) + t * a.stride;
  const bool softmax = a.router == 0;  // without a bias: ranked by its logits
  float x[HELD], m = -INFINITY, inv = 1.0f;
#pragma unroll
  for (int i = 0; i < HELD; ++i) {
    const int e = lane + 32 * i;
    x[i] = e < a.E ? to_f32(from[e]) : -INFINITY;
    m = fmaxf(m, x[i]);
  }
  if (softmax) {
    m = warp_max(m);
    if (m == -INFINITY) m = 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < HELD; ++i) sum += expf(x[i] - m);
    sum = warp_sum(sum);
    inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  }
  __syncwarp();
  float r[HELD];
#pragma unroll
  for (int i = 0; i < HELD; ++i) {
    const int e = lane + 32 * i;
    r[i] = x[i];
    if (e < a.E) {
      if (!softmax) r[i] = sigmoid(x[i]) + (a.bias != nullptr ? a.bias[e] : 0.0f);
      if (!(x[i] > -INFINITY) || !(r[i] > -INFINITY)) r[i] = -INFINITY;
      row[e] = r[i];
    }
  }
  __syncwarp();
  const int size = a.E / a.n_group;
  unsigned keep = ALL;
  if (a.n_group > 1) {
    float m1 = -INFINITY, m2 = -INFINITY;
    if (lane < a.n_group)
#pragma unroll 4
      for (int i = 0; i < size; ++i) merge_top2(m1, m2, row[lane * size + i], -INFINITY);
    if (softmax && a.group_top2) m1 = m1 > -INFINITY ? expf(m1 - m) : m1, m2 = m2 > -INFINITY ? expf(m2 - m) : m2;
    const float value = a.group_top2 && m2 > -INFINITY ? m1 + m2 : m1;
    int better = 0;
    for (int h = 0; h < a.n_group; ++h) {
      const float o = __shfl_sync(ALL, value, h);
      better += h < lane ? o >= value : o > value;
    }
    keep = __ballot_sync(ALL, lane < a.n_group && better < a.topk_group);
  }
  uint32_t key[HELD];  // 0: not in play, or taken
#pragma unroll
  for (int i = 0; i < HELD; ++i) {
    const int e = lane + 32 * i;
    key[i] = e < a.E && (a.n_group == 1 || (keep >> (e / size)) & 1u) ? ordered(r[i]) : 0u;
  }
  int my_e = 0;
  for (int j = 0; j < a.k; ++j) {
    uint32_t top = 0u;
    int at = 0;
#pragma unroll
    for (int i = 0; i < HELD; ++i)
      if (key[i] > top) top = key[i], at = i;
    const uint32_t best = __reduce_max_sync(ALL, top);
    const int e = __reduce_min_sync(ALL, top == best ? lane + 32 * at : MAX_EXPERTS);
#pragma unroll
    for (int i = 0; i < HELD; ++i)
      if (lane + 32 * i == e) key[i] = 0u;
    if (lane == j) my_e = e;
  }
  if (lane < a.k) {
    const float xe = to_f32(from[my_e]);
    *score = softmax ? expf(xe - m) * inv : sigmoid(xe);
  }
  return my_e;
}

constexpr int SM_SHARED = 228 * 1024, BLOCK_RESERVED = 1024 + 256;  // shared memory of an SM; of a block, beside ours
constexpr int SLOW_TOKENS = 32;  // at least a batch
constexpr int LIST = 64;
// A warp's shared memory, but for its rank values and sums.
struct __align__(16) Scratch {
  float value[2][LIST];      // rank values of the two tokens' listed experts, -inf behind them (read four at a time)
  uint16_t expert[2][LIST];
  int pick[32];               // selected experts of the tokens of a batch
  float shift[32], inv[32];   // of the softmax of each
  int64_t slow[SLOW_TOKENS];  // tokens left over
};
static_assert(sizeof(Scratch) % 16 == 0 && offsetof(Scratch, value) == 0, "read in words of 16 bytes");

// Bytes that a lane's C experts are read and written by.
template <int C, typename T>
constexpr int unit_of() {
  constexpr int BYTES = C * (int)sizeof(T);
  return BYTES % 16 == 0 ? 16 : BYTES % 8 == 0 ? 8 : 4;
}
// Floats from one lane's C values to the next lane's in shared memory: 8 lanes' accesses of 16 bytes (16 of 8) then
// fall on all 32 banks.
template <int C>
constexpr int lane_stride() {
  return C == 8 || C == 16 ? C + 4 : C;
}

// Bytes from one lane's logits to the next lane's in shared memory, with the same effect.
template <int C, typename TL>
constexpr int slot_bytes() {
  return sizeof(TL) == 4 ? lane_stride<C>() * 4 : C == 16 ? 48 : C * 2;
}
// A lane's copies of its experts' logits, `held` of C places, to shared memory (cp.async) and the reading of them.
template <int C, typename TL>
__device__ __forceinline__ void copy_part(uint32_t to, const TL* from, int held) {
  constexpr int BYTES = C * (int)sizeof(TL), UNIT = unit_of<C, TL>(), OF_UNIT = UNIT / (int)sizeof(TL);
#pragma unroll
  for (int j = 0; j < BYTES / UNIT; ++j) {
    if (j * OF_UNIT < held) {
      if constexpr (UNIT == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + j * UNIT), "l"(from + j * OF_UNIT) : "memory");
      else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to + j * UNIT), "l"(from + j * OF_UNIT), "n"(UNIT)
                     : "memory");
    }
  }
}
template <int C, typename TL>
__device__ __forceinline__ void read_part(const unsigned char* slot, float (&x)[C]) {
  constexpr int BYTES = C * (int)sizeof(TL), UNIT = unit_of<C, TL>();
  uint32_t w[BYTES / 4];
#pragma unroll
  for (int j = 0; j < BYTES / UNIT; ++j) {
    if constexpr (UNIT == 16) {
      const uint4 v = reinterpret_cast<const uint4*>(slot)[j];
      w[4 * j] = v.x, w[4 * j + 1] = v.y, w[4 * j + 2] = v.z, w[4 * j + 3] = v.w;
    } else if constexpr (UNIT == 8) {
      const uint2 v = reinterpret_cast<const uint2*>(slot)[j];
      w[2 * j] = v.x, w[2 * j + 1] = v.y;
    } else {
      w[j] = reinterpret_cast<const uint32_t*>(slot)[j];
    }
  }
#pragma unroll
  for (int j = 0; j < BYTES / 4; ++j) {
    if constexpr (sizeof(TL) == 4) x[j] = __uint_as_float(w[j]);
    else x[2 * j] = __uint_as_float(w[j] << 16), x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
  }
}
// The same from global memory, one at a time; -inf behind them.
template <int C, typename TL>
__device__ __forceinline__ void load_part(const TL* from, int held, float (&x)[C]) {
#pragma unroll
  for (int c = 0; c < C; ++c) {
    x[c] = -INFINITY;
    if (c < held) x[c] = to_f32(from[c]);
  }
}

// A lane's C values in shared (or 16-byte aligned global) memory.
template <int C>
__device__ __forceinline__ void put(float* to, const float (&v)[C]) {
  if constexpr (C % 4 == 0) {
#pragma unroll
    for (int c = 0; c < C; c += 4) *reinterpret_cast<float4*>(to + c) = make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]);
  } else {
#pragma unroll
    for (int c = 0; c < C; c += 2) *reinterpret_cast<float2*>(to + c) = make_float2(v[c], v[c + 1]);
  }
}
template <int C>
__device__ __forceinline__ void get(const float* from, float (&v)[C]) {
  if constexpr (C % 4 == 0) {
#pragma unroll
    for (int c = 0; c < C; c += 4) {
      const float4 f = *reinterpret_cast<const float4*>(from + c);
      v[c] = f.x, v[c + 1] = f.y, v[c + 2] = f.z, v[c + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int c = 0; c < C; c += 2) {
      const float2 f = *reinterpret_cast<const float2*>(from + c);
      v[c] = f.x, v[c + 1] = f.y;
    }
  }
}

__device__ __forceinline__ float min_nan(float a, float b, float c) {  // NaN if one is
  float r;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// bits with x's sign behind them
__device__ __forceinline__ uint32_t push_sign(uint32_t bits, float x) {
  return __funnelshift_l(__float_as_uint(x), bits, 1);
}

// The two largest of N values, none of them NaN.
template <int N>
__device__ __forceinline__ void two_largest(const float (&v)[N], float& first, float& second) {
  first = fmaxf(v[0], v[1]), second = fminf(v[0], v[1]);
#pragma unroll
  for (int c = 2; c < N; c += 2) {
    const float hi = fmaxf(v[c], v[c + 1]), lo = fminf(v[c], v[c + 1]);
    second = fmaxf(fmaxf(fminf(first, hi), second), lo), first = fmaxf(first, hi);
  }
}

// over the lanes of a token
template <int LANES>
__device__ __forceinline__ float token_max(float x) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(ALL, x, o));
  return x;
}
template <int LANES>
__device__ __forceinline__ float token_min(float x) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) x = fminf(x, __shfl_xor_sync(ALL, x, o));
  return x;
}
template <int LANES>
__device__ __forceinline__ float token_sum(float x) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) x += __shfl_xor_sync(ALL, x, o);
  return x;
}

// Writes the selected expert e of token t (`on`: this lane has one) and its gate, as the layer's ungrouped top-k
// forms it: the sum over the token's lanes, from `first` on, in the order of the selection (a lane without an expert
// adds 0).
template <typename TL, PairMode MODE>
__device__ __forceinline__ void store_selected(const RouteArgs& a, int64_t t, bool on, int j_of, int first, int e,
                                               float shift, float inv, int* counts) {
  float sel = 0.0f;
  if (on) {
    const float xe = to_f32(static_cast<const TL*>(a.logits)[t * a.stride + e]);
    sel = MODE == LOGITS ? expf(xe - shift) * inv : sigmoid(xe);
  }
  float sum = 0.0f;
  if (a.renorm) {
    if (a.slot_bits <= 3) {
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += j >> a.slot_bits ? 0.0f : __shfl_sync(ALL, sel, first + j);
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) sum += __shfl_sync(ALL, sel, first + j);
    }
  }
  if (on) {
    a.topk_idx[t * a.k + j_of] = e;
    if (a.gates != nullptr)
      a.gates[t * a.k + j_of] = (!a.renorm ? sel : sum == 0.0f ? 0.0f : sel * (1.0f / sum)) * a.scale;
    if (counts != nullptr) atomicAdd(&counts[e], 1);
  }
}

// How the experts lie on a token's lanes: a group on `lanes` of them, a power of two, C to a lane, the last ones fewer.
struct Place {
  int lanes, group;  // lanes of a group; this lane's
  int first, held;   // this lane's experts
  bool bounds;       // its segment has two experts or more
  bool choose, top2;
};

// The selection of a warp's tokens, one on each LANES lanes, from the lanes' rank values r (shift: of each softmax):
// the experts in pick.  FAST: r is approximate; what that leaves open is settled on exact values, of the token's logits
// `own` from this lane's first on and their bias.  False (on all lanes of a token): more than the list holds, or too few
// experts.
//
// An approximate rank value v = s + b is off by less than 4e-7 + 2^-23 |v|: the order of two is certain from twice that
// on, and more is taken.  The distance goes by the value itself: a far larger bias of another expert (the type's lowest
// value, as a mask) leaves the order of the others certain.
__device__ __forceinline__ float distance_of(float v) { return fmaf(5e-7f, fabsf(v), 1.5e-6f); }
template <int LANES, int C, bool LOGIT_VALUES, bool FAST, typename TL>
__device__ __forceinline__ bool select_pair(const RouteArgs& a, const Place& p, const TL* own, const float* bias,
                                            float (&r)[C], float shift, float group_distance, int lane, float* mine,
                                            Scratch& w, int* pick) {
  const int half = lane / LANES, part = lane % LANES;
  if (part < 16) w.value[half][part] = -INFINITY;
  if (FAST && part < a.k) pick[part] = -1;
  bool in_play = p.held > 0;
  float low;  // the segment's second largest
  for (bool exact = !FAST;; exact = true) {
    put(mine, r);
    // 1. the two largest of the lane, of its segment and of its group
    float m1, m2;
    two_largest(r, m1, m2);
    low = m2;
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) {
      if (o < p.lanes) {
        merge_top2(m1, m2, __shfl_xor_sync(ALL, m1, o), __shfl_xor_sync(ALL, m2, o));
        if (o < a.segment_lanes) low = m2;
      }
    }
    if (!p.choose) break;
    // 2. the groups.  Each lane of a group counts the better ones among every lanes-th group
    float value = m1;
    if (p.top2) {
      if (LOGIT_VALUES) value = m1 > -INFINITY ? expf(m1 - shift) + expf(m2 - shift) : m1;
      else value = m2 > -INFINITY ? m1 + m2 : m1;
    }
    const int first = part & (p.lanes - 1);
    auto count = [&](auto better) {
      int n = 0;
#pragma unroll 2
      for (int h = first; h - first < a.n_group; h += p.lanes) {
        const float o = __shfl_sync(ALL, value, half * LANES + h * p.lanes);
        n += h < a.n_group && better(h, o);
      }
#pragma unroll
      for (int o = 1; o < LANES; o <<= 1)
        if (o < p.lanes) n += __shfl_xor_sync(ALL, n, o);
      return n;
    };
    if (exact) {
      const int better = count([&](int h, float o) { return h < p.group ? o >= value : o > value; });
      in_play = p.held > 0 && better < a.topk_group;
      break;
    }
    // those that might be better, itself among them: up to topk_group of these, and it is chosen for certain
    const float reach = value - fmaf(3e-7f, fabsf(value), group_distance);
    const int near = count([&](int, float o) { return o > reach; });
    in_play = near <= a.topk_group && value > -INFINITY;
    const unsigned chosen = __ballot_sync(ALL, in_play) >> (half * LANES) & (ALL >> (32 - LANES));
    if (!__any_sync(ALL, __popc(chosen) != a.topk_group * p.lanes)) break;
    __syncwarp();
#pragma unroll 1
    for (int c = 0; c < C; ++c) {
      const float x = c < p.held ? to_f32(own[c]) : -INFINITY;
      mine[c] = x > -INFINITY ? sigmoid(x) + bias[c] : -INFINITY;
    }
    get(mine, r);
  }
  // 3. the listed experts, in their order
  float bound = token_min<LANES>(in_play && p.bounds ? low : INFINITY);
  const bool none = !(bound > -INFINITY);
  // (never -inf, the value of masked experts and of places without one)
  if (FAST) bound = fmaxf(bound - distance_of(bound), -FLT_MAX);
  unsigned listed = 0u;
#pragma unroll
  for (int c = 0; c < C; ++c) listed |= r[c] >= bound ? 1u << c : 0u;
  if (!in_play) listed = 0u;  // (with +inf among its values too)
  const int of_lane = __popc(listed);
  int before = of_lane;
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) {
    const int v = __shfl_up_sync(ALL, before, o, LANES);
    if (part >= o) before += v;
  }
  int n = __shfl_sync(ALL, before, lane | (LANES - 1));
  const bool out = none || n > LIST || n < a.k;  // the same on the token's lanes
  if (out) n = 0, listed = 0u;
  before -= of_lane;
  __syncwarp();  // behind the first values and picks
  while (listed != 0u) {
    const int c = __ffs(listed) - 1;
    listed &= listed - 1u;
    w.value[half][before] = mine[c];
    w.expert[half][before++] = p.first + c;
  }
  // 4. their places, 16 against 16; -inf behind the list, as far as the longer of the two lists is read
  const int longest = LANES == 32 ? n : max(n, __shfl_xor_sync(ALL, n, 16));
  if (longest > 16) {
    for (int at = 16 + part; at - part < longest; at += LANES)
      if (at >= n && at < LIST) w.value[half][at] = -INFINITY;
  }
  __syncwarp();
  if (FAST) {
    for (int at = part; at - part < longest; at += LANES) {  // how many might be better, itself among them
      const float v = w.value[half][at], far = v - distance_of(v);
      const F2 reach = f2(far, far);
      int better = -1;
      for (int block = 0; block < longest; block += 16) {
        uint32_t signs = 0u;
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const float4 o = *reinterpret_cast<const float4*>(&w.value[half][block + j]);
          float d0, d1, d2, d3;
          split(fma2(f2(o.x, o.y), f2(-1.0f, -1.0f), reach), d0, d1);
          split(fma2(f2(o.z, o.w), f2(-1.0f, -1.0f), reach), d2, d3);
          signs = push_sign(push_sign(push_sign(push_sign(signs, d0), d1), d2), d3);
        }
        better += __popc(signs);
      }
      // (-1 for +inf, of which nothing is certain: a difference that is NaN counts nothing, itself neither)
      if (at < n && (unsigned)better < (unsigned)a.k) pick[better] = w.expert[half][at];
    }
    // Where each of the best k is at least the distance above the next, it has its place; else the first that is not
    // leaves its own empty, and the places are counted again on the exact values.
    __syncwarp();
    if (!__any_sync(ALL, n > 0 && part < a.k && pick[part] < 0)) return !out;
    for (int at = part; at < n; at += LANES) {
      const int e = w.expert[half][at];
      w.value[half][at] = sigmoid(to_f32(own[e - p.first])) + fmaxf(a.bias[e], -INFINITY);
    }
    __syncwarp();
  }
  for (int at = part; at - part < longest; at += LANES) {
    const float v = w.value[half][at];
    int better = 0;
    for (int block = 0; block < longest; block += 16) {
#pragma unroll
      for (int j = 0; j < 16; j += 4) {  // ties to the expert before
        const float4 o = *reinterpret_cast<const float4*>(&w.value[half][block + j]);
        better += at > block + j ? o.x >= v : o.x > v;
        better += at > block + j + 1 ? o.y >= v : o.y > v;
        better += at > block + j + 2 ? o.z >= v : o.z > v;
        better += at > block + j + 3 ? o.w >= v : o.w > v;
      }
    }
    if (at < n && better < a.k) pick[better] = w.expert[half][at];
  }
  return !out;
}

template <int LANES, int C, typename TL, PairMode MODE>
__global__ void __launch_bounds__(THREADS, blocks_of_sm(MODE)) route_pairs_kernel(const RouteArgs a) {
  // [LANES] lanes' bias, [WARPS][32] lanes' rank values, [WARPS][32] lanes' logits; balance: [LANES C] counts,
  // [WARPS][32] lanes' sums
  extern __shared__ __align__(16) float sh[];
  constexpr int S = lane_stride<C>();
  __shared__ Scratch scratch[WARPS];
  constexpr bool FAST = MODE == SIGMOID_FAST;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = lane / LANES, part = lane % LANES;
  constexpr int TOKENS = 32 / LANES;
  const int E = a.E, k = a.k;
  const bool balance = a.ticket != nullptr;
  float* rows = sh + LANES * S;
  constexpr int SLOT = slot_bytes<C, TL>();
  unsigned char* slots = reinterpret_cast<unsigned char*>(rows + WARPS * 32 * S);
  int* counts = balance ? reinterpret_cast<int*>(slots + WARPS * 32 * SLOT) : nullptr;
  float* sums = reinterpret_cast<float*>(slots + WARPS * 32 * SLOT) + LANES * C;
  Scratch& w = scratch[warp];
  float* mine = rows + (warp * 32 + lane) * S;
  float* my_sums = sums + (warp * 32 + lane) * S;
  const float* bias = sh + part * S;
  const int size = a.group_size, lane_bits = a.n_group > 1 ? a.group_lane_bits : LANES == 32 ? 5 : 4, lanes = 1 << lane_bits;
  for (int i = threadIdx.x; i < LANES * C; i += THREADS) {
    const int l = i / C, c = i % C, group = l >> lane_bits, at = (l & (lanes - 1)) * C + c, e = group * size + at;
    const bool in = group < a.n_group && at < size;
    sh[l * S + c] = !in ? -INFINITY : a.bias != nullptr ? fmaxf(a.bias[e], -INFINITY) : 0.0f;  // no NaN
  }
  if (balance) {
    for (int e = threadIdx.x; e < LANES * C; e += THREADS) counts[e] = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) my_sums[c] = 0.0f;
  }
  __syncthreads();
  // A group's value is the sum of two, each off as distance_of has it, whatever is left of them in the sum; biases from
  // 2^26 on take every s without a trace, so that such a rank value is exact.
  float group_distance = 0.0f;
  if (FAST) {
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (fabsf(bias[c]) < 67108864.0f) group_distance = fmaxf(group_distance, fabsf(bias[c]));
    group_distance = 2.0f * distance_of(1.0f + warp_max(group_distance));
  }
  const int group = part >> lane_bits, in_group = (part & (lanes - 1)) * C;
  const int held = group < a.n_group ? max(0, min(C, size - in_group)) : 0;
  const Place place = {lanes, group, held > 0 ? group * size + in_group : 0, held,
                       held > 0 && (part & (lanes - a.segment_lanes)) * C + 1 < size,
                       a.topk_group < a.n_group, a.group_top2 != 0};
  const int slot = lane >> a.slot_bits, j_of = lane & ((1 << a.slot_bits) - 1);
  const int64_t step = (int64_t)gridDim.x * WARPS * a.batch;
  int64_t base = ((int64_t)blockIdx.x * WARPS + warp) * a.batch;
  const TL* logits = static_cast<const TL*>(a.logits);

  // The logits of the next tokens come under the arithmetic of these; a lane's own copies, so that there is no barrier.
  unsigned char* my_slot = slots + (warp * 32 + lane) * SLOT;
  const bool copied = a.words;
  auto fetch = [&](int64_t first) {
    if (copied && first < a.T)
      copy_part<C, TL>((uint32_t)__cvta_generic_to_shared(my_slot),
                       logits + min(first + half, a.T - 1) * a.stride + place.first, held);
  };
#pragma unroll
  for (int c = 0; c < C; ++c) from_f32(-INFINITY, reinterpret_cast<TL*>(my_slot) + c);
  fetch(base);
  while (base < a.T) {
    int slow_count = 0;
    for (; base < a.T && slow_count + a.batch <= SLOW_TOKENS; base += step) {
      const int count = (int)min((int64_t)a.batch, a.T - base);
      unsigned passed = 0u;  // tokens of the batch that are left over
      for (int i = 0; i < count; i += TOKENS) {
        const bool on = i + half < count;
        const int64_t t = base + (on ? i + half : i);
        float x[C], s[C], r[C];
        if (copied) {
          asm volatile("cp.async.wait_all;" ::: "memory");
          read_part<C, TL>(my_slot, x);
          fetch(i + TOKENS < count ? base + i + TOKENS : base + step);
        } else {
          load_part<C>(logits + t * a.stride + place.first, held, x);
        }
        float inv = 1.0f, shift = 0.0f, least = INFINITY;
#pragma unroll
        for (int c = 0; c < C; c += 2) least = min_nan(least, x[c], x[c + 1]);
        if constexpr (MODE == LOGITS) {
          shift = -INFINITY;
          float sum = 0.0f;
#pragma unroll
          for (int c = 0; c < C; ++c) shift = fmaxf(shift, x[c]);
          shift = token_max<LANES>(shift);
          if (shift == -INFINITY) shift = 0.0f;
#pragma unroll
          for (int c = 0; c < C; c += 2) {
            exp_pair(x[c], x[c + 1], shift, s[c], s[c + 1]);
            sum += s[c];
            sum += s[c + 1];
            r[c] = x[c], r[c + 1] = x[c + 1];
          }
          sum = token_sum<LANES>(sum);
          inv = sum == 0.0f ? 0.0f : 1.0f / sum;
          if (part == 0) w.shift[i + half] = shift, w.inv[i + half] = inv;
        } else {
          get(bias, r);
          if constexpr (FAST) {
#pragma unroll
            for (int c = 0; c < C; c += 2) {
              float e0, e1;
              split(mul2(f2(x[c], x[c + 1]), f2(-LOG2E, -LOG2E)), e0, e1);
              split(add2(f2(exp2_fast(e0), exp2_fast(e1)), f2(1.0f, 1.0f)), e0, e1);
              s[c] = inverse_fast(e0), s[c + 1] = inverse_fast(e1);
              split(add2(f2(s[c], s[c + 1]), f2(r[c], r[c + 1])), r[c], r[c + 1]);
            }
          } else {
#pragma unroll
            for (int c = 0; c < C; ++c) {
              s[c] = sigmoid(x[c]);
              r[c] += s[c];
            }
          }
        }
        if (__any_sync(ALL, held > 0 && !(least > -INFINITY))) {  // masked experts, or NaN
#pragma unroll
          for (int c = 0; c < C; ++c) r[c] = x[c] > -INFINITY ? r[c] : -INFINITY;
        }
        int* pick = w.pick + ((i + half) << a.slot_bits);
        const bool done = select_pair<LANES, C, MODE == LOGITS, FAST>(a, place, logits + t * a.stride + place.first, bias,
                                                                      r, shift, group_distance, lane, mine, w, pick);
        const unsigned skips = __ballot_sync(ALL, !done && on);
#pragma unroll
        for (int h = 0; h < TOKENS; ++h) {
          if (skips >> (h * LANES) & 1u) {
            passed |= 1u << (i + h);
            if (lane == 0) w.slow[slow_count] = base + i + h;
            ++slow_count;
          }
        }
        if (a.scores != nullptr && on && held > 0) {
          float* to = a.scores + t * E + place.first;
#pragma unroll
          for (int c = 0; c < C; ++c) r[c] = s[c] * inv;
          if (a.wide_scores) {
            put(to, r);
          } else {
#pragma unroll
            for (int c = 0; c < C; ++c)
              if (c < held) to[c] = r[c];
          }
        }
        if (balance) {
          float q = inv;
          if (MODE != LOGITS) {
            float total = 0.0f;
#pragma unroll
            for (int c = 0; c < C; ++c) total += s[c];  // 0 in places without an expert
            total = token_sum<LANES>(total);
            q = total == 0.0f ? 0.0f : 1.0f / total;
          }
          if (on) {
            float sum[C];
            get(my_sums, sum);
#pragma unroll
            for (int c = 0; c < C; ++c) sum[c] = fmaf(s[c], q, sum[c]);
            put(my_sums, sum);
          }
        }
        __syncwarp();  // the lists are free again, the picks can be read
      }
      // 5.
      const bool on = slot < count && j_of < k && !((passed >> slot) & 1u);
      store_selected<TL, MODE>(a, base + slot, on, j_of, slot << a.slot_bits, on ? w.pick[lane] : 0,
                               MODE == LOGITS && on ? w.shift[slot] : 0.0f, MODE == LOGITS && on ? w.inv[slot] : 1.0f,
                               counts);
      __syncwarp();  // the picks are free again
    }
    // the tokens left over, in a loop of their own: no call stands in the loop over the others
    for (int i = 0; i < slow_count; ++i) {
      const int64_t t = w.slow[i];
      float score = 0.0f;
      const int e = select_by_warp<TL, LANES * C / 32>(a, t, rows + warp * 32 * S, lane, &score);
      float sum = 0.0f;
      for (int j = 0; j < k; ++j) sum += __shfl_sync(ALL, score, j);
      if (lane < k) {
        a.topk_idx[t * k + lane] = e;
        if (a.gates != nullptr)
          a.gates[t * k + lane] = (!a.renorm ? score : sum == 0.0f ? 0.0f : score * (1.0f / sum)) * a.scale;
        if (balance) atomicAdd(&counts[e], 1);
      }
    }
    __syncwarp();
  }
  if (balance) {
    __syncthreads();
    finish_balance(a, counts, [&](int e) {
      float p = 0.0f;
      const int group = (int)(((float)e + 0.5f) * a.inv_group_size), at = e - group * size;
      const int l = (group << lane_bits) + at / C, c = at % C;
#pragma unroll
      for (int h = 0; h < TOKENS * WARPS; ++h) p += sums[(h * LANES + l) * S + c];
      return p;
    });
  }
}

// How the experts lie on lanes, if there is a kernel for it (token_lanes 0: there is none).  16 lanes for a token where
// they hold its groups, else 32.
struct Layout {
  int token_lanes, per_lane, group_lanes, segment_lanes;
};
Layout layout_of(const RouteArgs& a) {
  if (a.E > MAX_EXPERTS || (a.router == 0 && a.bias != nullptr)) return {};
  const int size = a.E / a.n_group;
  for (int token_lanes = 16; token_lanes <= 32; token_lanes *= 2) {
    for (const int C : {4, 8, 10, 12, 16}) {
      if (token_lanes == 32 && C < 12) continue;
      const int used = (size + C - 1) / C;
      int group_lanes = 1;
      while (group_lanes < used) group_lanes *= 2;
      if (group_lanes * a.n_group > token_lanes) continue;
      // the longest segments, of which topk_group groups hold k experts in segments of two or more
      for (int segment = group_lanes; segment > 0; segment /= 2) {
        const int places = segment * C, segments = size / places + (size % places >= 2);
        if (2 * a.topk_group * segments >= a.k) return {token_lanes, C, a.n_group > 1 ? group_lanes : token_lanes, segment};
      }
    }
  }
  return {};
}

template <int LANES, int C, typename TL, PairMode MODE>
cudaError_t launch_pairs(const RouteArgs& args, const Layout& layout, int n_sm, cudaStream_t st) {
  RouteArgs a = args;
  constexpr int UNIT = unit_of<C, TL>(), S = lane_stride<C>();
  const int size = a.E / a.n_group;
  a.group_size = size;
  a.inv_group_size = 1.0f / (float)size;
  a.group_lane_bits = 0;
  while (1 << a.group_lane_bits < layout.group_lanes) ++a.group_lane_bits;
  a.segment_lanes = layout.segment_lanes;
  const bool words = reinterpret_cast<uintptr_t>(a.logits) % UNIT == 0 && a.stride * (int64_t)sizeof(TL) % UNIT == 0 &&
                     size * (int)sizeof(TL) % UNIT == 0;
  a.words = words;
  constexpr int SCORES_UNIT = C % 4 == 0 ? 16 : 8;
  a.wide_scores = reinterpret_cast<uintptr_t>(a.scores) % SCORES_UNIT == 0 && a.E * 4 % SCORES_UNIT == 0 && size % C == 0;
  a.slot_bits = 0;
  while ((1 << a.slot_bits) < a.k) ++a.slot_bits;
  const bool balance = a.ticket != nullptr;
  const int smem = (LANES * S + WARPS * 32 * S + (balance ? LANES * C + WARPS * 32 * S : 0)) * 4 +
                   WARPS * 32 * slot_bytes<C, TL>();
  const int resident = std::min<int>(blocks_of_sm(MODE), SM_SHARED / (smem + (int)sizeof(Scratch) * WARPS + BLOCK_RESERVED));
  // tokens whose gates are formed together: as many as fill a warp, once every resident warp has a batch
  a.batch = 32 >> a.slot_bits;
  while (a.batch > 32 / LANES && a.T < (int64_t)a.batch * WARPS * resident * n_sm) a.batch >>= 1;
  auto kernel = route_pairs_kernel<LANES, C, TL, MODE>;
  if (smem > 36 * 1024) {
    const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
  }
  const int64_t want = (a.T + (int64_t)WARPS * a.batch - 1) / ((int64_t)WARPS * a.batch);
  const int blocks = (int)std::max<int64_t>(1, std::min<int64_t>(want, resident * n_sm));
  kernel<<<blocks, THREADS, smem, st>>>(a);
  return cudaGetLastError();
}

template <int LANES, int C, typename TL>
cudaError_t launch_mode(const RouteArgs& a, const Layout& l, int n_sm, cudaStream_t st) {
  if (a.router == 0) return launch_pairs<LANES, C, TL, LOGITS>(a, l, n_sm, st);
  // without a bias ties are common (equal logits), and the scores that are handed out are the exact ones
  if (a.bias != nullptr && a.scores == nullptr) return launch_pairs<LANES, C, TL, SIGMOID_FAST>(a, l, n_sm, st);
  return launch_pairs<LANES, C, TL, SIGMOID>(a, l, n_sm, st);
}

template <typename TL>
cudaError_t launch_type(const RouteArgs& a, int n_sm, cudaStream_t st) {
  const Layout l = layout_of(a);
  switch (l.token_lanes * 100 + l.per_lane) {
    case 1604: return launch_mode<16, 4, TL>(a, l, n_sm, st);
    case 1608: return launch_mode<16, 8, TL>(a, l, n_sm, st);
    case 1610: return launch_mode<16, 10, TL>(a, l, n_sm, st);
    case 1612: return launch_mode<16, 12, TL>(a, l, n_sm, st);
    case 1616: return launch_mode<16, 16, TL>(a, l, n_sm, st);
    case 3212: return launch_mode<32, 12, TL>(a, l, n_sm, st);
    case 3216: return launch_mode<32, 16, TL>(a, l, n_sm, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

bool route_pairs_fit(const RouteArgs& a) { return layout_of(a).token_lanes != 0; }

cudaError_t launch_route_pairs(const RouteArgs& a, bool bf16, int n_sm, cudaStream_t st) {
  return bf16 ? launch_type<__nv_bfloat16>(a, n_sm, st) : launch_type<float>(a, n_sm, st);
}

}  // namespace mok
