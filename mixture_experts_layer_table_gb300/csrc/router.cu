// Group-limited expert selection from router logits, with the load-balancing outputs, and its backward.
//
// One warp takes one token at a time; lane l holds the C consecutive experts from l * C on, C = ceil(E / 32)
// rounded up to a size there is a kernel for.  With s the scores (sigmoid, or softmax over the experts):
//   rank value r = s + bias; a softmax without a bias is ranked by its logits (it is increasing, and the logits
//   have no rounding of the sum in them).  A logit of -inf or NaN ranks behind every other.
//   group value: the largest r of the group, or the sum of its two largest (of e^(x - max) for the softmax
//   without a bias); the topk_group best groups stay, then the k best experts in them; ties to the lower index.
//   gate = scale * s, or scale * s / (the sum of the k selected s), 0 where that sum is 0.
// A warp keeps its row in registers, so that each round of the top-k is C maxima, one reduction over the warp and one
// ballot.  Few tokens are bound by the chain of these steps: 1 token of 256 experts 3.8 us, 8 tokens 4.3, 1,024 tokens
// 4.7.  Many tokens come here only where the other kernel has no form: a softmax with a bias (65,536 tokens of 256: 95 us)
// and more than 512 experts (16,384 tokens of 1,024: 190 us).
#include <algorithm>

#include "router_common.cuh"
#include "status.cuh"

namespace mok {

namespace {

constexpr int WARPS = 8;
constexpr int THREADS = 32 * WARPS;

template <int C, typename TL>
__device__ __forceinline__ void load_row(const TL* row, int lane, int E, float (&x)[C]) {
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int e = lane * C + c;
    x[c] = e < E ? to_f32(row[e]) : -INFINITY;
  }
}

// Softmax of a row held C to a lane: e^(x - max) in place of x, and 1 / sum (0 for a row of -inf).
template <int C>
__device__ __forceinline__ float softmax_row(float (&x)[C], float* max_out) {
  float m = -INFINITY;
#pragma unroll
  for (int c = 0; c < C; ++c) m = fmaxf(m, x[c]);
  m = warp_max(m);
  const float shift = m == -INFINITY ? 0.0f : m;
  float sum = 0.0f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    x[c] = expf(x[c] - shift);
    sum += x[c];
  }
  *max_out = shift;
  sum = warp_sum(sum);
  return sum == 0.0f ? 0.0f : 1.0f / sum;
}

template <int C, typename TL>
__global__ void __launch_bounds__(THREADS) route_kernel(const RouteArgs a) {
  extern __shared__ float sh[];  // [WARPS][E] a row of each warp; [E] counts
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = a.E, k = a.k;
  const bool balance = a.ticket != nullptr;
  float* my_row = sh + warp * E;
  int* sh_counts = reinterpret_cast<int*>(sh + WARPS * E);
  if (balance) {
    for (int e = threadIdx.x; e < E; e += THREADS) sh_counts[e] = 0;
    __syncthreads();
  }
  const int size = E / a.n_group;
  const int lanes = size / C;  // lanes of a group where groups are whole lanes
  const bool whole_lanes = size % C == 0 && (lanes & (lanes - 1)) == 0;

  float b[C], acc[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int e = lane * C + c;
    b[c] = a.bias != nullptr && e < E ? a.bias[e] : 0.0f;
    acc[c] = 0.0f;
  }

  for (int64_t t = (int64_t)blockIdx.x * WARPS + warp; t < a.T; t += (int64_t)gridDim.x * WARPS) {
    float x[C], s[C];
    load_row<C>(static_cast<const TL*>(a.logits) + t * a.stride, lane, E, x);
    float inv = 1.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) s[c] = x[c];
    if (a.router == 0) {
      float m;
      inv = softmax_row<C>(s, &m);
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c) s[c] = sigmoid(x[c]);
    }
    // rank values r and, for the groups, g
    float r[C], g[C];
    const bool by_logit = a.router == 0 && a.bias == nullptr;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float v = by_logit ? x[c] : s[c] * inv + b[c];
      float w = by_logit && a.group_top2 ? s[c] : v;
      if (!(x[c] > -INFINITY) || !(v > -INFINITY)) v = w = -INFINITY;
      r[c] = v;
      g[c] = w;
    }
    unsigned keep = ALL;  // whole_lanes: nonzero if this lane's group stays; else one bit for each group
    if (a.n_group > 1) {
      float value;
      if (whole_lanes) {
        float m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
        for (int c = 0; c < C; ++c) merge_top2(m1, m2, g[c], -INFINITY);
        for (int o = 1; o < lanes; o <<= 1) {
          const float o1 = __shfl_xor_sync(ALL, m1, o), o2 = __shfl_xor_sync(ALL, m2, o);
          merge_top2(m1, m2, o1, o2);
        }
        value = a.group_top2 && m2 > -INFINITY ? m1 + m2 : m1;
        const int mine = lane / lanes;
        int better = 0;
        for (int h = 0; h < a.n_group; ++h) {
          const float o = __shfl_sync(ALL, value, h * lanes);
          better += o > value || (o == value && h < mine);
        }
        keep = better < a.topk_group ? ALL : 0u;
      } else {
        __syncwarp();
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (lane * C + c < E) my_row[lane * C + c] = g[c];
        __syncwarp();
        float m1 = -INFINITY, m2 = -INFINITY;
        if (lane < a.n_group)
          for (int i = 0; i < size; ++i) merge_top2(m1, m2, my_row[lane * size + i], -INFINITY);
        value = a.group_top2 && m2 > -INFINITY ? m1 + m2 : m1;
        int better = 0;
        for (int h = 0; h < a.n_group; ++h) {
          const float o = __shfl_sync(ALL, value, h);
          better += o > value || (o == value && h < lane);
        }
        keep = __ballot_sync(ALL, lane < a.n_group && better < a.topk_group);
      }
    }
    // keys: 0 for what cannot be selected
    uint32_t key[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int e = lane * C + c;
      const bool in = e < E && (whole_lanes || a.n_group == 1 ? keep != 0u : (keep >> (e / size)) & 1u);
      key[c] = in ? ordered(r[c]) : 0u;
    }
    int my_e = 0;
    float my_s = 0.0f;
    for (int j = 0; j < k; ++j) {
      uint32_t top = 0u;
#pragma unroll
      for (int c = 0; c < C; ++c) top = max(top, key[c]);
      const uint32_t best = __reduce_max_sync(ALL, top);
      const int src = __ffs(__ballot_sync(ALL, top == best)) - 1;
      int ec = 0;
      float sc = 0.0f;
      bool found = false;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const bool here = !found && key[c] == best;
        if (here) {
          ec = lane * C + c;
          sc = s[c];
          if (lane == src) key[c] = 0u;
        }
        found = found || here;
      }
      ec = __shfl_sync(ALL, ec, src);
      sc = __shfl_sync(ALL, sc, src);
      if (lane == j) {
        my_e = ec;
        my_s = sc * inv;
      }
    }
    // the gates as the layer's ungrouped top-k forms them: the sum in the order of the selection
    float sum = 0.0f;
    if (a.renorm)
      for (int j = 0; j < k; ++j) sum += __shfl_sync(ALL, my_s, j);
    if (lane < k) {
      a.topk_idx[t * k + lane] = my_e;
      if (a.gates != nullptr)
        a.gates[t * k + lane] = (!a.renorm ? my_s : sum == 0.0f ? 0.0f : my_s * (1.0f / sum)) * a.scale;
      if (balance) atomicAdd(&sh_counts[my_e], 1);
    }
    if (a.scores != nullptr) {
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (lane * C + c < E) a.scores[t * E + lane * C + c] = s[c] * inv;
    }
    if (balance) {
      float q = inv;
      if (a.router == 1) {
        float total = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) total += lane * C + c < E ? s[c] : 0.0f;
        total = warp_sum(total);
        q = total == 0.0f ? 0.0f : 1.0f / total;
      }
#pragma unroll
      for (int c = 0; c < C; ++c) acc[c] = fmaf(s[c], q, acc[c]);
    }
  }
  if (!balance) return;

#pragma unroll
  for (int c = 0; c < C; ++c)
    if (lane * C + c < E) my_row[lane * C + c] = acc[c];
  __syncthreads();
  finish_balance(a, sh_counts, [&](int e) {
    float p = 0.0f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) p += sh[w * E + e];
    return p;
  });
}

// ----------------------------------------------------------------------------- backward
// With dg the gates' gradient and S the sum of the selected scores:
//   ds_j = scale (dg_j - sum_i dg_i s_i / S) / S (renormalised) or scale dg_j
//   sigmoid: dl = (ds + (dprob - sum_e q dprob) / sum_e s) s (1 - s), q = s / sum_e s
//   softmax: dl = p (D - sum_e p D), D = ds + dprob
// The dense row is stored first; then lane j stores the entry of the j-th selected expert over it.
// sigmoid's value and derivative, both without cancellation
__device__ __forceinline__ void sigmoid_and_slope(float x, float& s, float& slope) {  // s may be x itself
  const float e = expf(-fabsf(x)), f = 1.0f / (1.0f + e);
  s = x >= 0.0f ? f : e * f;
  slope = e * f * f;
}

// LANES lanes to a token (8 up to 256 experts, 16 up to 512, 32), 32 / LANES tokens to a warp; a row is read and written
// in words of 4 experts, lane p the words p, p + LANES, ..., so that a warp's accesses are whole 128-byte (bf16:
// 64-byte) pieces of its rows and the sums over a token take 3 to 5 exchanges for all its tokens at once; rows that
// are not aligned are read and written one expert at a time (222 experts, 65,536 tokens: 33 us; 256: 28).
// 65,536 tokens of 160 experts, softmax: 17.7 us, 4.9 TB/s, bound by the latency of a warp's steps (exponentials and
// four sums over the lanes) that 16 to 24 warps an SM cover in 58% of the cycles; 4,096 tokens of 256: 3.7 us.
// Q: words of a lane.  DENSE: the row's scores are needed (softmax, or dprob); without it the row is zero but for the
// selected experts, whose logits alone are read.
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}
// The same by the hardware's exponential and reciprocal (off by 2^-22 and by 2^-24 |x|): 8 instructions instead of 22
// for the entries that only the balance term reaches.
__device__ __forceinline__ void sigmoid_and_slope_fast(float x, float& s, float& slope) {
  const float e = exp2_fast(fabsf(x) * -LOG2E), f = inverse_fast(1.0f + e);
  s = x >= 0.0f ? f : e * f;
  slope = e * f * f;
}

// Experts e .. e + 3 of a row that is not aligned, -inf beyond E.
template <typename TL>
__device__ __forceinline__ float4 load_word(const TL* row, int e, int E) {
  return make_float4(e < E ? to_f32(row[e]) : -INFINITY, e + 1 < E ? to_f32(row[e + 1]) : -INFINITY,
                     e + 2 < E ? to_f32(row[e + 2]) : -INFINITY, e + 3 < E ? to_f32(row[e + 3]) : -INFINITY);
}
template <typename TL>
__device__ __forceinline__ void store_word(TL* row, int e, int E, bool wide, float4 v) {
  if (wide) {
    if (e < E) store4(row + e, v);
  } else {
    if (e < E) from_f32(v.x, row + e);
    if (e + 1 < E) from_f32(v.y, row + e + 1);
    if (e + 2 < E) from_f32(v.z, row + e + 2);
    if (e + 3 < E) from_f32(v.w, row + e + 3);
  }
}
template <int LANES>
__device__ __forceinline__ float token_sum(float x) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) x += __shfl_xor_sync(ALL, x, o);
  return x;
}
// 4 experts as they lie in a row
template <typename TL>
struct Word {
  using type = uint4;
};
template <>
struct Word<__nv_bfloat16> {
  using type = uint2;
};
__device__ __forceinline__ float4 unpack_word(uint4 v) {
  return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}
__device__ __forceinline__ float4 unpack_word(uint2 v) {
  return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                     __uint_as_float(v.y & 0xffff0000u));
}

// Blocks on an SM, and for dense rows the grid: more of them, of which the last find a part of the SMs idle, cost up to
// 20%; with fewer registers for one more block 256 experts took 36 us instead of 27.
constexpr int backward_blocks(int Q, bool dense) { return !dense ? 4 : Q <= 5 ? 3 : 2; }

// Aligned rows come through shared memory, the next tokens' under the arithmetic of these (cp.async), and the
// selected logits are read from there: no load waits for another.
template <int LANES, int Q, typename TL, int ROUTER, bool DENSE>
__global__ void __launch_bounds__(THREADS, backward_blocks(Q, DENSE)) route_backward_kernel(const RouteBackwardArgs a) {
  constexpr int TOKENS = 32 / LANES, HELD = LANES == 8 ? 2 : 1;  // selected experts of a lane: at most 16 in all
  __shared__ float4 d[Q * LANES];
  using W = typename Word<TL>::type;
  extern __shared__ __align__(16) unsigned char ring_bytes[];  // DENSE, aligned: [WARPS][2][Q][32] words
  W* ring = reinterpret_cast<W*>(ring_bytes) + (threadIdx.x >> 5) * (2 * Q * 32);
  const bool ringed = DENSE && a.wide;
  const int lane = threadIdx.x & 31, row = lane / LANES, part = lane % LANES;
  const int E = a.E, k = a.k;
  if (DENSE) {
    for (int e = threadIdx.x; e < Q * LANES * 4; e += THREADS)
      reinterpret_cast<float*>(d)[e] = a.dprob != nullptr && e < E ? a.dprob[e] : 0.0f;
    __syncthreads();
  }
  const int64_t step = (int64_t)gridDim.x * WARPS * TOKENS;
  int64_t base = ((int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5)) * TOKENS;
  const TL* logits = static_cast<const TL*>(a.logits);
  auto token = [&](int64_t first) { return min(first + row, a.T - 1); };
  auto fetch = [&](int64_t first, int stage) {
    if (ringed && first < a.T) {
      const TL* from = logits + token(first) * a.stride;
      const uint32_t to = (uint32_t)__cvta_generic_to_shared(ring + stage * (Q * 32) + lane);
#pragma unroll
      for (int i = 0; i < Q; ++i) {
        const int e = 4 * (part + LANES * i);
        if (e < E)
          asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to + i * 32 * (int)sizeof(W)), "l"(from + e),
                       "n"(sizeof(W))
                       : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // the selected experts, one or two to a lane, and their gates' gradients
  auto selected = [&](int64_t first, int (&e)[HELD], float (&dg)[HELD]) {
#pragma unroll
    for (int h = 0; h < HELD; ++h) {
      const int j = part + LANES * h;
      e[h] = -1, dg[h] = 0.0f;
      if (j < k && a.dgates != nullptr && first < a.T) {
        e[h] = a.topk_idx[token(first) * k + j];
        dg[h] = a.dgates[token(first) * k + j];
      }
    }
  };
  int e_next[HELD];
  float dg_next[HELD];
  fetch(base, 0);
  selected(base, e_next, dg_next);
  for (int stage = 0; base < a.T; base += step, stage ^= 1) {
    const bool on = base + row < a.T;
    const int64_t t = token(base);
    const TL* from = logits + t * a.stride;
    TL* out = static_cast<TL*>(a.dlogits) + t * a.out_stride;
    int e[HELD];
    float x[HELD], dg[HELD], dj[HELD];
#pragma unroll
    for (int h = 0; h < HELD; ++h) e[h] = e_next[h], dg[h] = dg_next[h], dj[h] = 0.0f;
    fetch(base + step, stage ^ 1);
    selected(base + step, e_next, dg_next);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncwarp();
    const W* words = ring + stage * (Q * 32);
    float4 s[Q];
    if (DENSE) {
#pragma unroll
      for (int i = 0; i < Q; ++i) {
        const int at = 4 * (part + LANES * i);
        if (ringed) s[i] = at < E ? unpack_word(words[i * 32 + lane]) : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        else s[i] = load_word(from, at, E);
      }
    }
#pragma unroll
    for (int h = 0; h < HELD; ++h) {
      x[h] = -INFINITY;
      if (part + LANES * h < k && a.dgates != nullptr) {
        if (e[h] < 0 || e[h] >= E) {
          report_status(a.status, MOK_DEV_INVALID_ROUTING, SITE_TOPK_INDEX);
          e[h] = -1, dg[h] = 0.0f;
        } else {
          const int q = e[h] >> 2;
          if (ringed)
            x[h] = to_f32(reinterpret_cast<const TL*>(words + q / LANES * 32 + row * LANES + q % LANES)[e[h] & 3]);
          else
            x[h] = to_f32(from[e[h]]);
          if (DENSE) dj[h] = reinterpret_cast<const float*>(d)[e[h]];
        }
      }
    }
    float shift = 0.0f, inv = 0.0f, sj[HELD], slope[HELD];
    if (ROUTER == 0) {
      shift = -INFINITY;
#pragma unroll
      for (int i = 0; i < Q; ++i) shift = fmaxf(fmaxf(shift, fmaxf(s[i].x, s[i].y)), fmaxf(s[i].z, s[i].w));
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) shift = fmaxf(shift, __shfl_xor_sync(ALL, shift, o));
      if (shift == -INFINITY) shift = 0.0f;
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < Q; ++i) {
        exp_pair(s[i].x, s[i].y, shift, s[i].x, s[i].y);
        exp_pair(s[i].z, s[i].w, shift, s[i].z, s[i].w);
        sum += (s[i].x + s[i].y) + (s[i].z + s[i].w);
      }
      sum = token_sum<LANES>(sum);
      inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
      for (int h = 0; h < HELD; ++h) sj[h] = e[h] >= 0 ? expf(x[h] - shift) * inv : 0.0f;
    } else {
#pragma unroll
      for (int h = 0; h < HELD; ++h) {
        sigmoid_and_slope(x[h], sj[h], slope[h]);
        if (e[h] < 0) sj[h] = slope[h] = 0.0f;
      }
    }
    float ds[HELD], of_lane = 0.0f;
#pragma unroll
    for (int h = 0; h < HELD; ++h) ds[h] = a.scale * dg[h], of_lane += sj[h];
    if (a.renorm) {
      const float S = token_sum<LANES>(of_lane);
      of_lane = 0.0f;
#pragma unroll
      for (int h = 0; h < HELD; ++h) of_lane = fmaf(dg[h], sj[h], of_lane);
      const float dot = token_sum<LANES>(of_lane);
      const float inv_s = S == 0.0f ? 0.0f : 1.0f / S;
#pragma unroll
      for (int h = 0; h < HELD; ++h) ds[h] = e[h] >= 0 ? a.scale * (dg[h] - dot * inv_s) * inv_s : 0.0f;
    }
    float dot = 0.0f;
    if (ROUTER == 0) {
#pragma unroll
      for (int i = 0; i < Q; ++i) {
        const float4 di = d[part + LANES * i];
        s[i].x *= inv, s[i].y *= inv, s[i].z *= inv, s[i].w *= inv;
        dot = fmaf(s[i].x, di.x, fmaf(s[i].y, di.y, fmaf(s[i].z, di.z, fmaf(s[i].w, di.w, dot))));
      }
#pragma unroll
      for (int h = 0; h < HELD; ++h) dot = fmaf(sj[h], ds[h], dot);
      dot = token_sum<LANES>(dot);
    } else if (DENSE) {
      float total = 0.0f;
#pragma unroll
      for (int i = 0; i < Q; ++i) {  // the slopes in place of the logits
        const float4 di = d[part + LANES * i];
        float4 v;
        sigmoid_and_slope_fast(s[i].x, v.x, s[i].x);
        sigmoid_and_slope_fast(s[i].y, v.y, s[i].y);
        sigmoid_and_slope_fast(s[i].z, v.z, s[i].z);
        sigmoid_and_slope_fast(s[i].w, v.w, s[i].w);
        total += (v.x + v.y) + (v.z + v.w);
        dot = fmaf(v.x, di.x, fmaf(v.y, di.y, fmaf(v.z, di.z, fmaf(v.w, di.w, dot))));
      }
      total = token_sum<LANES>(total);
      inv = total == 0.0f ? 0.0f : 1.0f / total;
      dot = token_sum<LANES>(dot) * inv;
    }
    if (on) {
#pragma unroll
      for (int i = 0; i < Q; ++i) {
        const int q = part + LANES * i;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (DENSE) {
          const float4 di = d[q];
          const float f = ROUTER == 0 ? 1.0f : inv;
          v = make_float4(s[i].x * ((di.x - dot) * f), s[i].y * ((di.y - dot) * f), s[i].z * ((di.z - dot) * f),
                          s[i].w * ((di.w - dot) * f));
        }
        store_word(out, 4 * q, E, a.wide, v);
      }
    }
    __syncwarp();  // the selected entries go over the row's
#pragma unroll
    for (int h = 0; h < HELD; ++h) {
      if (on && e[h] >= 0)
        from_f32(ROUTER == 0 ? sj[h] * (dj[h] + ds[h] - dot) : (ds[h] + (dj[h] - dot) * inv) * slope[h], out + e[h]);
    }
    // (the barrier above also frees this stage: every lane has read it)
  }
}

template <int LANES, int Q, typename TL>
cudaError_t launch_backward(const RouteBackwardArgs& a, int n_sm, cudaStream_t st) {
  auto kernel = route_backward_kernel<LANES, Q, TL, 1, false>;
  if (a.router == 0) kernel = route_backward_kernel<LANES, Q, TL, 0, true>;
  else if (a.dprob != nullptr) kernel = route_backward_kernel<LANES, Q, TL, 1, true>;
  const bool dense = a.router == 0 || a.dprob != nullptr;
  const int smem = dense && a.wide ? WARPS * 2 * Q * 32 * 4 * (int)sizeof(TL) : 0;
  if (smem > 40 * 1024) {
    const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
  }
  constexpr int TOKENS = 32 / LANES * WARPS;  // of a block
  const int64_t want = (a.T + TOKENS - 1) / TOKENS;
  const int most = dense ? backward_blocks(Q, true) : 8;
  kernel<<<(int)std::min<int64_t>(want, most * n_sm), THREADS, smem, st>>>(a);
  return cudaGetLastError();
}
template <typename TL>
cudaError_t launch_backward(const RouteBackwardArgs& args, int n_sm, cudaStream_t st) {
  RouteBackwardArgs a = args;
  const size_t unit = 4 * sizeof(TL);
  a.wide = a.E % 4 == 0 && a.stride % 4 == 0 && a.out_stride % 4 == 0 &&
           reinterpret_cast<uintptr_t>(a.logits) % unit == 0 && reinterpret_cast<uintptr_t>(a.dlogits) % unit == 0;
  const int q = (a.E + 31) / 32;  // words of 8 lanes
  if (q <= 1) return launch_backward<8, 1, TL>(a, n_sm, st);
  if (q <= 2) return launch_backward<8, 2, TL>(a, n_sm, st);
  if (q <= 4) return launch_backward<8, 4, TL>(a, n_sm, st);
  if (q <= 5) return launch_backward<8, 5, TL>(a, n_sm, st);
  if (q <= 6) return launch_backward<8, 6, TL>(a, n_sm, st);
  if (q <= 8) return launch_backward<8, 8, TL>(a, n_sm, st);
  if (q <= 12) return launch_backward<16, 6, TL>(a, n_sm, st);
  if (q <= 16) return launch_backward<16, 8, TL>(a, n_sm, st);
  return launch_backward<32, 8, TL>(a, n_sm, st);
}

template <int C, typename TL>
cudaError_t launch_route_c(const RouteArgs& a, int n_sm, cudaStream_t st) {
  const int64_t want = (a.T + WARPS - 1) / WARPS;
  const int blocks = (int)(want < 1 ? 1 : want > 6 * n_sm ? 6 * n_sm : want);
  route_kernel<C, TL><<<blocks, THREADS, (WARPS + 1) * a.E * 4, st>>>(a);
  return cudaGetLastError();
}
}  // namespace

// C experts to a lane: the least there is a kernel for.  3, 5, 6 and 12 keep groups whole lanes at 96, 160, 192
// and 384 experts.
#define ROUTE_BY_C(fn, TL)            \
  do {                                \
    const int c = (a.E + 31) / 32;    \
    if (c <= 1) return fn<1, TL>(a, n_sm, st);   \
    if (c <= 2) return fn<2, TL>(a, n_sm, st);   \
    if (c <= 3) return fn<3, TL>(a, n_sm, st);   \
    if (c <= 4) return fn<4, TL>(a, n_sm, st);   \
    if (c <= 5) return fn<5, TL>(a, n_sm, st);   \
    if (c <= 6) return fn<6, TL>(a, n_sm, st);   \
    if (c <= 8) return fn<8, TL>(a, n_sm, st);   \
    if (c <= 12) return fn<12, TL>(a, n_sm, st); \
    if (c <= 16) return fn<16, TL>(a, n_sm, st); \
    return fn<32, TL>(a, n_sm, st);   \
  } while (0)

// For many tokens, two of them to a warp: that kernel's steps for a token hardly grow with its experts, this one's do,
// and a call needs tokens for all its warps.  Microseconds here and there, f32 logits, sigmoid with a bias, k = 8 in
// 4 of 8 groups: 256 experts, 1024 tokens 4.5 and 4.8, 2048 tokens 5.8 and 4.9, 4096 tokens 9.7 and 6.0, 65536
// tokens 97 and 37; 128 experts, 4096 tokens 5.9 and 5.5, 65536 tokens 60 and 29; ungrouped: 384 experts, 1024 tokens
// 5.2 and 4.7, 4096 tokens 12.0 and 8.0; 64 experts, 4096 tokens 4.0 and 4.8, 16384 tokens 11.0 and 10.3, 65536
// tokens 33 and 23; 32 experts, 16384 tokens 6.8 and 8.7, 65536 tokens 21 and 20.
cudaError_t launch_route(const RouteArgs& a, bool bf16, int n_sm, cudaStream_t st) {
  if (a.T * a.E * a.E >= int64_t{3} << 25 && route_pairs_fit(a)) return launch_route_pairs(a, bf16, n_sm, st);
  if (bf16) ROUTE_BY_C(launch_route_c, __nv_bfloat16);
  ROUTE_BY_C(launch_route_c, float);
}

cudaError_t launch_route_backward(const RouteBackwardArgs& a, bool bf16, int n_sm, cudaStream_t st) {
  return bf16 ? launch_backward<__nv_bfloat16>(a, n_sm, st) : launch_backward<float>(a, n_sm, st);
}

}  // namespace mok
