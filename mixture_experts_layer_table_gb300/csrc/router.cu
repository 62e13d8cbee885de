// Group-limited expert selection from router logits, with the load-balancing outputs, and its backward.
//
// One warp takes one token at a time; lane l holds the C consecutive experts from l * C on, C = ceil(E / 32)
// rounded up to a size there is a kernel for.  With s the scores (sigmoid, or softmax over the experts):
//   rank value r = s + bias; a softmax without a bias is ranked by its logits (it is increasing, and the logits
//   have no rounding of the sum in them).  A logit of -inf or NaN ranks behind every other.
//   group value: the largest r of the group, or the sum of its two largest (of e^(x - max) for the softmax
//   without a bias); the topk_group best groups stay, then the k best experts in them; ties to the lower index.
//   gate = scale * s, or scale * s / (the sum of the k selected s), 0 where that sum is 0.
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
template <int C, typename TL>
__global__ void __launch_bounds__(THREADS) route_backward_kernel(const RouteBackwardArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = a.E, k = a.k;
  float d[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int e = lane * C + c;
    d[c] = a.dprob != nullptr && e < E ? a.dprob[e] : 0.0f;
  }
  for (int64_t t = (int64_t)blockIdx.x * WARPS + warp; t < a.T; t += (int64_t)gridDim.x * WARPS) {
    const TL* row = static_cast<const TL*>(a.logits) + t * a.stride;
    TL* out = static_cast<TL*>(a.dlogits) + t * a.out_stride;
    float s[C];
    load_row<C>(row, lane, E, s);
    // the selected experts, one to a lane
    int e = -1;
    float xj = -INFINITY, dg = 0.0f, dj = 0.0f;
    if (lane < k && a.dgates != nullptr) {
      e = a.topk_idx[t * k + lane];
      if (e < 0 || e >= E) {
        report_status(a.status, MOK_DEV_INVALID_ROUTING, SITE_TOPK_INDEX);
        e = -1;
      } else {
        xj = to_f32(row[e]);
        dg = a.dgates[t * k + lane];
        dj = a.dprob != nullptr ? a.dprob[e] : 0.0f;
      }
    }
    float sj, inv = 1.0f;
    if (a.router == 0) {
      float m;
      inv = softmax_row<C>(s, &m);
      sj = e >= 0 ? expf(xj - m) * inv : 0.0f;
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c) s[c] = lane * C + c < E ? sigmoid(s[c]) : 0.0f;
      sj = e >= 0 ? sigmoid(xj) : 0.0f;
    }
    float ds = e >= 0 ? a.scale * dg : 0.0f;
    if (a.renorm) {
      const float S = warp_sum(sj), dot = warp_sum(dg * sj);
      ds = e < 0 || S == 0.0f ? 0.0f : a.scale * (dg - dot / S) / S;
    }
    if (a.router == 0) {
      float dot = 0.0f;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        s[c] *= inv;
        dot = fmaf(s[c], d[c], dot);
      }
      dot = warp_sum(fmaf(sj, ds, dot));
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (lane * C + c < E) from_f32(s[c] * (d[c] - dot), out + lane * C + c);
      __syncwarp();
      if (e >= 0) from_f32(sj * (dj + ds - dot), out + e);
    } else {
      float total = 0.0f, dot = 0.0f;
      if (a.dprob != nullptr) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
          total += s[c];
          dot = fmaf(s[c], d[c], dot);
        }
        total = warp_sum(total);
        dot = warp_sum(dot);
        inv = total == 0.0f ? 0.0f : 1.0f / total;
        dot *= inv;
      } else {
        inv = 0.0f;
      }
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (lane * C + c < E) from_f32((d[c] - dot) * inv * s[c] * (1.0f - s[c]), out + lane * C + c);
      __syncwarp();
      if (e >= 0) from_f32((ds + (dj - dot) * inv) * sj * (1.0f - sj), out + e);
    }
  }
}

template <int C, typename TL>
cudaError_t launch_route_c(const RouteArgs& a, int n_sm, cudaStream_t st) {
  const int64_t want = (a.T + WARPS - 1) / WARPS;
  const int blocks = (int)(want < 1 ? 1 : want > 6 * n_sm ? 6 * n_sm : want);
  route_kernel<C, TL><<<blocks, THREADS, (WARPS + 1) * a.E * 4, st>>>(a);
  return cudaGetLastError();
}
template <int C, typename TL>
cudaError_t launch_route_backward_c(const RouteBackwardArgs& a, int n_sm, cudaStream_t st) {
  const int64_t want = (a.T + WARPS - 1) / WARPS;
  const int blocks = (int)(want > 6 * n_sm ? 6 * n_sm : want);
  route_backward_kernel<C, TL><<<blocks, THREADS, 0, st>>>(a);
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

// Two tokens to a warp from 2048 tokens on: 256 experts in 8 groups, without balance: 1024 tokens 4.7 us here and 4.9
// there, 4096 tokens 9.7 and 7.4, 65536 tokens 95 and 42.
cudaError_t launch_route(const RouteArgs& a, bool bf16, int n_sm, cudaStream_t st) {
  if (a.T >= 2048 && route_pairs_fit(a)) return launch_route_pairs(a, bf16, n_sm, st);
  if (bf16) ROUTE_BY_C(launch_route_c, __nv_bfloat16);
  ROUTE_BY_C(launch_route_c, float);
}

cudaError_t launch_route_backward(const RouteBackwardArgs& a, bool bf16, int n_sm, cudaStream_t st) {
  if (bf16) ROUTE_BY_C(launch_route_backward_c, __nv_bfloat16);
  ROUTE_BY_C(launch_route_backward_c, float);
}

}  // namespace mok
