// Arguments and launchers of the group-limited router kernels (internal to the library).
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace mok {

struct RouteArgs {
  const void* logits;      // f32 or bf16 rows of E, `stride` elements apart
  const float* bias;       // [E] or null
  int64_t T, stride;
  int E, k, router, renorm;
  float scale;
  int n_group, topk_group, group_top2;
  int32_t* topk_idx;       // [T][k]
  float* gates;            // [T][k] or null
  float* scores;           // [T][E] or null
  // load balancing: null unless wanted (sums needs acc)
  int32_t* counts;
  float* prob_sum;
  float* loss;
  float* dprob;
  float* bias_next;
  float dprob_unit;        // dprob[e] = dprob_unit * counts[e]
  float bias_rate;
  int sum_shift;           // probabilities are summed in units of 2^-sum_shift
  // set by the launcher: rows can be read, scores can be written in words of 8 or 16 bytes; tokens whose gates are
  // formed together; log2 of the next power of two of k; experts of a group and their inverse, log2 of its lanes;
  // lanes of a segment
  bool words, wide_scores;
  int batch, slot_bits, group_size, group_lane_bits, segment_lanes;
  float inv_group_size;
  unsigned* ticket;        // workspace: zero between calls
  unsigned* not_finite;
  unsigned long long* acc_prob;  // [ROUTE_COPIES][ROUTE_MAX_E]
  int32_t* acc_counts;
};

struct RouteBackwardArgs {
  const void* logits;
  int64_t T, stride, out_stride;
  int E, k, router, renorm;
  float scale;
  const int32_t* topk_idx;  // [T][k]
  const float* dgates;      // [T][k] or null
  const float* dprob;       // [E] or null
  void* dlogits;            // the logits' type
  int* status;              // or null
  bool wide;                // set by the launcher: rows can be read and written 4 experts at a time
};

constexpr int ROUTE_MAX_E = 1024;
constexpr int ROUTE_MAX_K = 16;
constexpr int ROUTE_MAX_GROUPS = 32;
// workspace: ticket and flag (256 bytes), then copies of u64 [1024] probability sums and of i32 [1024] counts; blocks
// add to them in turn (to one copy, 256 blocks' adds to the same 16 lines took 3 us of 13)
constexpr int ROUTE_COPIES = 8;
constexpr int ROUTE_WS_SUMS = 256;
constexpr int ROUTE_WS_COUNTS = ROUTE_WS_SUMS + ROUTE_COPIES * 8 * ROUTE_MAX_E;
constexpr int ROUTE_WS_BYTES = ROUTE_WS_COUNTS + ROUTE_COPIES * 4 * ROUTE_MAX_E;

inline bool route_balances(const RouteArgs& a) { return a.counts || a.prob_sum || a.loss || a.dprob || a.bias_next; }

// Two tokens to a warp, for many tokens (router_pairs.cu); launch_route chooses.
bool route_pairs_fit(const RouteArgs& a);
cudaError_t launch_route_pairs(const RouteArgs& a, bool bf16, int n_sm, cudaStream_t st);
cudaError_t launch_route(const RouteArgs& a, bool bf16, int n_sm, cudaStream_t st);
cudaError_t launch_route_backward(const RouteBackwardArgs& a, bool bf16, int n_sm, cudaStream_t st);

}  // namespace mok
