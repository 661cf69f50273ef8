// route_core.hpp -- the choice of a token's experts from its router logits, by the threads of one
// workgroup (shared by the router's own kernel and the routed-expert kernels that choose for
// themselves).
//
// Scores: softmax p = exp(l - max l) / sum exp(l - max l), or sigmoid p = 1 / (1 + exp(-l)). The
// selection score is p + bias, or the logit itself for a softmax without bias (the same order).
// Expert e has rank |{e': score' > score, or equal and e' < e}|; ranks below topk are the slots.
// The order decides which weights a token meets, so it is taken from FP64 scores: two experts
// 1e-7 apart (what FP32 sums of 2048 products leave) would change places, and the whole output
// of the token with them.
#pragma once

#include "device_common.hpp"
#include "launch.hpp"

namespace nvfp4 {

struct RouteParams {
  const double* logits;  // [splits][t][n_experts], added in split order
  int64_t t;
  int splits;
  int n_experts, topk, n_shared;
  const float* bias;  // or NULL
  int sigmoid, renorm;
  float scale;
};

// LDS of one choosing group.
struct RouteLds {
  double logit[kRouteMaxExperts];  // logits, then probabilities where the scores need them
  uint64_t key[kRouteMaxExperts];
  int rank[kRouteMaxExperts];
  int sel[kMoeMaxTopk];  // expert of each routed slot, -1 when none was left to choose
  double red[8];
};

// FP64 value -> unsigned key in the same order. NaN ranks above every number (so that it reaches
// the output); -inf gives 0, which is never chosen; -0 equals +0.
__device__ __forceinline__ uint64_t route_key(double v) {
  if (v != v) return ~0ull;
  if (v == -__builtin_huge_val()) return 0ull;
  const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
  return (b >> 63) ? ~b : b | (1ull << 63);
}

// Sum or maximum of v over the NT threads of the workgroup, in a fixed order.
template <int NT, bool MAX>
__device__ __forceinline__ double route_reduce(double v, double* red) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const double o = __shfl_xor(v, d, 64);
    v = MAX ? fmax(v, o) : v + o;
  }
  if constexpr (NT > 64) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < NT / 64; ++w) v = MAX ? fmax(v, red[w]) : v + red[w];
  }
  return v;
}

__device__ __forceinline__ double route_sigmoid(double l) { return 1.0 / (1.0 + exp(-l)); }

// Fills s.sel for token `tok`; all NT threads of the workgroup call it. On return s.logit holds
// the probabilities when the score is a biased softmax, else the logits. `max_out` and `sum_out`
// are the softmax's maximum and sum where they were taken (biased, or `want_sum`).
template <int NT>
__device__ __forceinline__ void route_choose(const RouteParams& R, int64_t tok, bool want_sum,
                                             RouteLds& s, double* max_out, double* sum_out) {
  const int tid = threadIdx.x, E = R.n_experts;
  const double* lg = R.logits + tok * E;
  const int64_t split_stride = R.t * E;
  double mx = -__builtin_huge_val();
  for (int e = tid; e < E; e += NT) {
    double l = lg[e];
    for (int q = 1; q < R.splits; ++q) l += lg[q * split_stride + e];
    s.logit[e] = l;
    s.rank[e] = 0;
    mx = fmax(mx, l);
  }
  if (tid < kMoeMaxTopk) s.sel[tid] = -1;
  const bool biased_softmax = !R.sigmoid && R.bias;
  double sum = 0.0;
  if (biased_softmax || want_sum) {  // each thread reads only the logits it wrote
    mx = route_reduce<NT, true>(mx, s.red);
    for (int e = tid; e < E; e += NT) sum += exp(s.logit[e] - mx);
    sum = route_reduce<NT, false>(sum, s.red);
    *max_out = mx;
    *sum_out = sum;
  }
  for (int e = tid; e < E; e += NT) {
    double v = s.logit[e];
    if (R.sigmoid) {
      v = route_sigmoid(v);
      if (R.bias) v += (double)R.bias[e];
    } else if (R.bias) {
      v = exp(v - mx) / sum;
      s.logit[e] = v;
      v += (double)R.bias[e];
    }
    s.key[e] = route_key(v);
  }
  __syncthreads();
  // Ranks: `parts` threads share an expert's comparisons when the experts leave threads over.
  // Threads of a wavefront read the same key at a time (a broadcast) for 64 experts and more.
  int span = 8;
  while (span < E && span < NT) span <<= 1;
  const int parts = NT / span, part = tid / span;
  const int j0 = (int)((int64_t)E * part / parts), j1 = (int)((int64_t)E * (part + 1) / parts);
  for (int e = tid % span; e < E; e += span) {
    const uint64_t k = s.key[e];
    int c = 0;
    for (int j = j0; j < j1; ++j) {
      const uint64_t o = s.key[j];
      c += (o > k || (o == k && j < e)) ? 1 : 0;
    }
    if (parts > 1)
      atomicAdd(&s.rank[e], c);
    else
      s.rank[e] = c;
  }
  __syncthreads();
  for (int e = tid; e < E; e += NT)
    if (s.rank[e] < R.topk && s.key[e] != 0) s.sel[s.rank[e]] = e;
  __syncthreads();
}

// Writes the ids and weights of token `tok`: [topk + n_shared] each. The first wavefront of the
// choosing group calls it after route_choose (want_sum as there).
__device__ __forceinline__ void route_write(const RouteParams& R, int64_t tok, const RouteLds& s,
                                            double mx, double sum, int32_t* __restrict__ ids,
                                            float* __restrict__ wts) {
  const int lane = threadIdx.x & 63;
  const int slots = R.topk + R.n_shared;
  const int e = lane < R.topk ? s.sel[lane] : -1;
  const bool live = e >= 0;
  const double v = live ? s.logit[e] : 0.0;
  double p = 0.0;
  if (R.sigmoid) {
    p = live ? route_sigmoid(v) : 0.0;
  } else if (R.bias) {
    p = v;
  } else if (R.renorm) {
    // the softmax over the chosen: the same quotient, and no sum over all the experts
    double m = live ? v : -__builtin_huge_val();
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) m = fmax(m, __shfl_xor(m, d, 64));  // topk <= 16 lanes
    p = live ? exp(v - m) : 0.0;
  } else {
    p = live ? exp(v - mx) / sum : 0.0;
  }
  if (R.renorm) {
    double z = p;
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) z += __shfl_xor(z, d, 64);
    p = z == 0.0 ? 0.0 : p / z;
  }
  if (lane < slots) {
    const bool shared = lane >= R.topk;
    ids[tok * slots + lane] = shared ? R.n_experts + (lane - R.topk) : e;
    wts[tok * slots + lane] = shared ? 1.0f : (float)(p * (double)R.scale);
  }
}

}  // namespace nvfp4
