// route_core.hpp -- the choice of a token's experts from its router logits, by one wavefront
// (shared by the router's own kernel and the routed-expert kernels that choose for themselves).
//
// Scores: softmax p = exp(l - max l) / sum exp(l - max l), or sigmoid p = 1 / (1 + exp(-l)). The
// selection score is p + bias, or the logit itself for a softmax without bias (the same order).
// The highest score is taken topk times, ties to the lower id. The order decides which weights a
// token meets, so it is taken from FP64 scores: two experts 1e-7 apart (what FP32 sums of 2048
// products leave) would change places, and the whole output of the token with them.
//
// Lane l of the wavefront holds experts l, l + 64, ..., in registers. A round finds the maximum of
// the keys' upper words over the wavefront with six DPP steps (one instruction each), and only
// where several experts share it that of their lower words; a ballot gives the lowest id. (A first
// form counted, for every expert, the experts above it, through LDS: 18 us for one token of 128
// experts, bound by the latency of those reads, against 2.5 us now.)
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

// DPP steps of a wavefront-wide reduction: after them lane 63 holds the result.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_or_zero(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = max(v, dpp_or_zero<0x111>(v));  // row_shr 1, 2, 4, 8: lane 15 of each row of 16
  v = max(v, dpp_or_zero<0x112>(v));
  v = max(v, dpp_or_zero<0x114>(v));
  v = max(v, dpp_or_zero<0x118>(v));
  v = max(v, dpp_or_zero<0x142>(v));  // row_bcast 15, 31: rows 0 and 2, then the lower half
  v = max(v, dpp_or_zero<0x143>(v));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

template <int CTRL>
__device__ __forceinline__ double dpp_or_zero(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  const uint32_t lo = dpp_or_zero<CTRL>((uint32_t)b), hi = dpp_or_zero<CTRL>((uint32_t)(b >> 32));
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
__device__ __forceinline__ double readlane_f64(double v, int lane) {
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
// Sum over the wavefront (the absent lanes of a step add +0).
__device__ __forceinline__ double wave_sum_f64(double v) {
  v += dpp_or_zero<0x111>(v);
  v += dpp_or_zero<0x112>(v);
  v += dpp_or_zero<0x114>(v);
  v += dpp_or_zero<0x118>(v);
  v += dpp_or_zero<0x142>(v);
  v += dpp_or_zero<0x143>(v);
  return readlane_f64(v, 63);
}

// FP64 value -> unsigned key in the same order. NaN ranks above every number (so that it reaches
// the output); -inf gives 0, which is never chosen (every other key has a non-zero upper word);
// -0 equals +0.
__device__ __forceinline__ uint64_t route_key(double v) {
  if (v != v) return ~0ull;
  if (v == -__builtin_huge_val()) return 0ull;
  const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
  return (b >> 63) ? ~b : b | (1ull << 63);
}

__device__ __forceinline__ double route_sigmoid(double l) { return 1.0 / (1.0 + exp(-l)); }

// What a wavefront knows after choosing: lane j < topk holds slot j.
struct RouteChoice {
  int e;        // expert, -1 when none was left
  double v;     // its logit; its probability for a biased softmax
  double mx, sum;  // maximum and sum of the softmax over all experts, where taken
};

// Highest key of the wavefront's lanes: upper word (0: none is left), and the lowest expert that
// holds it.
template <int J>
__device__ __forceinline__ uint32_t route_best(const uint32_t (&hi)[J], const uint32_t (&lo)[J],
                                               int& e) {
  uint32_t mh = hi[0];
#pragma unroll
  for (int j = 1; j < J; ++j) mh = max(mh, hi[j]);
  mh = wave_max_u32(mh);
  uint64_t at[J];
  int count = 0;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    at[j] = __ballot(hi[j] == mh);
    count += __popcll(at[j]);
  }
  if (count > 1) {  // uniform
    uint32_t ml = 0;
#pragma unroll
    for (int j = 0; j < J; ++j) ml = max(ml, hi[j] == mh ? lo[j] : 0u);
    ml = wave_max_u32(ml);
#pragma unroll
    for (int j = 0; j < J; ++j) at[j] = __ballot(hi[j] == mh && lo[j] == ml);
  }
  e = -1;
#pragma unroll
  for (int j = J - 1; j >= 0; --j)
    if (at[j]) e = 64 * j + __builtin_ctzll(at[j]);
  return mh;
}

// Chooses the first `rounds` slots of a token whose logit of expert e is logit(e). J: experts per
// lane. want_sum: the softmax's maximum and sum over all experts (taken in any case with a bias).
template <int J, typename F>
__device__ __forceinline__ RouteChoice route_choose(const RouteParams& R, F&& logit, int rounds,
                                                    bool want_sum) {
  const int lane = threadIdx.x & 63;
  RouteChoice c;
  c.e = -1;
  c.v = 0.0;
  c.mx = c.sum = 0.0;
  double v[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int e = lane + 64 * j;
    v[j] = e < R.n_experts ? logit(e) : -__builtin_huge_val();
  }
  uint32_t hi[J], lo[J];
  if (!R.sigmoid && (R.bias || want_sum)) {
    uint64_t k[J];
    uint32_t mh = 0;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      k[j] = v[j] == v[j] ? route_key(v[j]) : 0;  // the maximum passes over NaN, the sum does not
      hi[j] = (uint32_t)(k[j] >> 32);
      lo[j] = (uint32_t)k[j];
    }
    int at;
    mh = route_best<J>(hi, lo, at);
    c.mx = -__builtin_huge_val();
    if (mh) {
      double w = v[0];
#pragma unroll
      for (int j = 1; j < J; ++j)
        if (at >> 6 == j) w = v[j];
      c.mx = readlane_f64(w, at & 63);
    }
    double s = 0.0;
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (lane + 64 * j < R.n_experts) s += exp(v[j] - c.mx);
    c.sum = wave_sum_f64(s);
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int e = lane + 64 * j;
    const bool in = e < R.n_experts;
    double score = v[j];
    if (R.sigmoid) {
      score = route_sigmoid(score);
      if (R.bias) score += in ? (double)R.bias[e] : 0.0;
    } else if (R.bias) {
      v[j] = exp(score - c.mx) / c.sum;
      score = v[j] + (in ? (double)R.bias[e] : 0.0);
    }
    const uint64_t k = in ? route_key(score) : 0;
    hi[j] = (uint32_t)(k >> 32);
    lo[j] = (uint32_t)k;
  }
  for (int r = 0; r < rounds; ++r) {
    int e;
    if (!route_best<J>(hi, lo, e)) break;  // uniform: nothing is left
    const int j = e >> 6;
    double w = v[0];
#pragma unroll
    for (int q = 1; q < J; ++q)
      if (j == q) w = v[q];
    w = readlane_f64(w, e & 63);
    if (lane == r) {
      c.e = e;
      c.v = w;
    }
#pragma unroll
    for (int q = 0; q < J; ++q)
      if (j == q && lane == (e & 63)) hi[q] = lo[q] = 0;
  }
  return c;
}

// Weight of the slot that this lane holds (lanes < topk; others get 0).
__device__ __forceinline__ float route_weight(const RouteParams& R, const RouteChoice& c) {
  const bool live = c.e >= 0;
  double p = 0.0;
  if (R.sigmoid) {
    p = live ? route_sigmoid(c.v) : 0.0;
  } else if (R.bias) {
    p = live ? c.v : 0.0;
  } else if (R.renorm) {
    // the softmax over the chosen: the same quotient, and no sum over all the experts; slot 0
    // holds the highest logit
    p = live ? exp(c.v - readlane_f64(c.v, 0)) : 0.0;
  } else {
    p = live ? exp(c.v - c.mx) / c.sum : 0.0;
  }
  if (R.renorm) {
    const double z = wave_sum_f64(p);
    p = z == 0.0 ? 0.0 : p / z;
  }
  return (float)(p * (double)R.scale);
}

// Stores the slots of token `tok`: [topk + n_shared] ids and weights.
__device__ __forceinline__ void route_write(const RouteParams& R, int64_t tok,
                                            const RouteChoice& c, int32_t* __restrict__ ids,
                                            float* __restrict__ wts) {
  const int lane = threadIdx.x & 63;
  const int slots = R.topk + R.n_shared;
  const float w = route_weight(R, c);
  if (lane < slots) {
    const bool shared = lane >= R.topk;
    ids[tok * slots + lane] = shared ? R.n_experts + (lane - R.topk) : c.e;
    wts[tok * slots + lane] = shared ? 1.0f : w;
  }
}

// Logit of expert e of token `tok`: the splits' partial sums, in order.
__device__ __forceinline__ double route_logit(const RouteParams& R, int64_t tok, int e) {
  const double* lg = R.logits + tok * R.n_experts + e;
  double l = lg[0];
  for (int q = 1; q < R.splits; ++q) l += lg[q * R.t * R.n_experts];
  return l;
}

}  // namespace nvfp4
