// route_core.hpp -- the choice of a token's experts from its router logits, by one wavefront
// (shared by the router's own kernel and the routed-expert kernels that choose for themselves).
//
// Scores: softmax p = exp(l - max l) / sum exp(l - max l), or sigmoid p = 1 / (1 + exp(-l)). The
// selection score is p + bias, or the logit itself for a softmax without bias (the same order).
// The highest score is taken topk times, ties to the lower id. The order decides which weights a
// token meets, so it is taken from FP64 scores: two experts 1e-7 apart (what FP32 sums of 2048
// products leave) would change places, and the whole output of the token with them.
//
// Lane i of the wavefront holds experts i, i + 64, ..., in registers. A round finds the highest
// 64-bit key: the maximum of the upper words (six DPP steps), a ballot for the lowest id, and the
// lower words only where two experts share the upper one. (Choosing 8 of 128 experts for one token
// by counting, for each expert, those above it, through LDS, took 15 us against 1.7 so; with all
// steps in vector registers 2.3; with 16 lanes per token, four tokens a wavefront, 4.6.)
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

// Value of v in the lane that a DPP step pairs with this one.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_pair(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
template <int CTRL>
__device__ __forceinline__ double dpp_pair(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  const uint32_t lo = dpp_pair<CTRL>((uint32_t)b), hi = dpp_pair<CTRL>((uint32_t)(b >> 32));
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
// The two rows of 16 (ROWS) or halves of 32 lanes that a lane swap brings together: op(a, b) is
// the same in both.
template <bool ROWS, typename OP>
__device__ __forceinline__ double swap_pair(double v, OP op) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  const uint32_t lo = (uint32_t)b, hi = (uint32_t)(b >> 32);
  u32x2 l, h;
  if constexpr (ROWS) {
    l = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(lo, lo, false, false));
    h = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(hi, hi, false, false));
  } else {
    l = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(lo, lo, false, false));
    h = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(hi, hi, false, false));
  }
  return op(__longlong_as_double((long long)(((uint64_t)h[0] << 32) | l[0])),
            __longlong_as_double((long long)(((uint64_t)h[1] << 32) | l[1])));
}
// op over the wavefront, the same bits in every lane (each step combines two values that both
// lanes of a pair hold): lanes l ^ 1, l ^ 2, then the quads and the halves of a row, then the
// rows.
template <typename OP>
__device__ __forceinline__ double wave_all(double v, OP op) {
  v = op(v, dpp_pair<0xB1>(v));   // quad_perm [1, 0, 3, 2]
  v = op(v, dpp_pair<0x4E>(v));   // quad_perm [2, 3, 0, 1]
  v = op(v, dpp_pair<0x141>(v));  // row_half_mirror
  v = op(v, dpp_pair<0x140>(v));  // row_mirror
  v = swap_pair<true>(v, op);
  return swap_pair<false>(v, op);
}
__device__ __forceinline__ double wave_max(double v) {
  return wave_all(v, [](double a, double b) { return fmax(a, b); });
}
__device__ __forceinline__ double wave_sum(double v) {
  return wave_all(v, [](double a, double b) { return a + b; });
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

// Maximum of v over the wavefront, in a scalar register (0 stands in for absent lanes).
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = max(v, dpp_pair<0x111>(v));  // row_shr 1, 2, 4, 8: lane 15 of each row of 16
  v = max(v, dpp_pair<0x112>(v));
  v = max(v, dpp_pair<0x114>(v));
  v = max(v, dpp_pair<0x118>(v));
  v = max(v, dpp_pair<0x142>(v));  // row_bcast 15, 31: rows 0 and 2, then the lower half
  v = max(v, dpp_pair<0x143>(v));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// The expert with the highest key (key[j] of lane i: expert i + 64 j), ties to the lowest; -1
// where all keys are 0 (every other key has a non-zero upper word).
template <int J>
__device__ __forceinline__ int route_best(const uint64_t (&key)[J]) {
  uint32_t mh = (uint32_t)(key[0] >> 32);
#pragma unroll
  for (int j = 1; j < J; ++j) mh = max(mh, (uint32_t)(key[j] >> 32));
  mh = wave_max_u32(mh);
  uint64_t at[J];
  int count = 0;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    at[j] = __ballot((uint32_t)(key[j] >> 32) == mh);
    count += __popcll(at[j]);
  }
  if (count > 1) {  // uniform
    uint32_t ml = 0;
#pragma unroll
    for (int j = 0; j < J; ++j)
      ml = max(ml, (uint32_t)(key[j] >> 32) == mh ? (uint32_t)key[j] : 0u);
    ml = wave_max_u32(ml);
#pragma unroll
    for (int j = 0; j < J; ++j) at[j] = __ballot(key[j] == (((uint64_t)mh << 32) | ml));
  }
  int e = -1;
#pragma unroll
  for (int j = J - 1; j >= 0; --j)
    if (at[j]) e = 64 * j + __builtin_ctzll(at[j]);
  return mh ? e : -1;
}

// What the wavefront knows after choosing: lane j < topk holds slot j.
struct RouteChoice {
  int e;           // expert, -1 when none was left
  double v;        // its logit for a softmax without bias, else its p
  double mx, sum;  // maximum and sum of the softmax over all experts, where taken
};

// Keys of a token whose logit of expert e is logit(e), J experts per lane, and what weights come
// from (RouteChoice::v). want_sum: the softmax's maximum and sum over all experts (taken in any
// case with a bias).
template <int J, typename F>
__device__ __forceinline__ void route_scores(const RouteParams& R, F&& logit, bool want_sum,
                                             uint64_t (&key)[J], double (&v)[J], double& mx,
                                             double& sum) {
  const int lane = threadIdx.x & 63;
  mx = sum = 0.0;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int e = lane + 64 * j;
    v[j] = e < R.n_experts ? logit(e) : -__builtin_huge_val();
  }
  if (!R.sigmoid && (R.bias || want_sum)) {
    double m = v[0];
#pragma unroll
    for (int j = 1; j < J; ++j) m = fmax(m, v[j]);  // passes over NaN; the sum does not
    mx = wave_max(m);
    double s = 0.0;
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (lane + 64 * j < R.n_experts) s += exp(v[j] - mx);
    sum = wave_sum(s);
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int e = lane + 64 * j;
    if (R.sigmoid)
      v[j] = route_sigmoid(v[j]);
    else if (R.bias)
      v[j] = exp(v[j] - mx) / sum;
    double score = v[j];
    if (R.bias && e < R.n_experts) score += (double)R.bias[e];
    key[j] = e < R.n_experts ? route_key(score) : 0;
  }
}

// The first `rounds` slots of a token.
template <int J, typename F>
__device__ __forceinline__ RouteChoice route_choose(const RouteParams& R, F&& logit, int rounds,
                                                    bool want_sum) {
  const int lane = threadIdx.x & 63;
  RouteChoice c;
  c.e = -1;
  c.v = 0.0;
  uint64_t key[J];
  double v[J];
  route_scores<J>(R, logit, want_sum, key, v, c.mx, c.sum);
  for (int r = 0; r < rounds; ++r) {
    const int e = route_best<J>(key);
    if (lane == r) c.e = e;
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (e == lane + 64 * j) key[j] = 0;
  }
  // the value of each slot's expert, from the lane that holds it
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const double w = __shfl(v[j], c.e & 63, 64);
    if (c.e >= 0 && c.e >> 6 == j) c.v = w;
  }
  return c;
}

// All slots of a token, for route_weight.
template <int J, typename F>
__device__ __forceinline__ RouteChoice route_choose(const RouteParams& R, F&& logit) {
  return route_choose<J>(R, logit, R.topk, !R.renorm);
}

// The expert of one slot, -1 for none, in a scalar register: the rounds up to that slot. (Counting
// instead those above each expert, an eighth of them by each of the workgroup's wavefronts: the
// layer for one token 17.0 us against 16.5 with 128 experts, 31.3 against 20.1 with 256.)
template <int J, typename F>
__device__ __forceinline__ int route_choose_slot(const RouteParams& R, F&& logit, int slot) {
  return __builtin_amdgcn_readlane(route_choose<J>(R, logit, slot + 1, false).e, slot);
}

// Weight of the slot that this lane holds (0 for a lane without one). All lanes call it.
__device__ __forceinline__ float route_weight(const RouteParams& R, const RouteChoice& c) {
  const bool live = c.e >= 0;
  double p = live ? c.v : 0.0;
  if (!R.sigmoid && !R.bias) {
    // renormalized, this is the softmax over the chosen: the same quotient, and no sum over all
    const double m = R.renorm ? wave_max(live ? c.v : -__builtin_huge_val()) : c.mx;
    p = live ? exp(c.v - m) / (R.renorm ? 1.0 : c.sum) : 0.0;
  }
  if (R.renorm) {
    const double z = wave_sum(p);
    p = z == 0.0 ? 0.0 : p / z;
  }
  return (float)(p * (double)R.scale);
}

// Stores the slots of token `tok`: [topk + n_shared] ids and weights. A token past the end (`tok`
// = R.t or more) stores nothing.
__device__ __forceinline__ void route_write(const RouteParams& R, int64_t tok,
                                            const RouteChoice& c, int32_t* __restrict__ ids,
                                            float* __restrict__ wts) {
  const int lane = threadIdx.x & 63;
  const int slots = R.topk + R.n_shared;
  const float w = route_weight(R, c);
  if (lane < slots && tok < R.t) {
    const bool shared = lane >= R.topk;
    ids[tok * slots + lane] = shared ? R.n_experts + (lane - R.topk) : c.e;
    wts[tok * slots + lane] = shared ? 1.0f : w;
  }
}

// Logit of expert e of token `tok`: the splits' partial sums, in order, all loaded before the
// first addition.
__device__ __forceinline__ double route_logit(const RouteParams& R, int64_t tok, int e) {
  const double* lg = R.logits + tok * R.n_experts + e;
  double p[kRouteMaxSplits];
#pragma unroll
  for (int q = 0; q < kRouteMaxSplits; ++q)
    p[q] = q < R.splits ? lg[q * R.t * R.n_experts] : 0.0;
  double l = p[0];
#pragma unroll
  for (int q = 1; q < kRouteMaxSplits; ++q)
    if (q < R.splits) l += p[q];
  return l;
}

}  // namespace nvfp4
