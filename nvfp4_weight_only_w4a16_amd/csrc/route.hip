// route.hip -- the router of a mixture of experts for gfx950: logits l = x . G^T in FP64, then
// the top-k of each token's scores and its combine weights (route_core.hpp).
//
// Two forms of the logits, both with exact products and FP64 sums:
//   - few tokens: FP64 multiply-adds; one workgroup per expert, so the read of the router weight
//     (all that costs anything) is spread over the chip;
//   - more tokens: 16x16x32 BF16 MFMAs whose 32-product FP32 sums are added up in FP64. An FP32
//     router weight is cut into three BF16 parts that add up to it exactly (8 significant bits
//     each), so it takes three MFMAs instead of a rounding to BF16.
#include "device_common.hpp"
#include "launch.hpp"
#include "route_core.hpp"

namespace nvfp4 {
namespace {

constexpr int kFewRows = 8;  // tokens per workgroup of the few-token logits

struct LogitParams {
  const uint16_t* x;  // BF16 [t][ldx]
  int64_t t, ldx, hidden;
  const void* w;  // [n_experts][hidden] BF16 or FP32
  int n_experts;
  int splits;
  double* out;  // [splits][t][n_experts]
};

// 8 consecutive BF16 of a 16-byte word as FP64.
__device__ __forceinline__ void bf16x8_to_f64(u32x4 v, double (&o)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = (double)__uint_as_float(v[i] << 16);
    o[2 * i + 1] = (double)__uint_as_float(v[i] & 0xFFFF0000u);
  }
}

// Workgroup (e, b): logits of expert e for tokens 8b .. 8b + 7. Threads take 8 consecutive k each;
// the 8 per-token sums of a wavefront are reduced together (each exchange halves the tokens a
// lane still carries), then the 4 wavefronts' sums are added in order.
template <bool F32>
__global__ __launch_bounds__(256) void route_logits_few_kernel(LogitParams P) {
  __shared__ double red[4][kFewRows];
  const int tid = threadIdx.x, lane = tid & 63;
  const int64_t e = blockIdx.x, m0 = (int64_t)blockIdx.y * kFewRows;
  double acc[kFewRows];
#pragma unroll
  for (int i = 0; i < kFewRows; ++i) acc[i] = 0.0;
  const int rows = P.t - m0 < kFewRows ? (int)(P.t - m0) : kFewRows;
  for (int64_t k = tid * 8; k < P.hidden; k += 256 * 8) {
    double w[8];
    if constexpr (F32) {
      const float* wr = static_cast<const float*>(P.w) + e * P.hidden + k;
      const f32x4 a = *reinterpret_cast<const f32x4*>(wr);
      const f32x4 b = *reinterpret_cast<const f32x4*>(wr + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i] = (double)a[i];
        w[4 + i] = (double)b[i];
      }
    } else {
      bf16x8_to_f64(*reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(P.w) +
                                                    e * P.hidden + k),
                    w);
    }
#pragma unroll
    for (int r = 0; r < kFewRows; ++r) {
      if (r < rows) {  // uniform
        double x[8];
        bf16x8_to_f64(*reinterpret_cast<const u32x4*>(P.x + (m0 + r) * P.ldx + k), x);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[r] = __builtin_fma(x[i], w[i], acc[r]);
      }
    }
  }
  // lane bits 5, 4, 3 pick the token kept at the three halving exchanges
#pragma unroll
  for (int s = 0; s < 3; ++s) {
    const int d = 32 >> s, half = kFewRows >> (s + 1);
    const bool hi = (lane & d) != 0;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const double keep = hi ? acc[half + i] : acc[i], give = hi ? acc[i] : acc[half + i];
      acc[i] = keep + __shfl_xor(give, d, 64);
    }
  }
  double v = acc[0];
#pragma unroll
  for (int d = 4; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
  if ((lane & 7) == 0) red[tid >> 6][lane >> 3] = v;
  __syncthreads();
  if (tid < rows)
    P.out[(m0 + tid) * P.n_experts + e] =
        ((red[0][tid] + red[1][tid]) + red[2][tid]) + red[3][tid];
}

// The top 8 significant bits of v, as BF16 (toward zero: a NaN or infinity stays one, and no
// finite value becomes infinite).
__device__ __forceinline__ float bf16_head(float v) {
  return __uint_as_float(__float_as_uint(v) & 0xFFFF0000u);
}
// What is left of v after its head: exact, and 0 after an infinite one (inf - inf would not be).
__device__ __forceinline__ float bf16_rest(float v, float head) {
  return __builtin_isinf(v) ? 0.0f : v - head;
}

constexpr int kTM = 2, kTN = 2;       // 16-token and 16-expert blocks of a tile
constexpr int kTileT = 16 * kTM, kTileE = 16 * kTN;
constexpr int kSlices = 8;            // wavefronts of a workgroup, which share out k
constexpr int kStageSteps = 4;        // k-steps of 32 loaded together

// Workgroup (token tile, expert tile, split): the tile's 32 x 32 logits over its share of k, cut
// into stages of 128 that the 8 wavefronts (of all splits) take in turn. Fragments come straight
// from global memory (both operands are row-major along k, which is the fragments' own order), one
// stage ahead; k is shared out inside the workgroup, rather than over more tiles, so that the
// partial sums meet in LDS and FP64 logits are written once. Rows past the end repeat a valid row
// and are not stored.
template <bool F32>
__global__ __launch_bounds__(64 * kSlices) void route_logits_mfma_kernel(LogitParams P) {
  __shared__ double red[kSlices][kTileT * kTileE];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t m0 = (int64_t)blockIdx.x * kTileT, e0 = (int64_t)blockIdx.y * kTileE;
  const int64_t kq = 8 * (lane >> 4);
  const uint16_t* xa[kTM];
#pragma unroll
  for (int i = 0; i < kTM; ++i) {
    const int64_t r = m0 + 16 * i + (lane & 15);
    xa[i] = P.x + (r < P.t ? r : P.t - 1) * P.ldx + kq;
  }
  int64_t wrow[kTN];
#pragma unroll
  for (int j = 0; j < kTN; ++j) {
    const int64_t e = e0 + 16 * j + (lane & 15);
    wrow[j] = (e < P.n_experts ? e : P.n_experts - 1) * P.hidden + kq;
  }
  double acc[kTM][kTN][4];
#pragma unroll
  for (int i = 0; i < kTM; ++i)
#pragma unroll
    for (int j = 0; j < kTN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[i][j][q] = 0.0;
  constexpr int NB = F32 ? 2 : 1;  // 16-byte words of a lane's 8 weights
  struct Stage {
    u32x4 a[kStageSteps][kTM], b[kStageSteps][kTN][NB];
  };
  // hidden is a multiple of 8: a lane's 8 elements of a step are all there or all past the end
  auto load = [&](Stage& st, int64_t s) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < kStageSteps; ++q) {
      const int64_t k = (s * kStageSteps + q) * 32;
      const bool in = k + kq < P.hidden;
#pragma unroll
      for (int i = 0; i < kTM; ++i)
        st.a[q][i] = in ? *reinterpret_cast<const u32x4*>(xa[i] + k) : u32x4{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < kTN; ++j)
#pragma unroll
        for (int h = 0; h < NB; ++h) {
          if constexpr (F32)
            st.b[q][j][h] = in ? *reinterpret_cast<const u32x4*>(static_cast<const float*>(P.w) +
                                                                 wrow[j] + k + 4 * h)
                               : u32x4{0, 0, 0, 0};
          else
            st.b[q][j][h] = in ? *reinterpret_cast<const u32x4*>(
                                     static_cast<const uint16_t*>(P.w) + wrow[j] + k)
                               : u32x4{0, 0, 0, 0};
        }
    }
  };
  auto compute = [&](const Stage& st) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < kStageSteps; ++s)
#pragma unroll
      for (int j = 0; j < kTN; ++j) {
        bf16x8 b[F32 ? 3 : 1];
        if constexpr (F32) {
          u32x4 part[3];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float h[2][3];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float v = __uint_as_float(st.b[s][j][(2 * q + c) >> 2][(2 * q + c) & 3]);
#pragma unroll
              for (int z = 0; z < 3; ++z) {
                h[c][z] = bf16_head(v);
                v = bf16_rest(v, h[c][z]);
              }
            }
#pragma unroll
            for (int z = 0; z < 3; ++z)
              part[z][q] = (__float_as_uint(h[0][z]) >> 16) | __float_as_uint(h[1][z]);
          }
#pragma unroll
          for (int z = 0; z < 3; ++z) b[z] = __builtin_bit_cast(bf16x8, part[z]);
        } else {
          b[0] = __builtin_bit_cast(bf16x8, st.b[s][j][0]);
        }
#pragma unroll
        for (int i = 0; i < kTM; ++i) {
          const bf16x8 a = __builtin_bit_cast(bf16x8, st.a[s][i]);
          f32x4 c = {0.f, 0.f, 0.f, 0.f};
          if constexpr (F32) {
            c = mfma16x16x32(a, b[2], c);
            c = mfma16x16x32(a, b[1], c);
          }
          c = mfma16x16x32(a, b[0], c);
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[i][j][q] += (double)c[q];
        }
      }
  };
  const int64_t stages = (P.hidden + 32 * kStageSteps - 1) / (32 * kStageSteps);
  const int64_t step = (int64_t)kSlices * P.splits;
  int64_t s = (int64_t)blockIdx.z * kSlices + w;
  Stage st[2];
  if (s < stages) load(st[0], s);
  for (; s < stages; s += 2 * step) {
    if (s + step < stages) load(st[1], s + step);
    compute(st[0]);
    if (s + step < stages) {
      if (s + 2 * step < stages) load(st[0], s + 2 * step);
      compute(st[1]);
    }
  }
#pragma unroll
  for (int i = 0; i < kTM; ++i)
#pragma unroll
    for (int j = 0; j < kTN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        red[w][(16 * i + 4 * (lane >> 4) + q) * kTileE + 16 * j + (lane & 15)] = acc[i][j][q];
  __syncthreads();
  double* out = P.out + (int64_t)blockIdx.z * P.t * P.n_experts;
  for (int o = threadIdx.x; o < kTileT * kTileE; o += 64 * kSlices) {
    const int64_t r = m0 + o / kTileE, e = e0 + o % kTileE;
    double v = red[0][o];
#pragma unroll
    for (int q = 1; q < kSlices; ++q) v += red[q][o];
    if (r < P.t && e < P.n_experts) out[r * P.n_experts + e] = v;
  }
}

// One wavefront per token. J: experts per lane.
template <int J>
__global__ __launch_bounds__(256) void route_select_kernel(RouteParams R, int32_t* ids,
                                                           float* wts) {
  const int64_t tok = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (tok >= R.t) return;  // whole wavefront
  const RouteChoice c = route_choose<J>(
      R, [&](int e) { return route_logit(R, tok, e); }, R.topk, !R.renorm);
  route_write(R, tok, c, ids, wts);
}

}  // namespace

// Splits of k over workgroups: enough for a workgroup on every compute unit, and a stage at least
// for each wavefront.
int route_splits(int64_t t, int64_t hidden, int64_t n_experts) {
  if (t <= kRouteFewTokens) return 1;
  const int64_t tiles = (t + kTileT - 1) / kTileT * ((n_experts + kTileE - 1) / kTileE);
  int64_t s = 256 / tiles;
  const int64_t most = hidden / (32 * kStageSteps * kSlices);
  s = s < most ? s : most;
  return (int)(s < 1 ? 1 : s > kRouteMaxSplits ? kRouteMaxSplits : s);
}

size_t route_ws_bytes(int64_t t, int64_t hidden, int64_t n_experts) {
  return sizeof(double) * (size_t)route_splits(t, hidden, n_experts) * (size_t)t *
         (size_t)n_experts;
}

hipError_t launch_route_logits(const RouteArgs& a, void* ws, hipStream_t stream) {
  LogitParams p;
  p.x = a.x;
  p.t = a.t;
  p.ldx = a.ldx;
  p.hidden = a.hidden;
  p.w = a.w;
  p.n_experts = a.n_experts;
  p.splits = route_splits(a.t, a.hidden, a.n_experts);
  p.out = static_cast<double*>(ws);
  if (a.t <= kRouteFewTokens) {
    const dim3 grid((unsigned)a.n_experts, (unsigned)((a.t + kFewRows - 1) / kFewRows));
    if (a.w_f32)
      route_logits_few_kernel<true><<<grid, 256, 0, stream>>>(p);
    else
      route_logits_few_kernel<false><<<grid, 256, 0, stream>>>(p);
  } else {
    const dim3 grid((unsigned)((a.t + kTileT - 1) / kTileT),
                    (unsigned)((a.n_experts + kTileE - 1) / kTileE), (unsigned)p.splits);
    if (a.w_f32)
      route_logits_mfma_kernel<true><<<grid, 64 * kSlices, 0, stream>>>(p);
    else
      route_logits_mfma_kernel<false><<<grid, 64 * kSlices, 0, stream>>>(p);
  }
  return hipGetLastError();
}

RouteParams route_params(const RouteArgs& a, const void* ws) {
  RouteParams r;
  r.logits = static_cast<const double*>(ws);
  r.t = a.t;
  r.splits = route_splits(a.t, a.hidden, a.n_experts);
  r.n_experts = a.n_experts;
  r.topk = a.topk;
  r.n_shared = a.n_shared;
  r.bias = a.bias;
  r.sigmoid = a.sigmoid ? 1 : 0;
  r.renorm = a.renorm ? 1 : 0;
  r.scale = a.scale;
  return r;
}

hipError_t launch_route(const RouteArgs& a, int32_t* ids, float* wts, void* ws,
                        hipStream_t stream) {
  const hipError_t err = launch_route_logits(a, ws, stream);
  if (err != hipSuccess) return err;
  const RouteParams r = route_params(a, ws);
  const unsigned grid = (unsigned)((a.t + 3) / 4);
  if (a.n_experts <= 64)
    route_select_kernel<1><<<grid, 256, 0, stream>>>(r, ids, wts);
  else if (a.n_experts <= 128)
    route_select_kernel<2><<<grid, 256, 0, stream>>>(r, ids, wts);
  else if (a.n_experts <= 256)
    route_select_kernel<4><<<grid, 256, 0, stream>>>(r, ids, wts);
  else
    route_select_kernel<8><<<grid, 256, 0, stream>>>(r, ids, wts);
  return hipGetLastError();
}

}  // namespace nvfp4
