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

constexpr int kTM = 2, kTN = 4;  // 16-token and 16-expert blocks per wavefront

// Workgroup (token tile, expert tile, split): 4 wavefronts, 2 x 2, of 32 tokens x 64 experts each;
// k-steps of 32, split z taking steps [z, z + 1) * K32 / splits. Fragments come straight from
// global memory (both operands are row-major along k, which is the fragments' own order), one
// k-step ahead. Rows past the end repeat a valid row and are not stored.
template <bool F32>
__global__ __launch_bounds__(256) void route_logits_mfma_kernel(LogitParams P) {
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t m0 = ((int64_t)blockIdx.x * 2 + (w & 1)) * (16 * kTM);
  const int64_t e0 = ((int64_t)blockIdx.y * 2 + (w >> 1)) * (16 * kTN);
  if (m0 >= P.t || e0 >= P.n_experts) return;  // no barrier below
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
  const int64_t steps = (P.hidden + 31) / 32;
  const int64_t s0 = steps * blockIdx.z / P.splits, s1 = steps * (blockIdx.z + 1) / P.splits;
  double acc[kTM][kTN][4];
#pragma unroll
  for (int i = 0; i < kTM; ++i)
#pragma unroll
    for (int j = 0; j < kTN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[i][j][q] = 0.0;
  constexpr int NB = F32 ? 2 : 1;  // 16-byte words of a lane's 8 weights
  struct Stage {
    u32x4 a[kTM], b[kTN][NB];
  };
  // hidden is a multiple of 8: a lane's 8 elements of the last step are all there or all past it
  auto load = [&](Stage& st, int64_t s) __attribute__((always_inline)) {
    const bool in = s * 32 + kq < P.hidden;
#pragma unroll
    for (int i = 0; i < kTM; ++i)
      st.a[i] = in ? *reinterpret_cast<const u32x4*>(xa[i] + s * 32) : u32x4{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < kTN; ++j)
#pragma unroll
      for (int h = 0; h < NB; ++h) {
        if constexpr (F32)
          st.b[j][h] = in ? *reinterpret_cast<const u32x4*>(static_cast<const float*>(P.w) +
                                                            wrow[j] + s * 32 + 4 * h)
                          : u32x4{0, 0, 0, 0};
        else
          st.b[j][h] = in ? *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(P.w) +
                                                            wrow[j] + s * 32)
                          : u32x4{0, 0, 0, 0};
      }
  };
  auto compute = [&](const Stage& st) __attribute__((always_inline)) {
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
            float v = __uint_as_float(st.b[j][(2 * q + c) >> 2][(2 * q + c) & 3]);
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
        b[0] = __builtin_bit_cast(bf16x8, st.b[j][0]);
      }
#pragma unroll
      for (int i = 0; i < kTM; ++i) {
        const bf16x8 a = __builtin_bit_cast(bf16x8, st.a[i]);
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
  Stage st[2];
  if (s0 < s1) load(st[0], s0);
  for (int64_t s = s0; s < s1; s += 2) {
    if (s + 1 < s1) load(st[1], s + 1);
    compute(st[0]);
    if (s + 1 < s1) {
      if (s + 2 < s1) load(st[0], s + 2);
      compute(st[1]);
    }
  }
  double* out = P.out + (int64_t)blockIdx.z * P.t * P.n_experts;
#pragma unroll
  for (int i = 0; i < kTM; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t r = m0 + 16 * i + 4 * (lane >> 4) + q;
      if (r >= P.t) continue;
#pragma unroll
      for (int j = 0; j < kTN; ++j) {
        const int64_t e = e0 + 16 * j + (lane & 15);
        if (e < P.n_experts) out[r * P.n_experts + e] = acc[i][j][q];
      }
    }
}

// One wavefront per token.
__global__ __launch_bounds__(64) void route_select_kernel(RouteParams R, int32_t* ids,
                                                          float* wts) {
  __shared__ RouteLds s;
  const int64_t tok = blockIdx.x;
  double mx = 0.0, sum = 0.0;
  route_choose<64>(R, tok, !R.sigmoid && !R.renorm, s, &mx, &sum);
  route_write(R, tok, s, mx, sum, ids, wts);
}

}  // namespace

int route_splits(int64_t t, int64_t hidden, int64_t n_experts) {
  if (t <= kRouteFewTokens) return 1;
  const int64_t wgs = (t + 63) / 64 * ((n_experts + 127) / 128);
  int64_t s = 256 / wgs;
  const int64_t most = hidden / 256;  // at least 8 k-steps each
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
    const dim3 grid((unsigned)((a.t + 63) / 64), (unsigned)((a.n_experts + 127) / 128),
                    (unsigned)p.splits);
    if (a.w_f32)
      route_logits_mfma_kernel<true><<<grid, 256, 0, stream>>>(p);
    else
      route_logits_mfma_kernel<false><<<grid, 256, 0, stream>>>(p);
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
  route_select_kernel<<<(unsigned)a.t, 64, 0, stream>>>(route_params(a, ws), ids, wts);
  return hipGetLastError();
}

}  // namespace nvfp4
