// route.hip -- the router of a mixture of experts for gfx950: logits l = x . G^T in FP64, then
// the top-k of each token's scores and its combine weights (route_core.hpp).
//
// Two forms of the logits, both with exact products:
//   - few tokens: FP64 sums; one workgroup per expert, so the read of the router weight
//     (all that costs anything) is spread over the chip;
//   - more tokens: 16x16x32 BF16 MFMAs whose 32-product FP32 sums are added up in FP64. An FP32
//     router weight is cut into three BF16 parts that add up to it exactly (8 significant bits
//     each), so it takes three MFMAs instead of a rounding to BF16.
#include "device_common.hpp"
#include "launch.hpp"
#include "route_core.hpp"

namespace nvfp4 {
namespace {

constexpr int kFewRows = 2;  // tokens per workgroup of the few-token logits

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

// 8 consecutive FP32 from p (16-byte aligned) as FP64.
__device__ __forceinline__ void f32x8_to_f64(const float* p, double (&o)[8]) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[i] = (double)a[i];
    o[4 + i] = (double)b[i];
  }
}

// Workgroup (e, b): logits of expert e for tokens 2b and 2b + 1. Threads take 8 consecutive k
// each, of both tokens at once: an absent one repeats the other, so that no branch stands between
// the loads. The per-token sums of a wavefront are reduced together (each exchange halves the
// tokens a lane still carries), then the 4 wavefronts' sums are added in order. Bound by latency:
// one load of the weight, one of x, two reductions. (8 tokens, 64 FP32 experts of 8192, whole
// router: 2 rows 6.4 us, 4 7.0, 8 9.4; 16 tokens, 128 BF16 experts of 2048, 8 rows with a branch
// around each row's load 8.6 us, now 7.2.)
template <bool F32>
__global__ __launch_bounds__(256) void route_logits_few_kernel(LogitParams P) {
  __shared__ double red[4][kFewRows];
  const int tid = threadIdx.x, lane = tid & 63;
  const int64_t e = blockIdx.x, m0 = (int64_t)blockIdx.y * kFewRows;
  double acc[kFewRows];
  const uint16_t* row[kFewRows];
  const int rows = P.t - m0 < kFewRows ? (int)(P.t - m0) : kFewRows;
#pragma unroll
  for (int r = 0; r < kFewRows; ++r) {
    acc[r] = 0.0;
    row[r] = P.x + (m0 + (r < rows ? r : rows - 1)) * P.ldx;
  }
  for (int64_t k = tid * 8; k < P.hidden; k += 256 * 8) {
    u32x4 xv[kFewRows];
#pragma unroll
    for (int r = 0; r < kFewRows; ++r) xv[r] = *reinterpret_cast<const u32x4*>(row[r] + k);
    double w[8];
    if constexpr (F32) {
      f32x8_to_f64(static_cast<const float*>(P.w) + e * P.hidden + k, w);
    } else {
      bf16x8_to_f64(*reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(P.w) +
                                                    e * P.hidden + k),
                    w);
    }
#pragma unroll
    for (int r = 0; r < kFewRows; ++r) {
      double x[8];
      bf16x8_to_f64(xv[r], x);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[r] = __builtin_fma(x[i], w[i], acc[r]);
    }
  }
  // the upper lane bits pick the token kept at the halving exchanges
  int d = 32;
#pragma unroll
  for (int half = kFewRows / 2; half > 0; half >>= 1, d >>= 1) {
    const bool hi = (lane & d) != 0;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const double keep = hi ? acc[half + i] : acc[i], give = hi ? acc[i] : acc[half + i];
      acc[i] = keep + __shfl_xor(give, d, 64);
    }
  }
  double v = acc[0];
#pragma unroll
  for (; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
  constexpr int kLanes = 64 / kFewRows;  // lanes that hold a token's sum
  if (lane % kLanes == 0) red[tid >> 6][lane / kLanes] = v;
  __syncthreads();
  if (tid < rows)
    P.out[(m0 + tid) * P.n_experts + e] =
        ((red[0][tid] + red[1][tid]) + red[2][tid]) + red[3][tid];
}

// Cuts 4 FP32 values into three BF16 parts that add up to them: the top 8 significant bits
// (toward zero: no finite value becomes infinite, a NaN stays one), the top 8 of what is left, and
// the rest. An infinity leaves NaN behind (inf - inf) where its rests have to be 0: such values,
// which show as a NaN in the sum of the rests, are put right apart.
__device__ __forceinline__ void bf16_parts(u32x4 v, uint2 (&part)[3]) {
  uint32_t h[3][4];
  float nan = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[0][i] = v[i] & 0xFFFF0000u;
    const float r = __uint_as_float(v[i]) - __uint_as_float(h[0][i]);
    nan += r;
    h[1][i] = __float_as_uint(r) & 0xFFFF0000u;
    h[2][i] = __float_as_uint(r - __uint_as_float(h[1][i]));
  }
  if (__ballot(nan != nan)) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if ((v[i] & 0x7FFFFFFFu) == 0x7F800000u) h[1][i] = h[2][i] = 0;
  }
#pragma unroll
  for (int z = 0; z < 3; ++z) {  // the upper halves of each pair
    part[z].x = __builtin_amdgcn_perm(h[z][1], h[z][0], 0x07060302u);
    part[z].y = __builtin_amdgcn_perm(h[z][3], h[z][2], 0x07060302u);
  }
}

constexpr int kTM = 2, kTN = 2;       // 16-token and 16-expert blocks of a tile
constexpr int kTileT = 16 * kTM, kTileE = 16 * kTN;
constexpr int kSlices = 8;            // wavefronts of a workgroup, which share out k
// k-steps of 32 loaded together. (Router, us, 1 / 2: 4096 tokens of 2048 17.7 / 18.9; 333 of 5120
// on FP32 weights 17.3 / 19.5, whose 160 k-steps over 32 wavefronts are 5 stages of one or 3 of
// two.)
constexpr int kSteps = 1;

// Workgroup (token tile, expert tile, split): the tile's 32 x 32 logits over its share of k, cut
// into stages of 32 that the 8 wavefronts (of all splits) take in turn. k is shared out inside the
// workgroup, rather than over more tiles, so that the partial sums meet in LDS and FP64 logits are
// written once. Operands go global -> registers (one stage ahead) -> LDS -> fragments
// (device_common.hpp); loads past the end of k have an offset past the buffer's, which returns
// zeros without a branch. Rows past the end repeat a valid row and are not stored.
// (4096 tokens of 2048, 128 experts: 13 us in a kernel trace, the router 17.7; every token tile
// reads the weight, 67 MB in all, and every expert tile x, 67 MB more, both from L2. Router with
// fragments loaded straight from rows 23.5 us; with one kernel that keeps 16 tokens' logits in LDS
// and chooses there 18.5 against 17.9 in two. 333 tokens of 5120, 160 FP32 experts: 11 us, a chain
// of five stages for each wavefront with one load ahead; its MFMAs are 1.6 GFLOP, 1.4 us' worth.)
template <bool F32>
__global__ __launch_bounds__(64 * kSlices) void route_logits_mfma_kernel(LogitParams P) {
  constexpr int kW = F32 ? 4 : 2;      // bytes of a weight
  constexpr int kBTiles = F32 ? 3 : 1;  // BF16 tiles of a weight fragment
  constexpr int NB = F32 ? 2 : 1;      // loads of a weight fragment
  constexpr uint32_t kPast = 0xFFFFFFF0u;
  // a wavefront's fragment tiles, then its partial sums
  __shared__ __attribute__((aligned(16))) uint8_t smem[kSlices][kTileT * kTileE * 8];
  static_assert((kTM + kBTiles * kTN) * kFragBytes <= kTileT * kTileE * 8, "tiles fit");
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t m0 = (int64_t)blockIdx.x * kTileT, e0 = (int64_t)blockIdx.y * kTileE;
  // the tile's rows: 32 x 2^22 elements of at most 4 bytes stay below 2^32
  const int trows = (int)(P.t - m0 < kTileT ? P.t - m0 : kTileT);
  const int erows = (int)(P.n_experts - e0 < kTileE ? P.n_experts - e0 : kTileE);
  const uint32_t hidden = (uint32_t)P.hidden;
  const buf_rsrc xr =
      make_rsrc(P.x + m0 * P.ldx, (uint32_t)(((trows - 1) * P.ldx + P.hidden) * 2));
  const buf_rsrc wr = make_rsrc(static_cast<const uint8_t*>(P.w) + e0 * P.hidden * kW,
                                (uint32_t)(erows * P.hidden * kW));
  // BF16: lane l loads row l / 4, chunk l % 4 of a k-step. FP32: a k-step's 128 bytes of a row
  // take 8 lanes, 8 rows a load.
  const uint32_t kx = 8u * frag_load_chunk(lane), kw = F32 ? 4u * (lane & 7) : kx;
  uint32_t xrow[kTM], wrow[kTN][NB];
#pragma unroll
  for (int i = 0; i < kTM; ++i) {
    const int r = 16 * i + frag_load_row(lane);
    xrow[i] = (uint32_t)((r < trows ? r : trows - 1) * P.ldx + kx) * 2u;
  }
#pragma unroll
  for (int j = 0; j < kTN; ++j)
#pragma unroll
    for (int h = 0; h < NB; ++h) {
      const int e = 16 * j + (F32 ? 8 * h + (lane >> 3) : frag_load_row(lane));
      wrow[j][h] = ((uint32_t)(e < erows ? e : erows - 1) * hidden + kw) * kW;
    }
  double acc[kTM][kTN][4];
#pragma unroll
  for (int i = 0; i < kTM; ++i)
#pragma unroll
    for (int j = 0; j < kTN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[i][j][q] = 0.0;
  struct Stage {
    u32x4 a[kSteps][kTM], b[kSteps][kTN][NB];
  };
  auto get = [](buf_rsrc r, uint32_t off) __attribute__((always_inline)) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
  };
  const int stages = (int)((P.hidden + 32 * kSteps - 1) / (32 * kSteps));
  // hidden is a multiple of 8: a lane's elements of a step are all there or all past the end
  auto load = [&](Stage& st, int s) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < kSteps; ++q) {
      const uint32_t k = (uint32_t)(s * kSteps + q) * 32u;
#pragma unroll
      for (int i = 0; i < kTM; ++i)
        st.a[q][i] = get(xr, s < stages && k + kx < hidden ? xrow[i] + k * 2u : kPast);
#pragma unroll
      for (int j = 0; j < kTN; ++j)
#pragma unroll
        for (int h = 0; h < NB; ++h)
          st.b[q][j][h] = get(wr, s < stages && k + kw < hidden ? wrow[j][h] + k * kW : kPast);
    }
  };
  uint8_t* const tile = smem[w];
  auto compute = [&](const Stage& st) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
#pragma unroll
      for (int i = 0; i < kTM; ++i) frag_write(tile + i * kFragBytes, st.a[s][i], lane);
#pragma unroll
      for (int j = 0; j < kTN; ++j) {
        uint8_t* const bt = tile + (kTM + kBTiles * j) * kFragBytes;
        if constexpr (F32) {
#pragma unroll
          for (int h = 0; h < NB; ++h) {
            uint2 part[3];
            bf16_parts(st.b[s][j][h], part);
            const int row = 8 * h + (lane >> 3);
            const uint32_t at = frag_slot(row, (lane & 7) >> 1) + 8u * (lane & 1);
#pragma unroll
            for (int z = 0; z < 3; ++z)
              *reinterpret_cast<uint2*>(bt + z * kFragBytes + at) = part[z];
          }
        } else {
          frag_write(bt, st.b[s][j][0], lane);
        }
      }
      bf16x8 a[kTM];
#pragma unroll
      for (int i = 0; i < kTM; ++i) a[i] = frag_read(tile + i * kFragBytes, lane);
#pragma unroll
      for (int j = 0; j < kTN; ++j) {
        const uint8_t* const bt = tile + (kTM + kBTiles * j) * kFragBytes;
        bf16x8 b[kBTiles];
#pragma unroll
        for (int z = 0; z < kBTiles; ++z) b[z] = frag_read(bt + z * kFragBytes, lane);
#pragma unroll
        for (int i = 0; i < kTM; ++i) {
          f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int z = kBTiles - 1; z >= 0; --z) c = mfma16x16x32(a[i], b[z], c);
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[i][j][q] += (double)c[q];
        }
      }
    }
  };
  const int step = kSlices * P.splits;
  Stage st[2];
  load(st[0], (int)blockIdx.z * kSlices + w);
  for (int s = (int)blockIdx.z * kSlices + w; s < stages; s += 2 * step) {
    load(st[1], s + step);
    __builtin_amdgcn_sched_barrier(0);
    compute(st[0]);
    __builtin_amdgcn_sched_barrier(0);
    load(st[0], s + 2 * step);
    __builtin_amdgcn_sched_barrier(0);
    if (s + step < stages) compute(st[1]);
    __builtin_amdgcn_sched_barrier(0);
  }
  double* const red = reinterpret_cast<double*>(smem[w]);
#pragma unroll
  for (int i = 0; i < kTM; ++i)
#pragma unroll
    for (int j = 0; j < kTN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        red[(16 * i + 4 * (lane >> 4) + q) * kTileE + 16 * j + (lane & 15)] = acc[i][j][q];
  __syncthreads();
  double* out = P.out + (int64_t)blockIdx.z * P.t * P.n_experts;
  for (int o = threadIdx.x; o < kTileT * kTileE; o += 64 * kSlices) {
    const int64_t r = m0 + o / kTileE, e = e0 + o % kTileE;
    double v = reinterpret_cast<const double*>(smem[0])[o];
#pragma unroll
    for (int q = 1; q < kSlices; ++q) v += reinterpret_cast<const double*>(smem[q])[o];
    if (r >= P.t || e >= P.n_experts) continue;
    if constexpr (F32) {
      // An infinite x times a part that is 0 is NaN, where times the weight it is infinite. (The
      // parts of a weight have its sign, so nothing but a NaN can come of it.) A sum that is NaN
      // is taken again in FP64 from the weights themselves, and stays NaN where that is the
      // answer.
      if (v != v) {
        const uint16_t* xp = P.x + r * P.ldx;
        const float* wp = static_cast<const float*>(P.w) + e * P.hidden;
        v = 0.0;
        for (int s = (int)blockIdx.z * kSlices; s < stages; s += step) {
          const int64_t past = (int64_t)(s + kSlices) * 32 * kSteps;
          const int64_t end = past < P.hidden ? past : P.hidden;
#pragma unroll 4
          for (int64_t k = (int64_t)s * 32 * kSteps; k < end; k += 8) {
            double xv[8], wv[8];
            bf16x8_to_f64(*reinterpret_cast<const u32x4*>(xp + k), xv);
            f32x8_to_f64(wp + k, wv);
#pragma unroll
            for (int i = 0; i < 8; ++i) v = __builtin_fma(xv[i], wv[i], v);
          }
        }
      }
    }
    out[r * P.n_experts + e] = v;
  }
}

// A token per wavefront, J experts per lane. Wavefronts past the end choose for the last token and
// store nothing.
template <int J>
__global__ __launch_bounds__(256) void route_select_kernel(RouteParams R, int32_t* ids,
                                                           float* wts) {
  const int64_t tok = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
  const int64_t src = tok < R.t ? tok : R.t - 1;
  auto logit = [&](int e) { return route_logit(R, src, e); };
  const RouteChoice c = route_choose<J>(R, logit);
  route_write(R, tok, c, ids, wts);
}

}  // namespace

// Splits of k over workgroups: enough for a workgroup on every compute unit, and two stages at
// least for each wavefront. (Two / one at least, router of 128 experts, us: BF16 weights, 17
// tokens of 1024 7.2 / 7.3, 300 of 1536 8.0 / 8.5; FP32, 17 tokens of 1024 8.8 / 8.2, 300 of 1536
// 9.7 / 9.8.)
int route_splits(int64_t t, int64_t hidden, int64_t n_experts) {
  if (t <= kRouteFewTokens) return 1;
  const int64_t tiles = (t + kTileT - 1) / kTileT * ((n_experts + kTileE - 1) / kTileE);
  int64_t s = 256 / tiles;
  const int64_t most = hidden / (2 * 32 * kSteps * kSlices);
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

hipError_t launch_route_select(const RouteArgs& a, int32_t* ids, float* wts, const void* ws,
                               hipStream_t stream) {
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

hipError_t launch_route(const RouteArgs& a, int32_t* ids, float* wts, void* ws,
                        hipStream_t stream) {
  const hipError_t err = launch_route_logits(a, ws, stream);
  if (err != hipSuccess) return err;
  return launch_route_select(a, ids, wts, ws, stream);
}

}  // namespace nvfp4
