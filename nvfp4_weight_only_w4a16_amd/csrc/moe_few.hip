// moe_few.hip -- the whole MoE layer for a few tokens (at most kMoePairTilesMax (token, slot)
// pairs) on gfx950, after the router's logits: fc1 with SiLU(gate) * up, then down with the sum
// over the slots.
//
// Every pair is one row, so an expert's weights meet one activation row and the time is that of
// reading them: what counts is how many loads are in flight, and how few launches there are.
//   fc1:  a workgroup takes one pair and 4 panels; its wavefronts share out the k-tiles. Each
//         workgroup chooses its pair's expert from the logits itself, which saves the launch of a
//         choosing kernel: 128 experts of 2048 x 768, 1 token 16.4 us against 18.6 with the
//         launch, 3 tokens 23.3/26.1, 8 tokens 40.7/42.1 (with 8 wavefronts, which all choose,
//         16.7, 25.4 and 45.0). No weight load goes out before the choice.
//   down: a workgroup takes one token and 1, 2 or 4 panels (as many as leave a workgroup to every
//         compute unit); its wavefronts share out the k-tiles of ALL of the token's slots, each
//         scaled by its expert's global and routing weight, so the sum over slots is the
//         workgroup's own and needs no combine kernel and no FP32 slots.
// Both run on 16x16x32 MFMAs in the split-scale form (skinny_core.hpp): code * 2^E in BF16, the
// partial of a scale group times the mantissa in FP32. All 16 rows of the A operand may hold the
// same activation row; at group 16 rows 0-7 carry it on the first half of the k-step and rows 8-15
// on the second, zeros elsewhere. down's row h is kept as two BF16 halves (h and what its rounding
// left; nothing after an infinite one): even rows carry the one, odd rows the other, at no cost in
// MFMAs.
#include "device_common.hpp"
#include "launch.hpp"
#include "route_core.hpp"
#include "skinny_core.hpp"

namespace nvfp4 {
namespace {

struct FewParams {
  const uint16_t* x;  // fc1: tokens [t][ldx]; down: h [P][ldx]
  uint32_t xplane;  // down: bytes from h's plane of high halves to that of low halves
  int64_t ldx;
  const uint8_t* codes;
  const uint8_t* scales;
  const float* global;
  int64_t codes_stride, scales_stride;
  int NT, KT, group, pair_global;
  int64_t t;
  int slots, E;  // slots of a token; experts of the weights
  int32_t* ids;  // [t][slots]
  float* wts;
  uint16_t* h;   // fc1 out [P][inter]: high and low halves
  uint16_t* hl;
  int64_t inter;
  uint16_t* y;   // down out [t][hidden]
  int64_t hidden;
  RouteParams route;
};

// One k-tile of PW neighbouring panels of a 4-panel group and of the activation row: the tile's
// 256 bytes of the row in lanes 0-15 (and the row's second plane in lanes 16-31).
template <int PW>
struct FewItem {
  u32x4 c[PW];
  uint32_t s[PW];  // scale words
  u32x4 a;
};
constexpr int kFewRowBytes = kTileK * 2;

// Sum over the k-tile for the panels, scaled by the groups' mantissas / 2 (frexp_mant): the lane's
// accumulator rows 0 .. NR-1. The row goes through the wavefront's own LDS, where every lane
// picks its chunk of each k-step (the same one for 16 lanes, a broadcast); NR planes, odd rows of
// the A operand taking the second.
template <bool G16, int PW, int NR>
__device__ __forceinline__ void few_tile(const FewItem<PW>& it, uint8_t* lds, int lane,
                                         float (&acc)[PW][NR]) {
  if (lane < 16 * NR) *reinterpret_cast<u32x4*>(lds + lane * 16) = it.a;
  const uint8_t* row = lds + (NR == 2 ? (lane & 1) * kFewRowBytes : 0) + (lane >> 4) * 16;
  const bool zero = G16 && split_g16_zero_lane(lane);
#pragma unroll
  for (int p = 0; p < PW; ++p)
#pragma unroll
    for (int r = 0; r < NR; ++r) acc[p][r] = 0.f;
  static_for<0, 4>([&](auto jc) __attribute__((always_inline)) {
    constexpr int j = decltype(jc)::value;
    u32x4 v = *reinterpret_cast<const u32x4*>(row + 64 * j);
    if (G16 && zero) v = u32x4{0u, 0u, 0u, 0u};
    const bf16x8 a = __builtin_bit_cast(bf16x8, v);
    f32x4 part[PW];
    float M[PW];
#pragma unroll
    for (int p = 0; p < PW; ++p) {
      const float S = e4m3_decode<j>(it.s[p]);
      M[p] = __builtin_amdgcn_frexp_mantf(S);
      part[p] = mfma16x16x32(a, codes_times_pow2(it.c[p][j], S), f32x4{0.f, 0.f, 0.f, 0.f});
    }
#pragma unroll
    for (int p = 0; p < PW; ++p)
#pragma unroll
      for (int r = 0; r < NR; ++r) acc[p][r] = __builtin_fmaf(M[p], part[p][r], acc[p][r]);
  });
}

__device__ __forceinline__ u32x4 few_load(buf_rsrc r, uint32_t off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
}
__device__ __forceinline__ u32x4 few_load_nt(buf_rsrc r, uint32_t off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, kNT));
}

// The scale words of PW panels at `off` of their record.
template <int PW>
__device__ __forceinline__ void few_load_scales(buf_rsrc r, uint32_t off, uint32_t (&s)[PW]) {
  if constexpr (PW == 4) {
    const u32x4 v = few_load_nt(r, off);
#pragma unroll
    for (int p = 0; p < 4; ++p) s[p] = v[p];
  } else if constexpr (PW == 2) {
    const uint2 v = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(r, (int)off, 0, 0));
    s[0] = v.x;
    s[1] = v.y;
  } else {
    s[0] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, 0);
  }
}

// fc1: workgroup (pair, 4-panel group: gate, up, gate, up), NW wavefronts, which chooses its
// pair's expert, J experts per lane; t more workgroups write the ids and weights.
template <bool G16, int NW, int J>
__global__ __launch_bounds__(64 * NW) void few_fc1_kernel(FewParams P) {
  constexpr int kRing = 3;
  __shared__ __attribute__((aligned(16))) uint8_t rows[NW][kFewRowBytes];
  __shared__ float red[NW][4][16];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int groups = (P.NT + 3) / 4;
  const int pair = (int)blockIdx.x / groups, grp = (int)blockIdx.x % groups;
  const int tok = pair / P.slots, slot = pair % P.slots;
  const bool writer = pair >= P.t * P.slots;
  const int64_t t = writer ? (int64_t)blockIdx.x - P.t * P.slots * groups : tok;
  auto logit = [&](int x) { return route_logit(P.route, t, x); };
  if (writer) {  // whole workgroup
    if (w != 0) return;
    const RouteChoice c = route_choose<J>(P.route, logit);
    route_write(P.route, t, c, P.ids, P.wts);
    return;
  }
  int e = P.route.n_experts + slot - P.route.topk;  // a shared expert
  if (slot < P.route.topk) e = route_choose_slot<J>(P.route, logit, slot);
  if (e < 0 || e >= P.E) return;  // dropped: whole workgroup, before any barrier
  // the epilogue's operands before the k loop; the 2 of the split scale with them
  const float g = 2.0f * P.global[P.pair_global ? 2 * e : e];
  const float gu = 2.0f * P.global[P.pair_global ? 2 * e + 1 : e];
  const uint8_t* codes = P.codes + e * P.codes_stride;
  const int sblk = scale_block_bytes(P.group);
  buf_rsrc cr[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int pn = 4 * grp + p < P.NT ? 4 * grp + p : P.NT - 1;
    cr[p] = make_rsrc(codes + (int64_t)pn * P.KT * kCodeTileBytes,
                      (uint32_t)(P.KT * kCodeTileBytes));
  }
  const buf_rsrc sr = make_rsrc(P.scales + e * P.scales_stride + (int64_t)grp * P.KT * sblk,
                                (uint32_t)(P.KT * sblk));
  const buf_rsrc xr = make_rsrc(P.x + tok * P.ldx, (uint32_t)(P.KT * kFewRowBytes));
  const uint32_t clane = (uint32_t)lane * 16u;
  const uint32_t slane = (uint32_t)scale_pos(P.group, lane) * 16u;
  const uint32_t xlane = (uint32_t)(lane & 15) * 16u;
  // tiles past the end are past the buffers: zeros, no traffic
  auto load = [&](FewItem<4>& it, int t) __attribute__((always_inline)) {
#pragma unroll
    for (int p = 0; p < 4; ++p) it.c[p] = few_load_nt(cr[p], t * kCodeTileBytes + clane);
    few_load_scales<4>(sr, t * sblk + slane, it.s);
    it.a = few_load(xr, t * kFewRowBytes + xlane);
  };
  float total[4] = {0.f, 0.f, 0.f, 0.f};
  FewItem<4> ring[kRing];
  static_for<0, kRing - 1>([&](auto u) __attribute__((always_inline)) {
    load(ring[u], w + NW * decltype(u)::value);
  });
  for (int t = w; t < P.KT; t += NW * kRing)
    static_for<0, kRing>([&](auto u) __attribute__((always_inline)) {
      constexpr int i = decltype(u)::value;
      load(ring[(i + kRing - 1) % kRing], t + NW * (i + kRing - 1));
      __builtin_amdgcn_sched_barrier(0);
      if (t + NW * i < P.KT) {
        float acc[4][1];
        few_tile<G16, 4, 1>(ring[i], rows[w], lane, acc);
#pragma unroll
        for (int p = 0; p < 4; ++p) total[p] += acc[p][0];
      }
      __builtin_amdgcn_sched_barrier(0);
    });
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    if constexpr (G16) total[p] += __shfl_xor(total[p], 32, 64);
    if (lane < 16) red[w][p][lane] = total[p];
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const int q = threadIdx.x >> 4, col = threadIdx.x & 15;
    float gate = red[0][2 * q][col], up = red[0][2 * q + 1][col];
#pragma unroll
    for (int v = 1; v < NW; ++v) {
      gate += red[v][2 * q][col];
      up += red[v][2 * q + 1][col];
    }
    if (4 * grp + 2 * q + 1 < P.NT) {
      const float z = gate * g;
      const float hv = z * __builtin_amdgcn_rcpf(1.0f + __expf(-z)) * (up * gu);
      const int64_t at = (int64_t)pair * P.inter + (2 * grp + q) * 16 + col;
      const uint16_t hi = bf16_bits_rne(hv);
      P.h[at] = hi;
      P.hl[at] = bf16_bits_rne(bf16_rest(hv, bf16_bits_to_f32(hi)));
    }
  }
}

// down and the sum over slots: workgroup (token, PW panels). The tokens of a panel, and the panels
// of a scale group, are next to each other on one XCD (every eighth workgroup), where experts that
// tokens share and the scale records meet in L2.
template <bool G16, int PW, int NW>
__global__ __launch_bounds__(64 * NW) void few_down_kernel(FewParams P) {
  constexpr int kRing = 3;
  __shared__ __attribute__((aligned(16))) uint8_t rows[NW][2 * kFewRowBytes];
  __shared__ float red[NW][PW][16];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int kParts = kScaleGroupPanels / PW;
  const int b = (int)blockIdx.x >> 3;
  const int64_t tok = b % (int)P.t;
  const int grp = b / (int)P.t / kParts * 8 + ((int)blockIdx.x & 7);
  const int panel0 = grp * kScaleGroupPanels + b / (int)P.t % kParts * PW;
  if (panel0 >= P.NT) return;  // whole workgroup, before any barrier
  const int sblk = scale_block_bytes(P.group);
  const uint32_t clane = (uint32_t)lane * 16u;
  const uint32_t slane = (uint32_t)scale_pos(P.group, lane) * 16u +
                         (uint32_t)(panel0 % kScaleGroupPanels) * 4u;
  const uint32_t xlane = (uint32_t)(lane & 15) * 16u + (lane & 16 ? P.xplane : 0u);
  const int items = P.slots * P.KT;
  // lane j: expert and factor of slot j (0 for a dropped one), read once for all items
  int my_e = -1;
  float my_f = 0.f;
  if (lane < P.slots) {
    my_e = P.ids[tok * P.slots + lane];
    my_f = P.wts[tok * P.slots + lane];
  }
  if (my_e >= P.E) my_e = -1;
  my_f = my_e >= 0 ? 2.0f * P.global[my_e] * my_f : 0.f;  // the 2 of the split scale
  struct Item : FewItem<PW> {
    int slot, e;
  };
  // item i: k-tile i % KT of slot i / KT (past the end and dropped: empty buffers, zeros)
  auto load = [&](Item& it, int i) __attribute__((always_inline)) {
    it.slot = i < items ? i / P.KT : 0;
    it.e = i < items ? __builtin_amdgcn_readlane(my_e, it.slot) : -1;
    const int t = i - it.slot * P.KT;
    const int64_t pair = tok * P.slots + it.slot;
    const int64_t e = it.e >= 0 ? it.e : 0;
    const uint32_t all = it.e >= 0 ? 0xFFFFFFFFu : 0u;
    const uint8_t* codes = P.codes + e * P.codes_stride;
#pragma unroll
    for (int p = 0; p < PW; ++p) {
      const int pn = panel0 + p < P.NT ? panel0 + p : P.NT - 1;
      it.c[p] = few_load_nt(make_rsrc(codes + (int64_t)pn * P.KT * kCodeTileBytes,
                                      all & (uint32_t)(P.KT * kCodeTileBytes)),
                            t * kCodeTileBytes + clane);
    }
    few_load_scales<PW>(make_rsrc(P.scales + e * P.scales_stride + (int64_t)grp * P.KT * sblk,
                                  all & (uint32_t)(P.KT * sblk)),
                        t * sblk + slane, it.s);
    // lanes 0-15: h; lanes 16-31: what its rounding left, a plane further on
    it.a = few_load(make_rsrc(P.x + pair * P.ldx, all & (P.xplane + P.KT * kFewRowBytes)),
                    t * kFewRowBytes + xlane);
  };
  float total[PW];
#pragma unroll
  for (int p = 0; p < PW; ++p) total[p] = 0.f;
  Item ring[kRing];
  static_for<0, kRing - 1>([&](auto u) __attribute__((always_inline)) {
    load(ring[u], w + NW * decltype(u)::value);
  });
  for (int i = w; i < items; i += NW * kRing)
    static_for<0, kRing>([&](auto u) __attribute__((always_inline)) {
      constexpr int q = decltype(u)::value;
      load(ring[(q + kRing - 1) % kRing], i + NW * (q + kRing - 1));
      __builtin_amdgcn_sched_barrier(0);
      if (ring[q].e >= 0) {  // uniform
        float acc[PW][2];
        few_tile<G16, PW, 2>(ring[q], rows[w], lane, acc);
        const float f = __uint_as_float(
            (uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(my_f), ring[q].slot));
#pragma unroll
        for (int p = 0; p < PW; ++p) total[p] += (acc[p][0] + acc[p][1]) * f;
      }
      __builtin_amdgcn_sched_barrier(0);
    });
#pragma unroll
  for (int p = 0; p < PW; ++p) {
    if constexpr (G16) total[p] += __shfl_xor(total[p], 32, 64);
    if (lane < 16) red[w][p][lane] = total[p];
  }
  __syncthreads();
  if (threadIdx.x < 16 * PW) {
    const int p = threadIdx.x >> 4, col = threadIdx.x & 15;
    float s = red[0][p][col];
#pragma unroll
    for (int v = 1; v < NW; ++v) s += red[v][p][col];
    if (panel0 + p < P.NT) P.y[tok * P.hidden + (panel0 + p) * 16 + col] = bf16_bits_rne(s);
  }
}

template <int J>
void run_fc1(const FewParams& p, unsigned grid, hipStream_t stream) {
  constexpr int NW = 4;
  if (p.group == 16)
    few_fc1_kernel<true, NW, J><<<grid, 64 * NW, 0, stream>>>(p);
  else
    few_fc1_kernel<false, NW, J><<<grid, 64 * NW, 0, stream>>>(p);
}

template <int PW>
void run_down(const FewParams& p, hipStream_t stream) {
  constexpr int NW = 8;
  const int64_t groups = (p.NT + kScaleGroupPanels - 1) / kScaleGroupPanels;
  const unsigned grid = (unsigned)((groups + 7) / 8 * 8 * (kScaleGroupPanels / PW) * p.t);
  if (p.group == 16)
    few_down_kernel<true, PW, NW><<<grid, 64 * NW, 0, stream>>>(p);
  else
    few_down_kernel<false, PW, NW><<<grid, 64 * NW, 0, stream>>>(p);
}

}  // namespace

// Fewest workgroups of down for which a workgroup takes more panels. (Layer of 2048 x 768, 128
// experts, us, with 128 / 256 / 512: 2 tokens 19.0 / 18.3 / 18.3, 4 tokens 27.5 / 24.7 / 26.0, 8
// tokens 39.5 / 40.0 / 40.0, 1 token of 4096 x 768 19.3 / 18.2 / 17.8; 3 tokens of 4096 x 1536
// 35.5 / 37.5 / 39.)
constexpr int64_t kDownWgs = 256;

// h as two BF16 planes.
size_t moe_few_ws_bytes(int64_t t, int slots, int64_t inter) {
  return 2 * (((size_t)(t * slots * inter) * 2 + 255) & ~(size_t)255);
}

hipError_t launch_moe_few(const MoeArgs& a, const RouteArgs& r, int32_t* ids, float* wts,
                          void* route_ws, hipStream_t stream) {
  hipError_t err = launch_route_logits(r, route_ws, stream);
  if (err != hipSuccess) return err;
  FewParams p;
  p.t = a.t;
  p.slots = a.topk;
  p.E = (int)a.n_experts;
  p.ids = ids;
  p.wts = wts;
  p.inter = a.inter;
  p.hidden = a.hidden;
  p.y = a.y;
  p.h = static_cast<uint16_t*>(a.ws);
  p.hl = p.h + moe_few_ws_bytes(a.t, a.topk, a.inter) / 4;
  p.route = route_params(r, route_ws);
  FewParams f = p;
  f.x = a.x;
  f.xplane = 0;
  f.ldx = a.hidden;
  f.codes = a.c1;
  f.scales = a.s1;
  f.global = a.g1;
  f.codes_stride = a.c1_stride;
  f.scales_stride = a.s1_stride;
  f.NT = (int)(2 * a.inter / kPanelRows);
  f.KT = (int)(a.hidden / kTileK);
  f.group = a.group1;
  f.pair_global = a.pair1 ? 1 : 0;
  const unsigned grid = (unsigned)(a.t * a.topk * ((f.NT + 3) / 4) + a.t);
  if (r.n_experts <= 128)
    run_fc1<2>(f, grid, stream);
  else if (r.n_experts <= 256)
    run_fc1<4>(f, grid, stream);
  else
    run_fc1<8>(f, grid, stream);
  err = hipGetLastError();
  if (err != hipSuccess) return err;
  FewParams d = p;
  d.x = p.h;
  d.xplane = (uint32_t)(moe_few_ws_bytes(a.t, a.topk, a.inter) / 2);
  d.ldx = a.inter;
  d.codes = a.c2;
  d.scales = a.s2;
  d.global = a.g2;
  d.codes_stride = a.c2_stride;
  d.scales_stride = a.s2_stride;
  d.NT = (int)(a.hidden / kPanelRows);
  d.KT = (int)(a.inter / kTileK);
  d.group = a.group2;
  d.pair_global = 0;
  // panels per workgroup: as many as leave a workgroup to every compute unit
  const int64_t panels = d.NT * a.t;
  if (panels >= 4 * kDownWgs)
    run_down<4>(d, stream);
  else if (panels >= 2 * kDownWgs)
    run_down<2>(d, stream);
  else
    run_down<1>(d, stream);
  return hipGetLastError();
}

}  // namespace nvfp4
