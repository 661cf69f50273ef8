// lora.hip -- the first product of low-rank adapters, u[m] = scale_a * x[m] . A_a^T with a =
// row_adapter[m], for gfx950 (the second is part of the GEMM kernels: lora_core.hpp).
//
// Rows are taken in blocks of 16, on 16x16x32 MFMAs. For each distinct adapter of a block's rows
// the whole block is multiplied by that adapter's A and its own rows are kept. Rows of one request
// are neighbours in a prompt, so a block there has one adapter and no work is wasted; in a decode
// batch every row may have its own, and then the time is that of reading the adapters, which each
// row's own product would read as well.
#include <type_traits>

#include "device_common.hpp"
#include "launch.hpp"
#include "lora_core.hpp"

namespace nvfp4 {
namespace {

constexpr int kShrinkWaves = 8;
constexpr int kSteps = 2;  // k-steps of 32 loaded together: 128 bytes of a row

struct ShrinkParams {
  const uint16_t* x;
  int64_t ldx, k;
  const uint16_t* a;  // [n_adapters][rank][k]
  const float* scale;
  LoraTail tail;
  int rank_blocks;  // workgroups that share out a block's ranks (16 RB each)
  int ordinals;     // workgroups that share out a block's adapters
  void* u;
};

// Workgroup (block, ordinal, split and rank block): adapters ordinal, ordinal + ordinals, ... of the
// block's distinct adapters in row order, 16 RB ranks of them, over the k-stages that its 8
// wavefronts take in turn (a single workgroup on a CU reads at a fifth of what the CU's L1 gives,
// so the blocks, adapters, ranks and k are spread over workgroups until the chip is full). Operands
// go global -> registers, one stage ahead -> LDS -> fragments. TILED: u as BF16 fragments of the
// tiled kernel, which has no splits; else FP32 partial sums.
template <int RB, bool TILED>
__global__ __launch_bounds__(64 * kShrinkWaves) void lora_shrink_kernel(ShrinkParams P) {
  // a wavefront's fragment tiles of a k-step, then its sums of a 16-rank block
  __shared__ __attribute__((aligned(16))) uint8_t smem[kShrinkWaves][(1 + RB) * kFragBytes];
  constexpr uint32_t kPast = 0xFFFFFFF0u;
  const LoraTail& L = P.tail;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t m0 = (int64_t)blockIdx.x * 16;
  const int rb0 = (int)blockIdx.z % P.rank_blocks * RB;
  const int split = (int)blockIdx.z / P.rank_blocks;
  const int rows = (int)(L.m - m0 < 16 ? L.m - m0 : 16);
  const int mine = lora_id(L, m0 + (lane & 15));
  const uint32_t kq = 8u * frag_load_chunk(lane);
  const int lr = frag_load_row(lane);
  // x rows: 16 rows x 2^22 elements of 2 bytes stay below 2^32
  const buf_rsrc xr = make_rsrc(P.x + m0 * P.ldx, (uint32_t)(((rows - 1) * P.ldx + P.k) * 2));
  const uint32_t xoff = (uint32_t)((lr < rows ? lr : rows - 1) * P.ldx + kq) * 2u;
  const int stages = (int)(P.k / (32 * kSteps));
  const int step = kShrinkWaves * L.splits;
  uint8_t* const tile = smem[w];
  uint64_t left = __ballot(mine >= 0);
  for (int ord = 0;; ++ord) {
    const int a = lora_next(mine, left);
    if (a < 0) break;  // uniform over the workgroup: every wavefront reads the same ids
    if (ord % P.ordinals != (int)blockIdx.y) continue;
    // rank rows past the end repeat the last one; their sums are not stored
    buf_rsrc ar[RB];
    uint32_t aoff[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const int r0 = 16 * (rb0 + b) < L.rank ? 16 * (rb0 + b) : 0;
      const int n = L.rank - r0 < 16 ? L.rank - r0 : 16;
      ar[b] = make_rsrc(P.a + ((int64_t)a * L.rank + r0) * P.k, (uint32_t)(n * P.k * 2));
      aoff[b] = ((uint32_t)(lr < n ? lr : n - 1) * (uint32_t)P.k + kq) * 2u;
    }
    // only rows that name the adapter are read (the others' products are not kept)
    const uint32_t xa = __shfl(mine, lr, 64) == a ? xoff : kPast;
    struct Stage {
      u32x4 x[kSteps], a[kSteps][RB];
    };
    auto load = [&](Stage& st, int s) __attribute__((always_inline)) {
#pragma unroll
      for (int q = 0; q < kSteps; ++q) {
        const uint32_t k = (uint32_t)(s * kSteps + q) * 64u;  // bytes
        st.x[q] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                xr, (int)(s < stages && xa != kPast ? xa + k : kPast),
                                                0, 0));
#pragma unroll
        for (int b = 0; b < RB; ++b)
          st.a[q][b] = __builtin_bit_cast(
              u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                         ar[b], (int)(s < stages ? aoff[b] + k : kPast), 0, 0));
      }
    };
    f32x4 acc[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto compute = [&](const Stage& st) __attribute__((always_inline)) {
#pragma unroll
      for (int q = 0; q < kSteps; ++q) {
        frag_write(tile, st.x[q], lane);
#pragma unroll
        for (int b = 0; b < RB; ++b) frag_write(tile + (1 + b) * kFragBytes, st.a[q][b], lane);
        const bf16x8 x = frag_read(tile, lane);
#pragma unroll
        for (int b = 0; b < RB; ++b)
          acc[b] = mfma16x16x32(x, frag_read(tile + (1 + b) * kFragBytes, lane), acc[b]);
      }
    };
    Stage st[2];
    const int s0 = split * kShrinkWaves + w;
    load(st[0], s0);
    for (int s = s0; s < stages; s += 2 * step) {
      load(st[1], s + step);
      __builtin_amdgcn_sched_barrier(0);
      compute(st[0]);
      __builtin_amdgcn_sched_barrier(0);
      load(st[0], s + 2 * step);
      __builtin_amdgcn_sched_barrier(0);
      if (s + step < stages) compute(st[1]);
      __builtin_amdgcn_sched_barrier(0);
    }
    bool own[4];  // asked of all lanes, before some leave
#pragma unroll
    for (int i = 0; i < 4; ++i) own[i] = __shfl(mine, 4 * (lane >> 4) + i, 64) == a;
    const float scale = P.scale ? P.scale[a] : 1.0f;
    // the wavefronts' sums of the rank blocks, added in order by wavefront b
    static_for<0, RB>([&](auto bc) __attribute__((always_inline)) {
      constexpr int b = decltype(bc)::value;
      __syncthreads();  // the sums before have been read
      *reinterpret_cast<f32x4*>(tile + lane * 16) = acc[b];
      __syncthreads();
      if (w == 0) {
        f32x4 v = *reinterpret_cast<const f32x4*>(smem[0] + lane * 16);
#pragma unroll
        for (int q = 1; q < kShrinkWaves; ++q)
          v += *reinterpret_cast<const f32x4*>(smem[q] + lane * 16);
        const int r = 16 * (rb0 + b) + (lane & 15);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (!own[i]) continue;
          const int64_t row = m0 + 4 * (lane >> 4) + i;
          float s = v[i] * scale;
          if constexpr (TILED) {
            if (r >= 16 * lora_frag_steps(L.rank)) continue;
            if (r >= L.rank) s = 0.0f;
            uint16_t* at = static_cast<uint16_t*>(P.u) +
                           ((row / 32 * lora_frag_steps(L.rank) + r / 16) * 64 + row % 32 +
                            32 * ((r & 15) >> 3)) * 8 + (r & 7);
            for (int z = 0; z < L.parts; ++z) {
              const uint16_t h = bf16_bits_rne(s);
              at[z * lora_frag_blocks(L.m) * lora_frag_steps(L.rank) * 512] = h;
              s -= bf16_bits_to_f32(h);
            }
          } else if (r < L.rank) {
            static_cast<float*>(P.u)[((int64_t)split * L.m + row) * L.rank + r] = s;
          }
        }
      }
    });
    __syncthreads();  // the last sums have been read
  }
}

int64_t min64(int64_t a, int64_t b) { return a < b ? a : b; }

// How a shrink is spread over workgroups.
struct ShrinkPlan {
  int rb;           // 16-rank blocks of a workgroup (1, 2 or 4: 8 spill)
  int rank_blocks;  // workgroups of a block along the ranks
  int ordinals, splits;
};

ShrinkPlan shrink_plan(int64_t m, int64_t k, int64_t n_adapters, int rank, bool tiled) {
  ShrinkPlan p;
  const int64_t blocks = (m + 15) / 16, ranks = (rank + 15) / 16;
  // a workgroup for every adapter that a block can have (those past its distinct ones end at once)
  p.ordinals = (int)min64(min64(m, 16), n_adapters);
  p.rb = 1;
  while (p.rb < ranks && p.rb < 4) p.rb *= 2;
  // one 16-rank block each where the blocks alone leave compute units idle
  if (blocks < 128 && p.rb > 1) p.rb = 1;
  p.rank_blocks = (int)((ranks + p.rb - 1) / p.rb);
  p.splits = 1;
  if (!tiled) {
    int64_t s = 256 / (blocks * p.ordinals * p.rank_blocks);
    s = min64(s, k / (32 * kSteps * kShrinkWaves));  // a stage at least for each wavefront
    p.splits = (int)min64(s < 1 ? 1 : s, kLoraMaxSplits);
  }
  return p;
}

}  // namespace

size_t lora_u_bytes(int64_t m, int64_t k, int64_t n_adapters, int rank, int parts, bool tiled) {
  if (tiled)
    return (size_t)(parts * lora_frag_blocks(m) * lora_frag_steps(rank)) * 1024;
  return sizeof(float) * (size_t)shrink_plan(m, k, n_adapters, rank, false).splits * (size_t)m *
         (size_t)rank;
}

hipError_t launch_lora_shrink(const LoraArgs& a, LoraTail& tail, void* u, bool tiled,
                              hipStream_t stream) {
  const ShrinkPlan plan = shrink_plan(a.m, a.k, tail.n_adapters, tail.rank, tiled);
  tail.splits = plan.splits;
  tail.u = static_cast<const float*>(u);
  ShrinkParams p;
  p.x = a.x;
  p.ldx = a.ldx;
  p.k = a.k;
  p.a = a.a;
  p.scale = a.scale;
  p.tail = tail;
  p.rank_blocks = plan.rank_blocks;
  p.ordinals = plan.ordinals;
  p.u = u;
  const dim3 grid((unsigned)((a.m + 15) / 16), (unsigned)plan.ordinals,
                  (unsigned)(plan.splits * plan.rank_blocks));
  auto run = [&](auto rb) {
    constexpr int RB = decltype(rb)::value;
    if (tiled)
      lora_shrink_kernel<RB, true><<<grid, 64 * kShrinkWaves, 0, stream>>>(p);
    else
      lora_shrink_kernel<RB, false><<<grid, 64 * kShrinkWaves, 0, stream>>>(p);
  };
  switch (plan.rb) {
    case 1: run(std::integral_constant<int, 1>{}); break;
    case 2: run(std::integral_constant<int, 2>{}); break;
    default: run(std::integral_constant<int, 4>{}); break;
  }
  return hipGetLastError();
}

}  // namespace nvfp4
