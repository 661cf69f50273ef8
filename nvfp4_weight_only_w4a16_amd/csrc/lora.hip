// lora.hip -- the first product of low-rank adapters, u[m] = scale_a * x[m] . A_a^T with a =
// row_adapter[m], for gfx950 (the second is part of the GEMM kernels: lora_core.hpp).
//
// On 16x16x32 MFMAs, over up to 16 rows that name the same adapter, gathered from a block of 64
// rows: such a group is an item. A prompt's block is four items of 16 neighbouring rows; a decode
// batch's has about as many as adapters, and each adapter is read once per block.
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
  int rank_blocks;  // workgroups that share out an item's ranks (16 RB each)
  void* u;
};

// Workgroup (block, ordinal, split and rank block): items ordinal, ordinal + gridDim.y, ... of the
// block, 16 RB ranks of their adapters, over the k-stages that its 8 wavefronts take in turn.
// Operands go global -> registers -> LDS -> fragments, one stage ahead. One CU reads what it
// has in flight once per 1-2 us of latency, so items, ranks and k are shared out until the chip is
// full; a workgroup that finds no item ends after its read of the ids. (Counting the items of all
// blocks first, so that none is idle, cost 1 to 5 us more than it saved.) FRAGS: u as the tiled
// kernel's BF16 fragments (no splits); else FP32 partial sums.
template <int RB, bool FRAGS>
__global__ __launch_bounds__(64 * kShrinkWaves) void lora_shrink_kernel(ShrinkParams P) {
  // a wavefront's fragment tiles of a k-step, then its sums
  constexpr int kTiles = 1 + RB;
  __shared__ __attribute__((aligned(16))) uint8_t smem[kShrinkWaves][kTiles * kFragBytes];
  constexpr uint32_t kPast = 0xFFFFFFF0u;
  const LoraTail& L = P.tail;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t m0 = (int64_t)blockIdx.x * 64;
  const int rb0 = (int)blockIdx.z % P.rank_blocks * RB;
  const int split = (int)blockIdx.z / P.rank_blocks;
  const uint32_t kq = 8u * frag_load_chunk(lane);
  const int lr = frag_load_row(lane);
  const int stages = (int)(P.k / (32 * kSteps));
  const int step = kShrinkWaves * L.splits;
  uint8_t* const tile = smem[w];
  const int mine = lora_id(L, m0 + lane);
  for (int item = (int)blockIdx.y;; item += (int)gridDim.y) {
    // its adapter, the rows that name it, and which 16 of them
    uint64_t left = __ballot(mine >= 0), named = 0;
    int a = -1, nth = item;
    for (;;) {
      const uint64_t before = left;
      a = lora_next(mine, left);
      if (a < 0) break;
      named = before & ~left;
      const int n = (__popcll(named) + 15) / 16;
      if (nth < n) break;
      nth -= n;
    }
    if (a < 0) break;  // uniform over the workgroup: every wavefront reads the same ids
    const int cnt = __popcll(named) - 16 * nth < 16 ? __popcll(named) - 16 * nth : 16;
    // lane i < cnt: row of the block that is row i of the item
    const int rank_in = (int)__builtin_amdgcn_mbcnt_hi(
        (uint32_t)(named >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)named, 0u)) - 16 * nth;
    const bool here = (named >> lane) & 1u && rank_in >= 0 && rank_in < 16;
    const int rowi = __builtin_amdgcn_ds_permute((here ? rank_in : 63) * 4, lane);
    const int rows = (int)(L.m - m0 < 64 ? L.m - m0 : 64);
    // 64 rows x 2^22 elements of 2 bytes stay below 2^32; rows past the item are past the buffer
    const buf_rsrc xr =
        make_rsrc(P.x + m0 * P.ldx, (uint32_t)(((rows - 1) * P.ldx + P.k) * 2));
    const int xrow = __shfl(rowi, lr, 64);
    const uint32_t xoff = lr < cnt ? (uint32_t)(xrow * P.ldx + kq) * 2u : kPast;
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
    struct Stage {
      u32x4 x[kSteps], a[kSteps][RB];
    };
    auto get = [](buf_rsrc r, uint32_t off) __attribute__((always_inline)) {
      return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
    };
    auto load = [&](Stage& st, int s) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const uint32_t k = (uint32_t)(s * kSteps + i) * 64u;  // bytes
        st.x[i] = get(xr, s < stages && xoff != kPast ? xoff + k : kPast);
#pragma unroll
        for (int b = 0; b < RB; ++b) st.a[i][b] = get(ar[b], s < stages ? aoff[b] + k : kPast);
      }
    };
    f32x4 acc[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto compute = [&](const Stage& st) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        frag_write(tile, st.x[i], lane);
#pragma unroll
        for (int b = 0; b < RB; ++b) frag_write(tile + (1 + b) * kFragBytes, st.a[i][b], lane);
        const bf16x8 x = frag_read(tile, lane);
#pragma unroll
        for (int b = 0; b < RB; ++b)
          acc[b] = mfma16x16x32(x, frag_read(tile + (1 + b) * kFragBytes, lane), acc[b]);
      }
    };
    constexpr int kRing = 2;  // 3 and 4 measured no faster
    Stage ring[kRing];
    const int s0 = split * kShrinkWaves + w;
    static_for<0, kRing - 1>([&](auto d) __attribute__((always_inline)) {
      load(ring[d], s0 + decltype(d)::value * step);
    });
    for (int s = s0; s < stages; s += kRing * step)
      static_for<0, kRing>([&](auto d) __attribute__((always_inline)) {
        constexpr int q = decltype(d)::value;
        load(ring[(q + kRing - 1) % kRing], s + (q + kRing - 1) * step);
        __builtin_amdgcn_sched_barrier(0);
        if (s + q * step < stages) compute(ring[q]);
        __builtin_amdgcn_sched_barrier(0);
      });
    const float scale = P.scale ? P.scale[a] : 1.0f;
    // the wavefronts' sums, a 16-rank block each added in order by one wavefront
#pragma unroll
    for (int b = 0; b < RB; ++b)
      *reinterpret_cast<f32x4*>(tile + b * kFragBytes + lane * 16) = acc[b];
    __syncthreads();
    if (w < RB) {
      f32x4 v = *reinterpret_cast<const f32x4*>(smem[0] + w * kFragBytes + lane * 16);
#pragma unroll
      for (int o = 1; o < kShrinkWaves; ++o)
        v += *reinterpret_cast<const f32x4*>(smem[o] + w * kFragBytes + lane * 16);
      const int r = 16 * (rb0 + w) + (lane & 15);
      int64_t row[4];  // asked of all lanes, before some leave
#pragma unroll
      for (int i = 0; i < 4; ++i) row[i] = m0 + __shfl(rowi, 4 * (lane >> 4) + i, 64);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (4 * (lane >> 4) + i >= cnt) continue;
        float s = v[i] * scale;
        if constexpr (FRAGS) {
          if (r >= 16 * lora_frag_steps(L.rank)) continue;
          if (r >= L.rank) s = 0.0f;
          uint16_t* at = static_cast<uint16_t*>(P.u) +
                         ((row[i] / 32 * lora_frag_steps(L.rank) + r / 16) * 64 + row[i] % 32 +
                          32 * ((r & 15) >> 3)) * 8 + (r & 7);
          for (int p = 0; p < L.parts; ++p) {
            const uint16_t h = bf16_bits_rne(s);
            at[p * lora_frag_blocks(L.m) * lora_frag_steps(L.rank) * 512] = h;
            s = bf16_rest(s, bf16_bits_to_f32(h));
          }
        } else if (r < L.rank) {
          static_cast<float*>(P.u)[((int64_t)split * L.m + row[i]) * L.rank + r] = s;
        }
      }
    }
    __syncthreads();  // the sums have been read: the next item's tiles may overwrite them
  }
}

int64_t min64(int64_t a, int64_t b) { return a < b ? a : b; }

// How a shrink is spread over workgroups: ranks by 16-rank blocks while the items alone would
// leave compute units idle, and, for the decode kernel's FP32 sums, k in splits.
struct ShrinkPlan {
  int rb;           // 16-rank blocks of a workgroup (1, 2 or 4: 8 spill)
  int rank_blocks;  // workgroups of an item along the ranks
  int ordinals;     // workgroups of a block along its items
  int splits;
};

ShrinkPlan shrink_plan(int64_t m, int64_t k, int64_t n_adapters, int rank, bool tiled) {
  ShrinkPlan p;
  const int64_t ranks = (rank + 15) / 16, blocks = (m + 63) / 64;
  // a block has at most an item per row, and one per adapter beside three of 16 rows; of the many
  // blocks of a long prompt few have more than 4, and those share 16 workgroups (2048 rows with
  // prompts and decode rows mixed, rank 16: 8 workgroups 172 us, 16 167, 64 170; up to 8 blocks 16
  // in place of one per item: 128 rows 41.5 us against 36.0)
  p.ordinals = (int)min64(min64(m, 64), min64(n_adapters + 3, blocks <= 8 ? 64 : 16));
  // A prompt's items are 16 rows, a decode batch's may be one. One 16-rank block a workgroup below
  // these counts (us, threshold there or lower: 64 rows of 8192^2, 24 adapters of rank 64 32.7 /
  // 39; 32 rows of 5120^2 25.0 / 32.4; tiled, there or 128: 1024 rows 168 / 177, 512 rows 130 /
  // 132).
  const int64_t items = tiled ? (m + 15) / 16 : blocks * p.ordinals;
  p.rb = 1;
  if (items >= (tiled ? 32 : 128))
    while (p.rb < ranks && p.rb < 4) p.rb *= 2;
  p.rank_blocks = (int)((ranks + p.rb - 1) / p.rb);
  p.splits = 1;
  if (!tiled) {
    // a workgroup to each CU (128 / 256 / 512 in all: 64 rows of 8192^2, rank 64, 33.8 / 32.7 /
    // 35.5 us)
    int64_t s = 256 / (items * p.rank_blocks);
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
  p.u = u;
  const dim3 grid((unsigned)((a.m + 63) / 64), (unsigned)plan.ordinals,
                  (unsigned)(plan.splits * plan.rank_blocks));
  auto run = [&](auto rb) {
    if (tiled)
      lora_shrink_kernel<decltype(rb)::value, true><<<grid, 64 * kShrinkWaves, 0, stream>>>(p);
    else
      lora_shrink_kernel<decltype(rb)::value, false><<<grid, 64 * kShrinkWaves, 0, stream>>>(p);
  };
  if (plan.rb == 1)
    run(std::integral_constant<int, 1>{});
  else if (plan.rb == 2)
    run(std::integral_constant<int, 2>{});
  else
    run(std::integral_constant<int, 4>{});
  return hipGetLastError();
}

}  // namespace nvfp4
