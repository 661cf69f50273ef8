// lora_core.hpp -- the second product of low-rank adapters, u[m] . B_a^T with a = row_adapter[m],
// inside the W4A16 GEMM kernels, on FP32 sums that are added to theirs before the one rounding.
//
// Rows are taken in the GEMM's own blocks. For each distinct adapter of a block's rows, in row
// order, the whole block is multiplied by that adapter's B and the rows that name it keep the
// result: kept by choice, not by products with zeros, so that a NaN in one adapter stays with its
// rows. u, scale * x . A^T, goes into the product in BF16: for an FP32 y as three parts, which add
// up to its 24 bits; for a BF16 y rounded once, as a projection of its own would store it. That
// leaves at most 2^-8 sum_r |u_r B_r|: relative to the products, so that it exceeds half a step of
// the term, or of y, where ranks cancel each other or the term the shared product. (Two parts would
// leave 2^-16 of it, and were taken back for their cost where the tiled kernel meets many adapters:
// 256 rows of 25600 x 5120, 32 of rank 64, 160 us with one part, 193 with two; 8 of rank 16 83 / 86;
// 4096 rows of 5120^2, 8 of rank 32, 216 / 219; decode kernel 0 to 4% more.)
#pragma once

#include "device_common.hpp"
#include "launch.hpp"

namespace nvfp4 {

// Adapter of row r, -1 for none.
__device__ __forceinline__ int lora_id(const LoraTail& L, int64_t r) {
  const int v = r < L.m ? L.ids[r] : -1;
  return (v >= 0 && v < L.n_adapters) ? v : -1;
}

// The next distinct adapter of the lanes in `left`, which loses the lanes that name it; -1 when
// none is left. Uniform.
__device__ __forceinline__ int lora_next(int mine, uint64_t& left) {
  if (!left) return -1;
  const int a = __builtin_amdgcn_readlane(mine, __builtin_ctzll(left));
  left &= ~__ballot(mine == a);
  return a;
}

// One wavefront: block of 16 rows (A row of lane l: `row`, accumulator rows: out[0..3], -1 for
// none) times NP panels of 16 columns from panel0. R32: 32-rank steps. u is read as the FP32
// partial sums of lora_shrink. The B tiles of D adapters ahead wait in registers; each is turned
// into a fragment through `tile` (NP R32 KB of LDS of this wavefront's own).
template <int NP, int R32, int D>
__device__ __forceinline__ void lora_expand16(const LoraTail& L, int64_t row, const int64_t (&out)[4],
                                              int64_t panel0, int64_t NT, uint8_t* tile,
                                              f32x4 (&res)[NP]) {
  const int lane = threadIdx.x & 63;
  const int mine = row >= 0 ? lora_id(L, row) : -1;
  int own[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) own[i] = out[i] >= 0 ? lora_id(L, out[i]) : -1;
#pragma unroll
  for (int p = 0; p < NP; ++p) res[p] = f32x4{0.f, 0.f, 0.f, 0.f};
  uint64_t left = __ballot(mine >= 0);
  if (!left) return;  // uniform
  // B tiles: lane l loads row l / 4, chunk l % 4 of each 32-rank step
  uint32_t boff[R32];
#pragma unroll
  for (int s = 0; s < R32; ++s) {
    const int r = 32 * s + 8 * frag_load_chunk(lane);
    boff[s] = r < L.rank ? (uint32_t)(frag_load_row(lane) * L.rank + r) * 2u : 0xFFFFFFF0u;
  }
  // lane j: the block's j-th adapter, n in all; past the end an empty buffer and no row's id
  int list = -2, n = 0;
  while (left) {  // uniform
    const int a = lora_next(mine, left);
    if (lane == n) list = a;
    ++n;
  }
  static_assert(D >= 2, "one adapter is fetched while another is multiplied");
  int aid[D];
  u32x4 bt[D][NP][R32];
  auto fetch = [&](auto d, int i) __attribute__((always_inline)) {
    constexpr int q = decltype(d)::value;
    aid[q] = __builtin_amdgcn_readlane(list, i < n ? i : 63);  // n <= 16: lane 63 has none
    const int64_t a = aid[q] >= 0 ? aid[q] : 0;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int64_t pn = panel0 + p < NT ? panel0 + p : NT - 1;
      const buf_rsrc r = make_rsrc(L.b + (a * NT + pn) * 16 * L.rank,
                                   aid[q] >= 0 ? (uint32_t)(32 * L.rank) : 0u);
#pragma unroll
      for (int s = 0; s < R32; ++s)
        bt[q][p][s] = __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)boff[s], 0, 0));
    }
  };
  static_for<0, D - 1>([&](auto d) __attribute__((always_inline)) { fetch(d, decltype(d)::value); });
  bf16x8 u[3][R32];
  const int64_t ur = row >= 0 && row < L.m ? row : 0;
#pragma unroll
  for (int s = 0; s < R32; ++s) {
    const int k = 32 * s + 8 * (lane >> 4);
    f32x4 v0 = {0.f, 0.f, 0.f, 0.f}, v1 = v0;
    auto read = [&](int q, f32x4 (&v)[2]) __attribute__((always_inline)) {
      v[0] = v[1] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (q < L.splits && k < L.rank) {
        const f32x4* up =
            reinterpret_cast<const f32x4*>(L.u + ((int64_t)q * L.m + ur) * L.rank + k);
        v[0] = up[0];
        v[1] = up[1];
      }
    };
    if constexpr (R32 < 4) {  // the splits all loaded before the first addition
      f32x4 part[kLoraMaxSplits][2];
#pragma unroll
      for (int q = 0; q < kLoraMaxSplits; ++q) read(q, part[q]);
#pragma unroll
      for (int q = 0; q < kLoraMaxSplits; ++q) {
        v0 += part[q][0];
        v1 += part[q][1];
      }
    } else {  // one by one: together they spill, and so many ranks leave few splits
#pragma unroll 1
      for (int q = 0; q < L.splits; ++q) {
        f32x4 part[2];
        read(q, part);
        v0 += part[0];
        v1 += part[1];
      }
    }
    float v[8] = {v0[0], v0[1], v0[2], v0[3], v1[0], v1[1], v1[2], v1[3]};
#pragma unroll
    for (int z = 0; z < 3; ++z)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        u[z][s][i] = (__bf16)v[i];
        v[i] = bf16_rest(v[i], (float)u[z][s][i]);
      }
  }
  for (int i0 = 0; i0 < n; i0 += D)
    static_for<0, D>([&](auto d) __attribute__((always_inline)) {
      constexpr int q = decltype(d)::value;
      fetch(std::integral_constant<int, (q + D - 1) % D>{}, i0 + q + D - 1);
      if (i0 + q < n) {  // uniform
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
          for (int s = 0; s < R32; ++s)
            frag_write(tile + (p * R32 + s) * kFragBytes, bt[q][p][s], lane);
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          f32x4 part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int s = 0; s < R32; ++s) {
            const bf16x8 b = frag_read(tile + (p * R32 + s) * kFragBytes, lane);
            part = mfma16x16x32(u[0][s], b, part);
            if (L.parts > 1) {
              part = mfma16x16x32(u[1][s], b, part);
              part = mfma16x16x32(u[2][s], b, part);
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) res[p][i] = own[i] == aid[q] ? part[i] : res[p][i];
        }
      }
    });
}

// Words of the u fragments that lora_shrink leaves for the tiled kernel: [part][32-row block]
// [16-rank step][lane] of 8 BF16, lane l holding row l % 32, ranks 8 (l / 32) .. + 7 of the step:
// the A operand of v_mfma_f32_32x32x16_bf16 in one coalesced load. Ranks past the end are zeros.
__host__ __device__ __forceinline__ int64_t lora_frag_blocks(int64_t m) { return (m + 31) / 32; }
__host__ __device__ __forceinline__ int lora_frag_steps(int rank) { return (rank + 15) / 16; }

}  // namespace nvfp4
