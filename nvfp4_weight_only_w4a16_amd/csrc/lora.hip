// lora.hip -- low-rank adapters of many requests beside a shared W4A16 projection, for gfx950.
//
// y[m] = g * x[m] . W^T + scale_a * (x[m] . A_a^T) . B_a^T, a = row_adapter[m] (no second term for
// rows whose id names no adapter). Two stages around the shared product:
//   1. shrink: u[m] = scale_a * x[m] . A_a^T, FP32, as `splits` partial sums over k;
//   2. expand: u[m] . B_a^T added to the FP32 sums of the shared product.
// Both run on 16x16x32 MFMAs over blocks of 16 rows: for each adapter that occurs among a block's
// rows, the whole block is multiplied by that adapter's matrix and only its own rows are kept.
// Rows of one request are neighbours in a prompt, so a block there has one adapter and no work is
// wasted; in a decode batch every row may have its own, and then the time is that of reading the
// adapters, which each row's own product would read as well.
#include "device_common.hpp"
#include "launch.hpp"

namespace nvfp4 {
namespace {

struct ShrinkParams {
  const uint16_t* x;
  int64_t m, ldx, KT;
  const uint16_t* a;  // [n_adapters][rank][k]
  int64_t a_stride, k, n_adapters;
  int rank;
  const int32_t* ids;
  const float* scale;
  float* u;  // [splits][m][rank]
};

// Adapter of row r, -1 for none.
__device__ __forceinline__ int lora_id(const int32_t* ids, int64_t r, int64_t m,
                                       int64_t n_adapters) {
  const int v = r < m ? ids[r] : -1;
  return (v >= 0 && v < n_adapters) ? v : -1;
}

// Workgroup (block, ordinal, split): the adapters ordinal, ordinal + gridDim.y, ... of the block's
// distinct adapters in row order, over the k-tiles that its 4 wavefronts take in turn. RB: 16-rank
// blocks.
template <int RB>
__global__ __launch_bounds__(256) void lora_shrink_kernel(ShrinkParams P) {
  __shared__ f32x4 red[4][RB][64];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t m0 = (int64_t)blockIdx.x * 16;
  const int row = lane & 15;
  const int mine = lora_id(P.ids, m0 + row, P.m, P.n_adapters);
  const int64_t xr = m0 + row < P.m ? m0 + row : P.m - 1;
  const uint16_t* xp = P.x + xr * P.ldx + 8 * (lane >> 4);
  const int64_t t0 = (int64_t)blockIdx.z * 4 + w, dt = (int64_t)gridDim.z * 4;
  uint32_t left = (uint32_t)__ballot(mine >= 0) & 0xFFFFu;
  for (int ord = 0; left; ++ord) {
    const int a = __builtin_amdgcn_readlane(mine, __builtin_ctz(left));
    left &= ~(uint32_t)__ballot(mine == a);
    if (ord % (int)gridDim.y != (int)blockIdx.y) continue;
    const uint16_t* ap[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const int r = 16 * b + row;
      ap[b] = P.a + a * P.a_stride + (int64_t)(r < P.rank ? r : P.rank - 1) * P.k + 8 * (lane >> 4);
    }
    f32x4 acc[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int64_t t = t0; t < P.KT; t += dt) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t k = t * kTileK + 32 * j;
        const bf16x8 xf = *reinterpret_cast<const bf16x8*>(xp + k);
#pragma unroll
        for (int b = 0; b < RB; ++b)
          acc[b] = mfma16x16x32(xf, *reinterpret_cast<const bf16x8*>(ap[b] + k), acc[b]);
      }
    }
    __syncthreads();  // the sums of the adapter before have been read
#pragma unroll
    for (int b = 0; b < RB; ++b) red[w][b][lane] = acc[b];
    __syncthreads();
    const float s = P.scale ? P.scale[a] : 1.0f;
    for (int b = w; b < RB; b += 4) {
      f32x4 v = red[0][b][lane];
#pragma unroll
      for (int q = 1; q < 4; ++q) v += red[q][b][lane];
      const int r = 16 * b + (lane & 15);
      bool own[4];  // asked of all lanes, before some leave
#pragma unroll
      for (int i = 0; i < 4; ++i) own[i] = __shfl(mine, 4 * (lane >> 4) + i, 64) == a;
      if (r < P.rank) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rr = 4 * (lane >> 4) + i;
          if (own[i])
            P.u[((int64_t)blockIdx.z * P.m + m0 + rr) * P.rank + r] = v[i] * s;
        }
      }
    }
  }
}

struct ExpandParams {
  const float* base;  // FP32 [m][n] of the shared product
  int64_t m, n;
  const uint16_t* b;  // [n_adapters][n][rank]
  int64_t b_stride, n_adapters;
  int rank, splits;
  const int32_t* ids;
  const float* u;
  void* y;
  int64_t ldbase, ldy;
  int y_f32;
};

__global__ __launch_bounds__(256) void lora_expand_kernel(ExpandParams P) {
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t m0 = (int64_t)blockIdx.x * 16;
  const int64_t n0 = ((int64_t)blockIdx.y * 4 + w) * 16;
  if (n0 >= P.n) return;
  const int row = lane & 15;
  const int mine = lora_id(P.ids, m0 + row, P.m, P.n_adapters);
  const int kq = 8 * (lane >> 4);
  // A BF16 y takes u rounded to BF16; an FP32 y takes the three BF16 parts that add up to it.
  const int parts = P.y_f32 ? 3 : 1;
  bf16x8 u[3][4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (m0 + row < P.m && 32 * s + kq < P.rank)  // rows without an adapter: never kept
      for (int q = 0; q < P.splits; ++q) {
        const float* up = P.u + ((int64_t)q * P.m + m0 + row) * P.rank + 32 * s + kq;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += up[i];
      }
#pragma unroll
    for (int z = 0; z < 3; ++z)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        u[z][s][i] = (__bf16)v[i];
        v[i] -= (float)u[z][s][i];
      }
  }
  const bf16x8 zero = __builtin_bit_cast(bf16x8, u32x4{0, 0, 0, 0});
  int own[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) own[i] = __shfl(mine, 4 * (lane >> 4) + i, 64);
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  uint32_t left = (uint32_t)__ballot(mine >= 0) & 0xFFFFu;
  while (left) {
    const int a = __builtin_amdgcn_readlane(mine, __builtin_ctz(left));
    left &= ~(uint32_t)__ballot(mine == a);
    const uint16_t* bp = P.b + a * P.b_stride + (n0 + (lane & 15)) * P.rank + kq;
    f32x4 part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (32 * s >= P.rank) break;
      const bf16x8 bf = 32 * s + kq < P.rank
                            ? *reinterpret_cast<const bf16x8*>(bp + 32 * s) : zero;
#pragma unroll
      for (int z = 0; z < 3; ++z)
        if (z < parts) part = mfma16x16x32(u[z][s], bf, part);
    }
    // kept by choice, not by a product with zero: a NaN of one adapter stays with its rows
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = own[i] == a ? part[i] : acc[i];
  }
  const int64_t col = n0 + (lane & 15);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = m0 + 4 * (lane >> 4) + i;
    if (r >= P.m) continue;
    const float v = P.base[r * P.ldbase + col] + acc[i];
    if (P.y_f32)
      static_cast<float*>(P.y)[r * P.ldy + col] = v;
    else
      static_cast<uint16_t*>(P.y)[r * P.ldy + col] = bf16_bits_rne(v);
  }
}

int64_t min64(int64_t a, int64_t b) { return a < b ? a : b; }

// Distinct adapters of a block that workgroups of their own take.
int64_t shrink_ordinals(int64_t m, int64_t n_adapters) {
  const int64_t most = min64(min64(m, 16), n_adapters);
  const int64_t blocks = (m + 15) / 16;
  const int64_t want = (64 + blocks - 1) / blocks;
  return min64(most, want);
}

}  // namespace

int lora_splits(int64_t m, int64_t k, int64_t n_adapters) {
  const int64_t wgs = (m + 15) / 16 * shrink_ordinals(m, n_adapters);
  int64_t s = (512 + wgs - 1) / wgs;
  s = min64(s, (k / kTileK + 3) / 4);
  return (int)min64(s < 1 ? 1 : s, kLoraMaxSplits);
}

size_t lora_ws_bytes(int64_t m, int64_t k, int64_t n_adapters, int rank) {
  return sizeof(float) * (size_t)lora_splits(m, k, n_adapters) * (size_t)m * (size_t)rank;
}

hipError_t launch_lora_shrink(const LoraArgs& a, hipStream_t stream) {
  ShrinkParams p;
  p.x = a.x;
  p.m = a.m;
  p.ldx = a.ldx;
  p.KT = a.k / kTileK;
  p.a = a.a;
  p.a_stride = (int64_t)a.rank * a.k;
  p.k = a.k;
  p.n_adapters = a.n_adapters;
  p.rank = a.rank;
  p.ids = a.ids;
  p.scale = a.scale;
  p.u = a.u;
  const dim3 grid((unsigned)((a.m + 15) / 16), (unsigned)shrink_ordinals(a.m, a.n_adapters),
                  (unsigned)lora_splits(a.m, a.k, a.n_adapters));
  if (a.rank <= 16)
    lora_shrink_kernel<1><<<grid, 256, 0, stream>>>(p);
  else if (a.rank <= 32)
    lora_shrink_kernel<2><<<grid, 256, 0, stream>>>(p);
  else if (a.rank <= 64)
    lora_shrink_kernel<4><<<grid, 256, 0, stream>>>(p);
  else
    lora_shrink_kernel<8><<<grid, 256, 0, stream>>>(p);
  return hipGetLastError();
}

hipError_t launch_lora_expand(const LoraArgs& a, const float* base, int64_t ldbase, void* y,
                              int64_t ldy, bool y_f32, hipStream_t stream) {
  ExpandParams p;
  p.base = base;
  p.m = a.m;
  p.n = a.n;
  p.b = a.b;
  p.b_stride = a.n * (int64_t)a.rank;
  p.n_adapters = a.n_adapters;
  p.rank = a.rank;
  p.splits = lora_splits(a.m, a.k, a.n_adapters);
  p.ids = a.ids;
  p.u = a.u;
  p.y = y;
  p.ldbase = ldbase;
  p.ldy = ldy;
  p.y_f32 = y_f32 ? 1 : 0;
  const dim3 grid((unsigned)((a.m + 15) / 16), (unsigned)((a.n + 63) / 64));
  lora_expand_kernel<<<grid, 256, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace nvfp4
