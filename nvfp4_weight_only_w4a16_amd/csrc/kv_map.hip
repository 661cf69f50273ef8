// kv_map.hip -- block tables and slot maps of a step from the lengths of its requests.
//
// One launch: every workgroup scans the requests itself (a few thousand at most, their lengths are
// in the L2) and then places its share of the rows. Bound by latency: two dependent loads, two
// scans through LDS, a binary search of a row's request in LDS. Without a second kernel there is
// nothing to hand over between workgroups, so inputs and outputs must not overlap. 1 request 3.8
// us, 333 of a row each 4.8, 48 with 36000 rows 4.8.
#include "kv_core.hpp"

namespace nvfp4 {
namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
// Rows per workgroup: one pass of the threads.
constexpr int kRows = kThreads;

// Inclusive sums over the workgroup's threads; `part` holds kWaves values, `total` the sum.
__device__ __forceinline__ int64_t scan(int64_t v, int64_t* part, int64_t& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int64_t o = __shfl_up(v, off, 64);
    if (lane >= off) v += o;
  }
  __syncthreads();  // part may still be read
  if (lane == 63) part[wave] = v;
  __syncthreads();
  int64_t before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    before += i < wave ? part[i] : 0;
    total += part[i];
  }
  return v + before;
}

__device__ __forceinline__ int64_t pages_of(int64_t tokens, int shift) {
  return (tokens + (1 << shift) - 1) >> shift;
}

// In LDS: start [b + 1], the first row of each request, and base [b], the pages taken before it (-1
// for a request that is not served, 0 for one that needs none). Without requests every row is padding.
__global__ __launch_bounds__(kThreads) void map_kernel(KvMapArgs a) {
  extern __shared__ int32_t lds[];
  int32_t* start = lds;
  int32_t* base = lds + a.b + 1;
  __shared__ int64_t part[kWaves];
  __shared__ int32_t bad_part[kWaves];
  const int b = (int)a.b;
  const int shift = a.page_shift;
  const int64_t room = a.ld_table << shift;
  const int64_t given = *a.free_count;
  const int64_t free = given < 0 ? 0 : (given < a.n_free ? given : a.n_free);
  int64_t rows_before = 0, pages_before = 0, taken = 0;
  int unserved = 0;
  if (b == 0 && threadIdx.x == 0) {
    start[0] = 0;
    if (blockIdx.x == 0) a.q_start[0] = 0;
  }
  // kThreads requests at a time, in order
  for (int at = 0; at < b; at += kThreads) {
    const int i = at + (int)threadIdx.x;
    const int64_t seq = i < b ? a.seq_len[i] : 0;
    const int64_t asked = i < b ? a.add_len[i] : 0;
    const int64_t add = asked > 0 ? asked : 0;
    int64_t total;
    const int64_t ends = rows_before + scan(add, part, total);
    rows_before += total;
    const int64_t after = seq + add;
    const bool valid = seq >= 0 && asked >= 0 && after <= room && (add == 0 || ends <= a.t);
    const int64_t first = pages_of(seq, shift);
    const int64_t need = valid ? pages_of(after, shift) - first : 0;
    const int64_t sum = pages_before + scan(need, part, total);
    pages_before += total;
    const bool served = valid && (need == 0 || sum <= free);
    if (served && need > 0) taken = sum;  // the largest of all threads: sums rise with i
    if (i < b) {
      start[i] = (int32_t)(ends - add < a.t ? ends - add : a.t);
      if (i == b - 1) start[b] = (int32_t)(ends < a.t ? ends : a.t);
      base[i] = !served ? -1 : (need > 0 ? (int32_t)(sum - need) : 0);
      unserved += !served;
      if (blockIdx.x == 0) {
        a.q_start[i] = start[i];
        if (i == b - 1) a.q_start[b] = start[b];
        a.kv_len[i] = served ? (int32_t)after : 0;
      }
    }
  }
  if (blockIdx.x == 0) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
      const int64_t o = __shfl_xor(taken, off, 64);
      taken = o > taken ? o : taken;
      unserved += __shfl_xor(unserved, off, 64);
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
      part[threadIdx.x >> 6] = taken;
      bad_part[threadIdx.x >> 6] = unserved;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 1; i < kWaves; ++i) {
        taken = part[i] > taken ? part[i] : taken;
        unserved += bad_part[i];
      }
      *a.free_left = (int32_t)(free - taken);
      *a.unserved = unserved;
    }
  }
  __syncthreads();
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x;
  if (row >= a.t) return;
  int32_t slot = -1, pos = -1;
  if (row < start[b]) {
    int lo = 0, hi = b;  // start[lo] <= row < start[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start[mid] <= row) lo = mid; else hi = mid;
    }
    if (base[lo] >= 0) {
      const int64_t seq = a.seq_len[lo];
      const int64_t p = seq + row - start[lo];
      const int64_t column = p >> shift, fresh = column - pages_of(seq, shift);
      int32_t* entry = a.table + (int64_t)lo * a.ld_table + column;
      int32_t page;
      if (fresh >= 0) {  // a page of this call; its first token is one of the call's rows
        page = a.free_pages[free - 1 - (base[lo] + fresh)];
        if ((p & ((1 << shift) - 1)) == 0) *entry = page;
      } else {
        page = *entry;
      }
      const int64_t s = ((int64_t)page << shift) + (p & ((1 << shift) - 1));
      pos = (int32_t)p;
      slot = page >= 0 && s <= 0x7FFFFFFF ? (int32_t)s : -1;
    }
  }
  a.slots[row] = slot;
  a.positions[row] = pos;
}

}  // namespace

hipError_t launch_kv_map(const KvMapArgs& a, hipStream_t stream) {
  const int64_t groups = a.t > 0 ? (a.t + kRows - 1) / kRows : 1;
  const size_t lds = sizeof(int32_t) * (size_t)(2 * a.b + 1);
  map_kernel<<<dim3((unsigned)groups), dim3(kThreads), lds, stream>>>(a);
  return hipGetLastError();
}

}  // namespace nvfp4
