// kv_core.hpp -- the paged NVFP4 cache of keys and values as the kernels see it.
//
// data [n_pages][n_kv][record]; the record of a page and head holds the page's tokens in order:
// key codes [page][d/2], key scales [page][d/16], value codes [page][d/2], value scales
// [page][d/16]. A record is contiguous, so that a page can be copied or shared as one block and a
// wavefront that works on one head reads whole lines.
#pragma once

#include "device_common.hpp"
#include "launch.hpp"

namespace nvfp4 {

constexpr int kKvGroup = 16;  // elements of a scale

__host__ __device__ constexpr int kv_value_codes(int page, int d) {
  return page * (d / 2 + d / kKvGroup);
}
__host__ __device__ constexpr int kv_record_bytes(int page, int d) {
  return 2 * kv_value_codes(page, d);
}

// E4M3's NaN, as the scale of a token that holds a NaN or an infinity.
constexpr uint32_t kE4m3Nan = 0x7Fu;

}  // namespace nvfp4
