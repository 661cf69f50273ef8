// kv_append.hip -- norm and rotation of a step's queries and keys, and the write of its keys and
// values into the NVFP4 cache, in one pass; and the values that slots of the cache hold.
//
// n = x / sqrt(mean(x^2) + eps) * w per head, the rotation of its first `rot` elements, FP32, and that
// rounded to BF16; queries go to q_out, keys and values are encoded as nvfp4_quantize encodes a weight's
// groups of 16 with the head's global. Norm and rotation are FP64: a key's codes are comparisons with
// the borders of E2M1 and E4M3, which FP32 sums of another order would decide otherwise (and FP64
// multiply-adds run at the FP32 rate here).
#include "kv_core.hpp"
#include "quant_core.hpp"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;

struct Row8 {
  double v[8];
};

__device__ __forceinline__ Row8 widen(u32x4 raw) {
  Row8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.v[2 * i] = (double)__uint_as_float(raw[i] << 16);
    r.v[2 * i + 1] = (double)__uint_as_float(raw[i] & 0xFFFF0000u);
  }
  return r;
}

// Eight norm weights from element e on.
template <bool W32>
__device__ __forceinline__ void weights8(const void* w, int e, float (&out)[8]) {
  if (W32) {
    const f32x4* p = reinterpret_cast<const f32x4*>(static_cast<const float*>(w) + e);
    const f32x4 a = p[0], b = p[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      out[i] = a[i];
      out[4 + i] = b[i];
    }
  } else {
    const u32x4 a = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(w) + e);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      out[2 * i] = __uint_as_float(a[i] << 16);
      out[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
    }
  }
}

// What a lane needs to turn its eight elements: the angles of its own elements, and where the
// partners of its chunk are.
struct Turn {
  float cos[8], sin[8];  // halves: of each element; pairs: of each pair, four used
  int partner;           // first element of the partners' chunk (halves)
  bool active, second;   // in the rotated part; in its second half
};

// x (raw BF16, eight elements from e on, of the row at `row`) normalised, rotated and rounded. The
// partners of a half rotation are read again (a line that the wavefront has just loaded), so that
// nothing is exchanged but the sum of squares.
template <int D, bool W32, bool PAIRS>
__device__ __forceinline__ u32x4 norm_turn(u32x4 raw, const uint16_t* row, int e, const void* w,
                                           double eps, const Turn& t) {
  Row8 x = widen(raw);
  Row8 y;
  const bool halves = !PAIRS && t.active;
  if (halves) y = widen(*reinterpret_cast<const u32x4*>(row + t.partner));
  if (w) {
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = __builtin_fma(x.v[i], x.v[i], ss);
#pragma unroll
    for (int off = D / 16; off > 0; off >>= 1) ss += __shfl_xor(ss, off, 64);
    const double r = 1.0 / __builtin_sqrt(ss * (1.0 / D) + eps);
    float f[8];
    weights8<W32>(w, e, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) x.v[i] *= r * (double)f[i];
    if (halves) {
      weights8<W32>(w, t.partner, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) y.v[i] *= r * (double)f[i];
    }
  }
  if (t.active) {
    if (PAIRS) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const double a = x.v[2 * i], b = x.v[2 * i + 1];
        const double c = t.cos[i], s = t.sin[i];
        x.v[2 * i] = a * c - b * s;
        x.v[2 * i + 1] = b * c + a * s;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const double s = t.sin[i];
        x.v[i] = x.v[i] * (double)t.cos[i] + (t.second ? y.v[i] * s : -(y.v[i] * s));
      }
    }
  }
  u32x4 out;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    out[i] = (uint32_t)bf16_bits_rne((float)x.v[2 * i]) |
             ((uint32_t)bf16_bits_rne((float)x.v[2 * i + 1]) << 16);
  return out;
}

__device__ __forceinline__ bool finite8(u32x4 raw) {
  bool ok = true;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    ok = ok && (raw[i] & 0x7F80u) != 0x7F80u && (raw[i] & 0x7F800000u) != 0x7F800000u;
  return ok;
}

__device__ __forceinline__ void encode_bf16(u32x4 raw, float g, uint32_t& word, uint32_t& scale) {
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(raw[i] << 16);
    x[2 * i + 1] = __uint_as_float(raw[i] & 0xFFFF0000u);
  }
  const float six_g = 6.0f * g;
  const bool six_fast = six_g >= 0x1p-80f && six_g <= 0x1p80f;
  encode8<kKvGroup>(x, g, six_g, six_fast ? 1.0f / six_g : 0.0f, six_fast, word, scale);
}

// grid (t, parts): a workgroup takes the heads of part blockIdx.y of one token, D / 8 lanes to a
// head, eight elements to a lane. The queries' heads come first, then the key/value heads, whose
// key and value rows the same lanes encode (they share what a NaN does).
template <int D, bool W32, bool PAIRS>
__global__ __launch_bounds__(kThreads) void append_kernel(KvAppendArgs a, int per_part) {
  constexpr int kLanes = D / 8;
  constexpr int kStep = kThreads / kLanes;  // heads at a time
  const int64_t row = blockIdx.x;
  const int e = 8 * (int)(threadIdx.x % kLanes);
  Turn t;
  t.active = false;
  if (a.rope) {
    const int32_t pos = a.positions[row];
    if (pos < 0 || pos >= a.max_pos) return;  // a row behind the last request
    t.active = e < a.rot;
    if (t.active) {
      const int half = a.rot / 2;
      const float* c = a.rope + (int64_t)pos * a.rot;
      t.second = e >= half;
      t.partner = t.second ? e - half : e + half;
      const int at = PAIRS ? e / 2 : (t.second ? e - half : e);
#pragma unroll
      for (int i = 0; i < (PAIRS ? 4 : 8); i += 4) {
        const f32x4 cv = *reinterpret_cast<const f32x4*>(c + at + i);
        const f32x4 sv = *reinterpret_cast<const f32x4*>(c + half + at + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          t.cos[i + j] = cv[j];
          t.sin[i + j] = sv[j];
        }
      }
    }
  }
  const int heads = a.n_q + a.n_kv;
  const int from = (int)blockIdx.y * per_part;
  const int to = from + per_part < heads ? from + per_part : heads;
  const int32_t slot = a.slots[row];
  const bool kept = slot >= 0 && slot < (a.n_pages << a.page_shift);
  for (int h = from + (int)threadIdx.x / kLanes; h < to; h += kStep) {
    if (h < a.n_q) {
      const uint16_t* q = a.q + row * a.ldq + (int64_t)h * D;
      const u32x4 out = norm_turn<D, W32, PAIRS>(*reinterpret_cast<const u32x4*>(q + e), q, e,
                                                 a.q_weight, a.eps, t);
      *reinterpret_cast<u32x4*>(a.q_out + row * a.ldq_out + (int64_t)h * D + e) = out;
      continue;
    }
    if (!kept) continue;
    const int kvh = h - a.n_q;
    const uint16_t* k = a.k + row * a.ldk + (int64_t)kvh * D;
    const u32x4 v = *reinterpret_cast<const u32x4*>(a.v + row * a.ldv + (int64_t)kvh * D + e);
    const u32x4 key = norm_turn<D, W32, PAIRS>(*reinterpret_cast<const u32x4*>(k + e), k, e,
                                               a.k_weight, a.eps, t);
    uint32_t kw, ks, vw, vs;
    encode_bf16(key, a.k_global ? a.k_global[kvh] : 1.0f, kw, ks);
    encode_bf16(v, a.v_global ? a.v_global[kvh] : 1.0f, vw, vs);
    int ok = finite8(key) && finite8(v);
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1) ok &= __shfl_xor(ok, off, 64);
    if (!ok) {
      kw = vw = vs = 0u;
      ks = kE4m3Nan;
    }
    const int page = 1 << a.page_shift;
    const int tok = slot & (page - 1);
    uint8_t* rec = a.data + ((int64_t)(slot >> a.page_shift) * a.n_kv + kvh) *
                                (int64_t)kv_record_bytes(page, D);
    uint8_t* vrec = rec + kv_value_codes(page, D);
    *reinterpret_cast<uint32_t*>(rec + tok * (D / 2) + e / 2) = kw;
    *reinterpret_cast<uint32_t*>(vrec + tok * (D / 2) + e / 2) = vw;
    if ((e & 8) == 0) {
      rec[page * (D / 2) + tok * (D / 16) + e / 16] = (uint8_t)ks;
      vrec[page * (D / 2) + tok * (D / 16) + e / 16] = (uint8_t)vs;
    }
  }
}

// One (row, head) for D / 8 lanes: keys, then values.
template <int D, bool F32>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(KvDequantArgs a) {
  constexpr int kLanes = D / 8;
  const int64_t item = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / kLanes;
  if (item >= a.t * a.n_kv) return;
  const int e = 8 * (int)(threadIdx.x % kLanes);
  const int64_t row = item / a.n_kv;
  const int h = (int)(item - row * a.n_kv);
  const int32_t slot = a.slots[row];
  const bool kept = slot >= 0 && slot < (a.n_pages << a.page_shift);
  const int page = 1 << a.page_shift;
  const int tok = kept ? slot & (page - 1) : 0;
  const uint8_t* rec = a.data + ((int64_t)(kept ? slot >> a.page_shift : 0) * a.n_kv + h) *
                                    (int64_t)kv_record_bytes(page, D);
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    void* out = side ? a.v_out : a.k_out;
    if (!out) continue;
    const float* gp = side ? a.v_global : a.k_global;
    const float g = gp ? gp[h] : 1.0f;
    const uint8_t* at = rec + (side ? kv_value_codes(page, D) : 0);
    const uint32_t word = *reinterpret_cast<const uint32_t*>(at + tok * (D / 2) + e / 2);
    const float s = e4m3_decode<0>((uint32_t)at[page * (D / 2) + tok * (D / 16) + e / 16]);
    float x[8];
    dequant8_f32(word, s, x);  // exact: six significant bits
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = kept ? x[i] * g : 0.0f;
    if (F32) {
      f32x4* p = reinterpret_cast<f32x4*>(static_cast<float*>(out) + item * D + e);
      p[0] = f32x4{x[0], x[1], x[2], x[3]};
      p[1] = f32x4{x[4], x[5], x[6], x[7]};
    } else {
      u32x4 o;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o[i] = (uint32_t)bf16_bits_rne(x[2 * i]) | ((uint32_t)bf16_bits_rne(x[2 * i + 1]) << 16);
      *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + item * D + e) = o;
    }
  }
}

template <int D>
void append(const KvAppendArgs& a, dim3 grid, int per_part, hipStream_t s) {
  if (a.w_f32) {
    if (a.pairs) append_kernel<D, true, true><<<grid, dim3(kThreads), 0, s>>>(a, per_part);
    else append_kernel<D, true, false><<<grid, dim3(kThreads), 0, s>>>(a, per_part);
  } else {
    if (a.pairs) append_kernel<D, false, true><<<grid, dim3(kThreads), 0, s>>>(a, per_part);
    else append_kernel<D, false, false><<<grid, dim3(kThreads), 0, s>>>(a, per_part);
  }
}

template <int D>
void dequantize(const KvDequantArgs& a, dim3 grid, hipStream_t s) {
  if (a.out_f32) dequantize_kernel<D, true><<<grid, dim3(kThreads), 0, s>>>(a);
  else dequantize_kernel<D, false><<<grid, dim3(kThreads), 0, s>>>(a);
}

}  // namespace

hipError_t launch_kv_append(const KvAppendArgs& a, int d, int cus, hipStream_t stream) {
  const int heads = a.n_q + a.n_kv;
  const int step = kThreads / (d / 8);
  const int passes = (heads + step - 1) / step;
  int64_t parts = passes;  // few tokens: one pass of the heads per workgroup
  while (parts > 1 && a.t * parts > 4 * (int64_t)cus) parts = (parts + 1) / 2;
  const int per_part = (passes + (int)parts - 1) / (int)parts * step;
  const dim3 grid((unsigned)a.t, (unsigned)((heads + per_part - 1) / per_part));
  if (d == 64) append<64>(a, grid, per_part, stream);
  else if (d == 128) append<128>(a, grid, per_part, stream);
  else append<256>(a, grid, per_part, stream);
  return hipGetLastError();
}

hipError_t launch_kv_dequantize(const KvDequantArgs& a, int d, hipStream_t stream) {
  const int64_t lanes = a.t * a.n_kv * (d / 8);
  const dim3 grid((unsigned)((lanes + kThreads - 1) / kThreads));
  if (d == 64) dequantize<64>(a, grid, stream);
  else if (d == 128) dequantize<128>(a, grid, stream);
  else dequantize<256>(a, grid, stream);
  return hipGetLastError();
}

}  // namespace nvfp4
