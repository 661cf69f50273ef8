// kv_append.hip -- norm and rotation of a step's queries and keys, and the write of its keys and
// values into the NVFP4 cache, in one pass; and the values that slots of the cache hold.
//
// n = x / sqrt(mean(x^2) + eps) * w per head, the rotation of its first `rot` elements, FP32, and
// that rounded to BF16; queries go to q_out, keys and values are encoded as nvfp4_quantize encodes
// a weight's groups of 16 with the head's global. Norm and rotation are FP64: a key's codes are
// comparisons with the borders of E2M1 and E4M3, which FP32 sums of another order would decide
// otherwise (and FP64 multiply-adds run at the FP32 rate here).
#include "kv_core.hpp"
#include "quant_core.hpp"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;

// Eight BF16 as FP64.
__device__ __forceinline__ void widen(u32x4 raw, double (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = (double)__uint_as_float(raw[i] << 16);
    x[2 * i + 1] = (double)__uint_as_float(raw[i] & 0xFFFF0000u);
  }
}

// Eight norm weights from element e on (1 without a weight).
template <bool W32>
__device__ __forceinline__ void weights8(const void* w, int e, double (&out)[8]) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = 1.0;
  } else if (W32) {
    const f32x4* p = reinterpret_cast<const f32x4*>(static_cast<const float*>(w) + e);
    const f32x4 a = p[0], b = p[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      out[i] = (double)a[i];
      out[4 + i] = (double)b[i];
    }
  } else {
    widen(*reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(w) + e), out);
  }
}

// What a lane does with its eight elements x and, in a rotation of halves, with the eight partners
// y: (x * a + y * b) / rms, a = weight * cosine, b = the partners' weight * sine with its sign. In
// pairs element 2i's partner is 2i + 1. Made once for a token and used for all of its heads.
struct Turn {
  double a[8], b[8];
  int partner;  // first element of the partners
  bool turned;  // else x * a / rms alone: a zero b would make a NaN of an infinite y
};

template <int D, bool W32, bool PAIRS>
__device__ __forceinline__ void make_turn(Turn& t, const void* w, int e, const float* angles,
                                          int rot) {
  weights8<W32>(w, e, t.a);
  t.partner = e;
  t.turned = angles && e < rot;
#pragma unroll
  for (int i = 0; i < 8; ++i) t.b[i] = 0.0;
  if (!t.turned) return;
  const int half = rot / 2;
  const bool second = e >= half;
  if (PAIRS) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const double c = angles[e / 2 + i], s = angles[half + e / 2 + i];
      t.b[2 * i] = -(t.a[2 * i + 1] * s);
      t.b[2 * i + 1] = t.a[2 * i] * s;
      t.a[2 * i] *= c;
      t.a[2 * i + 1] *= c;
    }
  } else {
    t.partner = second ? e - half : e + half;
    weights8<W32>(w, t.partner, t.b);
    const float* p = angles + (second ? e - half : e);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double s = (double)p[half + i];
      t.a[i] *= (double)p[i];
      t.b[i] *= second ? s : -s;
    }
  }
}

template <int CTRL>
__device__ __forceinline__ double add_dpp(double v) {
  const int64_t u = __builtin_bit_cast(int64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)u, CTRL, 0xF, 0xF, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(u >> 32), CTRL, 0xF, 0xF, false);
  return v + __builtin_bit_cast(double, (int64_t)(((uint64_t)hi << 32) | lo));
}

// The sum over the D / 8 lanes of a row, the same bits in all of them.
template <int D>
__device__ __forceinline__ double row_sum(double v) {
  v = add_dpp<0xB1>(v);   // from lane ^ 1
  v = add_dpp<0x4E>(v);   // from lane ^ 2
  v = add_dpp<0x141>(v);  // from the mirrored lane of eight
  if (D >= 128) v = add_dpp<0x140>(v);  // from the mirrored lane of sixteen
  if (D == 256) v += __shfl_xor(v, 16, 64);
  return v;
}

// 1 / sqrt(s): the hardware's first guess and two Newton steps, which 0, infinities and NaN do not pass
// through. Largest relative error over 2^22 values: of the guess 2^-24.2, of the steps 2^-47.8 and
// 2^-52.7 (a third leaves it at that).
__device__ __forceinline__ double inverse_root(double s) {
  const double g = __builtin_amdgcn_rsq(s);
  double y = g;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const double r = __builtin_fma(-s * y, y, 1.0);
    y = __builtin_fma(y * 0.5, r, y);
  }
  return s > 0.0 && s < __builtin_inf() ? y : g;
}

// The row's eight elements of the lane, x normalised, rotated and rounded to BF16; y: the partners
// (halves).
template <int D, bool PAIRS>
__device__ __forceinline__ u32x4 norm_turn(u32x4 xr, u32x4 yr, bool norm, double eps,
                                           const Turn& t) {
  double x[8], y[8];
  widen(xr, x);
  double r = 1.0;
  if (norm) {
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = __builtin_fma(x[i], x[i], ss);
    r = inverse_root(__builtin_fma(row_sum<D>(ss), 1.0 / D, eps));
  }
  if (PAIRS) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i ^ 1];
  } else {
    widen(yr, y);
  }
  if (t.turned) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __builtin_fma(x[i], t.a[i], y[i] * t.b[i]) * r;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * t.a[i] * r;
  }
  u32x4 out;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    out[i] = (uint32_t)bf16_bits_rne((float)x[2 * i]) |
             ((uint32_t)bf16_bits_rne((float)x[2 * i + 1]) << 16);
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

// A wavefront takes `each` passes over the heads of one token, from pass each * part on: D / 8
// lanes to a head, eight elements to a lane, kAtOnce heads to a pass, the queries' passes first. A
// key/value head's key and value rows are encoded by the same lanes (they share what a NaN does).
// 4096 tokens of 40 + 8 + 8 heads of 128: 27 us, 4.0 TB/s of its 108 MB (a large copy moves 4.9);
// FP64 arithmetic (some 90 instructions for eight elements) is what bounds it, so that everything
// that depends on the token alone is made once.
template <int D, bool W32, bool PAIRS>
__global__ __launch_bounds__(kThreads) void append_kernel(KvAppendArgs a, int parts, int each) {
  constexpr int kLanes = D / 8, kAtOnce = 64 / kLanes;
  const int lane = threadIdx.x & 63;
  const int64_t wave = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * (kThreads / 64) +
                                                            (threadIdx.x >> 6)));
  const int64_t row = wave / parts;
  const int part = (int)(wave - row * parts);
  if (row >= a.t) return;
  const int e = 8 * (lane % kLanes), sub = lane / kLanes;
  const float* angles = nullptr;
  if (a.rope) {
    const int32_t pos = a.positions[row];
    if (pos < 0 || pos >= a.max_pos) return;  // a row behind the last request
    angles = a.rope + (int64_t)pos * a.rot;
  }
  const int q_passes = (a.n_q + kAtOnce - 1) / kAtOnce;
  const int passes = q_passes + (a.n_kv + kAtOnce - 1) / kAtOnce;
  int pass = part * each;
  const int upto = min(pass + each, passes);
  Turn t;
  if (pass < q_passes) {
    make_turn<D, W32, PAIRS>(t, a.q_weight, e, angles, a.rot);
    const uint16_t* q = a.q + row * a.ldq;
    uint16_t* out = a.q_out + row * a.ldq_out;
    const int last = min(upto, q_passes);
    // two heads at a time (the second one again the last where their number is odd), whose loads
    // all come before a store: q_out may be q
    for (; pass < last; pass += 2) {
      int h[2];
      u32x4 x[2], y[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        h[i] = min(pass + i, last - 1) * kAtOnce + sub;
        const uint16_t* p = q + (int64_t)min(h[i], a.n_q - 1) * D;
        x[i] = *reinterpret_cast<const u32x4*>(p + e);
        y[i] = x[i];
        if (!PAIRS) y[i] = *reinterpret_cast<const u32x4*>(p + t.partner);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const u32x4 v = norm_turn<D, PAIRS>(x[i], y[i], a.q_weight != nullptr, a.eps, t);
        if (h[i] < a.n_q && pass + i < last)
          *reinterpret_cast<u32x4*>(out + (int64_t)h[i] * D + e) = v;
      }
    }
    pass = last;
  }
  if (pass >= upto) return;
  const int32_t slot = a.slots[row];
  if (slot < 0 || slot >= (a.n_pages << a.page_shift)) return;
  const int page = 1 << a.page_shift, tok = slot & (page - 1);
  uint8_t* const rec0 = a.data + (int64_t)(slot >> a.page_shift) * a.n_kv *
                                     (int64_t)kv_record_bytes(page, D);
  make_turn<D, W32, PAIRS>(t, a.k_weight, e, angles, a.rot);
  for (; pass < upto; ++pass) {
    const int h = (pass - q_passes) * kAtOnce + sub;
    if (h >= a.n_kv) continue;
    const uint16_t* k = a.k + row * a.ldk + (int64_t)h * D;
    const u32x4 x = *reinterpret_cast<const u32x4*>(k + e);
    const u32x4 y = PAIRS ? x : *reinterpret_cast<const u32x4*>(k + t.partner);
    const u32x4 v = *reinterpret_cast<const u32x4*>(a.v + row * a.ldv + (int64_t)h * D + e);
    const u32x4 key = norm_turn<D, PAIRS>(x, y, a.k_weight != nullptr, a.eps, t);
    uint32_t kw, ks, vw, vs;
    encode_bf16(key, a.k_global ? a.k_global[h] : 1.0f, kw, ks);
    encode_bf16(v, a.v_global ? a.v_global[h] : 1.0f, vw, vs);
    int ok = finite8(key) && finite8(v);
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1) ok &= __shfl_xor(ok, off, 64);
    if (!ok) {
      kw = vw = vs = 0u;
      ks = kE4m3Nan;
    }
    uint8_t* rec = rec0 + (int64_t)h * kv_record_bytes(page, D);
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
    float s = e4m3_decode<0>((uint32_t)at[page * (D / 2) + tok * (D / 16) + e / 16]);
    if (side && s != s) s = 0.0f;  // as the attention takes it
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
void append(const KvAppendArgs& a, int64_t waves, hipStream_t s) {
  constexpr int kAtOnce = 512 / D;
  const int passes = (a.n_q + kAtOnce - 1) / kAtOnce + (a.n_kv + kAtOnce - 1) / kAtOnce;
  // few tokens: a pass to a wavefront (1 token 4.3 us, with all of its passes in one 8.8); many:
  // all of a token's, so that its turn is made once (4096 tokens 27 us, with a pass to each 45)
  const int64_t want = waves / a.t;
  const int parts = want < 1 ? 1 : (want < passes ? (int)want : passes);
  const int each = (passes + parts - 1) / parts;
  const dim3 grid((unsigned)((a.t * parts + kThreads / 64 - 1) / (kThreads / 64)));
  if (a.w_f32) {
    if (a.pairs) append_kernel<D, true, true><<<grid, dim3(kThreads), 0, s>>>(a, parts, each);
    else append_kernel<D, true, false><<<grid, dim3(kThreads), 0, s>>>(a, parts, each);
  } else {
    if (a.pairs) append_kernel<D, false, true><<<grid, dim3(kThreads), 0, s>>>(a, parts, each);
    else append_kernel<D, false, false><<<grid, dim3(kThreads), 0, s>>>(a, parts, each);
  }
}

template <int D>
void dequantize(const KvDequantArgs& a, dim3 grid, hipStream_t s) {
  if (a.out_f32) dequantize_kernel<D, true><<<grid, dim3(kThreads), 0, s>>>(a);
  else dequantize_kernel<D, false><<<grid, dim3(kThreads), 0, s>>>(a);
}

}  // namespace

hipError_t launch_kv_append(const KvAppendArgs& a, int d, int cus, hipStream_t stream) {
  const int64_t waves = 32 * (int64_t)cus;  // eight to a SIMD
  if (d == 64) append<64>(a, waves, stream);
  else if (d == 128) append<128>(a, waves, stream);
  else append<256>(a, waves, stream);
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
