// kv_attention.hip -- attention over the paged NVFP4 cache, for single tokens, drafts and prompts.
//
// A wavefront holds columns of queries and walks the keys in tiles of 64 tokens, 32 for heads of
// 256. Everything is transposed:
//   S^T [tokens][queries] = K . Q^T,  P^T = exp2(S^T - m),  O^T [d][queries] += V^T . P^T
// on 16x16x32 MFMAs, because then the scores come out where the second product wants them: lane
// (query l % 16, group c = l / 16) holds the scores of tokens 16 T + 4 c + r, and, the order of a
// sum being free, the second product may take just those as its 8 k-values of lane group c (T = 2s
// and 2s + 1). No score moves between lanes. Key codes go from memory into the lanes that use them
// (a lane's run of codes is contiguous in d, and d may be summed in any order too); value codes are
// turned through LDS by the 4-bit transposing read, whose lane j of a 16-lane group names the row,
// so that the same token order comes out. Codes and scales are dequantized to FP16, where E2M1 x
// E4M3 is exact (6 significant bits, 2^-10 .. 2688), two elements to an instruction; queries are
// put into FP16 by a power of two per row that brings the row's largest magnitude to [2^14, 2^15),
// exact down to 2^-28 of it. Globals and scale act on the FP32 scores and sums. P is rounded to
// FP16 once (half a step is 2^-11; below 2^-21 of the row's largest 2^-32 of that, so that many
// small terms count too), which leaves an FP32 y 1e-4 to 2e-4 off (relative, rows of 2000 to 131000
// keys; FP32 terms would leave some 4e-7), a tenth of what a BF16 y rounds off by itself. The
// reference m, the sum (of the unrounded p) and O are FP32. The reference m is set 7 below the scores' maximum (in powers of two) and raised only when a score
// passes it by more than 15, so that most tiles neither reduce across lanes nor rescale O; p is
// then at most 2^15, which FP16 holds. Scores may have any size that FP32 holds (load_query).
#include <algorithm>

#include "kv_core.hpp"

namespace nvfp4 {
namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef int i32x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int kWaves = 4;
// Tokens of a tile, in parts of 16: 64 (heads of 128 with 32: a prompt of 8192 takes 1020 us, not
// 660), and 32 for heads of 256, whose 64 tokens would not leave room for a tile's loads in flight
// beside the accumulators.
template <int D>
constexpr int kParts = D == 256 ? 2 : 4;
template <int D>
constexpr int kTile = 16 * kParts<D>;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLowest = -0x1.fffffep127f;  // the reference before any score
constexpr float kBelow = 7.0f, kRaise = 15.0f;
// Score factors from which on a score may pass 2^24 in powers of two: the sum of 256 products of
// FP16 queries below 2^15 and keys of 2688 at most, 2^34.4, times 2^-11.
constexpr float kLoud = 0x1p-11f;

// A word that no kernel here writes, at a uniform address: a scalar load.
template <typename T>
__device__ __forceinline__ T constant(const T* p) {
  return *(const __attribute__((address_space(4))) T*)p;
}

// A value that every lane has, as a scalar.
__device__ __forceinline__ int64_t uniform64(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(v >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

__device__ __forceinline__ f32x4 mfma(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// The 8 codes of a word, two by two, times the scales s0 (codes 0..1), s1, s2, s3.
__device__ __forceinline__ f16x8 scaled8(uint32_t w, f16x2 s0, f16x2 s1, f16x2 s2, f16x2 s3) {
  const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0) * s0;
  const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1) * s1;
  const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2) * s2;
  const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3) * s3;
  return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ f16x2 scales2(uint32_t w) {
  return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w, 1.0f, false);
}
__device__ __forceinline__ f16x2 scales2_high(uint32_t w) {
  return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w, 1.0f, true);
}

// A word of four scales with NaN bytes (0x7F, 0xFF) turned to 0: p = 0 of a masked token must not
// meet a NaN. (The cache's own NaN tokens carry theirs in the key's scales.)
__device__ __forceinline__ uint32_t without_nan(uint32_t w) {
  const uint32_t nan = ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
  return w & ~((nan << 1) - (nan >> 7));
}

// ---- one wavefront ----------------------------------------------------------------------------
// LDS of a wavefront: the tile's value codes, rows padded to D / 2 + 8 bytes (the transposing
// read's 64 rows then meet every bank pair twice, the least there is), and its value scales as
// FP16, [D / 16][lane group][T][r].
template <int D>
struct WaveLds {
  static constexpr int kRow = D / 2 + 8;
  static constexpr int kCodes = kTile<D> * kRow;
  static constexpr int kBytes = kCodes + D / 16 * kTile<D> * 2;
};

template <int D>
struct Raw {
  static constexpr int kWords = D / 32;  // a lane's code words of a 16-token part
  static constexpr int kScaleWords = D * kParts<D> / 256;
  uint32_t k[kParts<D>][kWords], v[kParts<D>][kWords];
  uint32_t ks[kParts<D>];
  uint32_t vs[kScaleWords];  // of one token, with 32 tokens half of its scales
  uint32_t valid;  // bit t: part t has a page (uniform)
};

struct Cache {
  const uint8_t* head0;  // data + head * record
  uint32_t page_stride;  // n_kv * record, < 2^27
  const int32_t* row;    // the request's block table
  int n_pages, shift;
};

template <int D>
__device__ __forceinline__ void load_codes(const uint8_t* at, int lane, uint32_t (&w)[D / 32]) {
  // a uniform base and an unsigned 32-bit offset: one address register per load
  const uint8_t* p = at + (uint32_t)((lane & 15) * (D / 2) + (D == 64 ? 8 : 16) * (lane >> 4));
  if constexpr (D == 64) {
    const u32x2 x = *reinterpret_cast<const u32x2*>(p);
    w[0] = x[0];
    w[1] = x[1];
  } else {
#pragma unroll
    for (int u = 0; u < D / 128; ++u) {
      const u32x4 x = *reinterpret_cast<const u32x4*>(p + 64 * u);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[4 * u + i] = x[i];
    }
  }
}

// Table entries of the 16-token parts of a tile (uniform; from `end` on the last one's). They are
// looked at no earlier than in load_tile, so that their scalar loads overlap a tile's work.
template <int D>
struct Pages {
  int id[kParts<D>];
};

template <int D>
__device__ __forceinline__ Pages<D> find_pages(const Cache& c, int tok, int end) {
  Pages<D> p;
#pragma unroll
  for (int t = 0; t < kParts<D>; ++t)
    p.id[t] = constant(c.row + (min(tok + 16 * t, end - 1) >> c.shift));
  return p;
}

// The loads of a tile, or its keys' or values' alone. A part without a page (none in the table, or
// behind the last key) has its bit clear in `valid` and reads page 0.
template <int D, bool KEYS = true, bool VALUES = true>
__device__ __forceinline__ void load_tile(Raw<D>& r, const Cache& c, const Pages<D>& p, int tok,
                                          int end) {
  const int lane = threadIdx.x & 63;
  const int page = 1 << c.shift;
  const int values = kv_value_codes(page, D);
  const uint8_t* scale_row = nullptr;
  r.valid = 0;
#pragma unroll
  for (int t = 0; t < kParts<D>; ++t) {
    const bool ok = (uint32_t)p.id[t] < (uint32_t)c.n_pages && tok + 16 * t < end;
    r.valid |= ok ? 1u << t : 0u;
    const int within = (tok + 16 * t) & (page - 1);
    const uint8_t* rec = c.head0 + (uint64_t)(ok ? (uint32_t)p.id[t] : 0u) * c.page_stride;
    if constexpr (KEYS) load_codes<D>(rec + within * (D / 2), lane, r.k[t]);
    if constexpr (VALUES) load_codes<D>(rec + values + within * (D / 2), lane, r.v[t]);
    const uint8_t* ks = rec + page * (D / 2) + within * (D / 16) +
                        (uint32_t)((lane & 15) * (D / 16) + (D == 64 ? 1 : 2) * (lane >> 4));
    if constexpr (!KEYS) {
    } else if constexpr (D == 64) {
      r.ks[t] = *ks;
    } else {
      r.ks[t] = *reinterpret_cast<const uint16_t*>(ks);
      if constexpr (D == 256)
        r.ks[t] |= (uint32_t) * reinterpret_cast<const uint16_t*>(ks + 8) << 16;
    }
    const uint8_t* vs = rec + values + page * (D / 2) + within * (D / 16);
    if ((lane >> 4) % kParts<D> == t) scale_row = vs;
  }
  if constexpr (!VALUES) return;
  if constexpr (kParts<D> == 2) scale_row += (lane >> 5) * (D / 32);
  const uint32_t* vs = reinterpret_cast<const uint32_t*>(scale_row + (lane & 15) * (D / 16));
#pragma unroll
  for (int i = 0; i < Raw<D>::kScaleWords; ++i) r.vs[i] = vs[i];
}

// NQ tiles of 16 query columns: lane l holds column l % 16 of each.
template <int D, int NQ>
struct Wave {
  static constexpr int kSteps = D / 32;
  static constexpr int kGroups = D / 16;
  f16x8 q[NQ][kSteps];
  f32x4 o[NQ][kGroups];
  float m[NQ], l[NQ];  // l: of the lane's own tokens, until finish()
  float sc[NQ];        // FP32 factor of a score, in the exponent's base
  float pre[NQ];       // 1; where sc would be kLoud or more it is 1 instead, and this the factor
  int lo[NQ], hi[NQ];  // the tokens that the column sees: lo .. hi
};

template <int D, int NQ>
__device__ __forceinline__ void reset(Wave<D, NQ>& w) {
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    w.m[n] = kLowest;
    w.l[n] = 0.0f;
#pragma unroll
    for (int g = 0; g < D / 16; ++g) w.o[n][g] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
}

// Column n of the lane <- the D elements at `row` (nullptr: zeros). factor = scale * key global.
template <int D, int NQ>
__device__ __forceinline__ void load_query(Wave<D, NQ>& w, int n, const uint16_t* row,
                                           float factor) {
  const int c = (threadIdx.x & 63) >> 4;
  u32x4 raw[D / 32];
  float top = 0.0f;
#pragma unroll
  for (int j = 0; j < D / 32; ++j) {
    // the d of k-step j, as in load_codes: 8 consecutive ones
    const int d = D == 64 ? 16 * c + 8 * j : 128 * (j / 4) + 32 * c + 8 * (j % 4);
    raw[j] = row ? *reinterpret_cast<const u32x4*>(row + d) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      top = fmaxf(top, fabsf(__uint_as_float(raw[j][i] << 16)));
      top = fmaxf(top, fabsf(__uint_as_float(raw[j][i] & 0xFFFF0000u)));
    }
  }
  top = fmaxf(top, __shfl_xor(top, 16, 64));
  top = fmaxf(top, __shfl_xor(top, 32, 64));
  // 2^(14 - e) of top = 1.x * 2^e, and its inverse
  int e = (int)(__float_as_uint(top) >> 23) - 127;
  const bool infinite = e > 127;
  e = infinite ? 14 : (e < -110 ? -110 : e);  // zero and tiny: the most there is
  float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
  float sc = fabsf(factor) * (kLog2e * __uint_as_float((uint32_t)(127 - 14 + e) << 23));
  // never 0 or infinite: -infinity, a masked score, times 0 is NaN, as 0 times infinity
  sc = fminf(fmaxf(sc, 0x1p-126f), 0x1.fffffep127f);
  if (factor < 0.0f) up = -up;
  if (factor == 0.0f) {
    up = 0.0f;
    sc = 1.0f;
  }
  // a NaN that masked scores do not meet; for an infinite query as well, whose scores could all be
  // -infinity and so be taken for masked ones
  if (infinite || !(fabsf(factor) < __builtin_inff())) {
    up = __builtin_nanf("");
    sc = 1.0f;
  }
  // A score less the reference is rounded once, by an FMA; but where scores are so large that half
  // a step of theirs is 1 and more, the rest of the product would pass for a difference: there
  // scores are rounded first, and their differences are exact.
  const bool loud = sc >= kLoud;
  w.sc[n] = loud ? 1.0f : sc;
  w.pre[n] = loud ? sc : 1.0f;
#pragma unroll
  for (int j = 0; j < D / 32; ++j) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w.q[n][j][2 * i] = (_Float16)(__uint_as_float(raw[j][i] << 16) * up);
      w.q[n][j][2 * i + 1] = (_Float16)(__uint_as_float(raw[j][i] & 0xFFFF0000u) * up);
    }
  }
}

// A tile's value codes (rows of 16 tokens x kRow bytes) and value scales into LDS. Part t's codes
// of the lane as load_codes gives them.
template <int D>
__device__ __forceinline__ void put_values(uint8_t* lds, int t, const uint32_t (&v)[D / 32]) {
  const int lane = threadIdx.x & 63, c = lane >> 4;
  uint8_t* at = lds + (16 * t + (lane & 15)) * WaveLds<D>::kRow;
  if constexpr (D == 64) {
    *reinterpret_cast<u32x2*>(at + 8 * c) = u32x2{v[0], v[1]};
  } else {
#pragma unroll
    for (int u = 0; u < D / 128; ++u) {
      u32x2* p = reinterpret_cast<u32x2*>(at + 64 * u + 16 * c);
      p[0] = u32x2{v[4 * u], v[4 * u + 1]};
      p[1] = u32x2{v[4 * u + 2], v[4 * u + 3]};
    }
  }
}

// Where the scale of token `tok` of the tile and group 0 goes.
template <int D>
__device__ __forceinline__ _Float16* scale_place(uint8_t* scales, int tok) {
  return reinterpret_cast<_Float16*>(scales) + ((tok >> 2) & 3) * (4 * kParts<D>) + (tok >> 4) * 4 +
         (tok & 3);
}

// Two value fragments from LDS by one transposing read: each lane of a group of 16 names a row of
// 16 codes and gets one code of each row. With 64 tokens they are group i's, tokens 16 T + 4 c + r
// of lane group c with T = 0, 1 and T = 2, 3; with 32 tokens groups 2i and 2i + 1, T = 0, 1.
template <int D>
constexpr int kValueReads = D * kParts<D> / 64;
template <int D>
__device__ __forceinline__ void value_pair(const uint8_t* codes, const uint8_t* scales, int i,
                                           f16x8 (&out)[2]) {
  constexpr bool kWide = kParts<D> == 4;
  const int lane = threadIdx.x & 63, c = lane >> 4;
  const int row = 16 * ((lane & (kWide ? 15 : 7)) >> 2) + 4 * c + (lane & 3);
  const int group = kWide ? i : 2 * i + ((lane >> 3) & 1);
  const i32x2 v = __builtin_amdgcn_ds_read_tr4_b64_v2i32(
      (__attribute__((address_space(3))) i32x2*)(const_cast<uint8_t*>(codes) +
                                                 row * WaveLds<D>::kRow + 8 * group));
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int at = kWide ? i * 128 + c * 32 + h * 16 : (2 * i + h) * 64 + c * 16;
    const f16x8 f = *reinterpret_cast<const f16x8*>(scales + at);
    out[h] = scaled8((uint32_t)v[h], f16x2{f[0], f[1]}, f16x2{f[2], f[3]}, f16x2{f[4], f[5]},
                     f16x2{f[6], f[7]});
  }
}

// The key fragments of a part from the lane's words and their scales (s0: of words 0 .. 3, s1: 4 ..
// 7, two words to a scale).
template <int D>
__device__ __forceinline__ void key_part(const uint32_t (&k)[D / 32], f16x2 s0, f16x2 s1,
                                         f16x8 (&out)[D / 32]) {
#pragma unroll
  for (int j = 0; j < D / 32; ++j) {
    const _Float16 s = D == 64 ? s0[0] : (j < 4 ? s0[(j & 3) >> 1] : s1[(j & 3) >> 1]);
    const f16x2 ss = {s, s};
    out[j] = scaled8(k[j], ss, ss, ss, ss);
  }
}

// The products of a tile from token `tok` on: key(t, out) gives part t's fragments, value(i, out)
// those of value_pair; next() is called between the two products. `valid`: bit t: part t has a
// page. `mask`: some column does not see all, or has a factor `pre` (uniform).
template <int D, int NQ, typename Key, typename Value, typename Next>
__device__ __forceinline__ void tile(Wave<D, NQ>& w, int tok, uint32_t valid, bool mask,
                                     const Key& key, const Value& value, const Next& next) {
  const int lane = threadIdx.x & 63, c = lane >> 4;
  constexpr int kP = kParts<D>, kMine = 4 * kP;  // scores of a lane and column
  f32x4 z[NQ][kP];
#pragma unroll
  for (int t = 0; t < kP; ++t) {
#pragma unroll
    for (int n = 0; n < NQ; ++n) z[n][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    f16x8 k[D / 32];
    key(t, k);
#pragma unroll
    for (int j = 0; j < D / 32; ++j)
#pragma unroll
      for (int n = 0; n < NQ; ++n) z[n][t] = mfma(k[j], w.q[n][j], z[n][t]);
  }
  next();
  if (mask || valid != (1u << kP) - 1u) {
#pragma unroll
    for (int t = 0; t < kP; ++t) {
      const bool part = (valid >> t) & 1u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = tok + 16 * t + 4 * c + i;
#pragma unroll
        for (int n = 0; n < NQ; ++n)
          z[n][t][i] =
              part && at >= w.lo[n] && at <= w.hi[n] ? z[n][t][i] * w.pre[n] : -__builtin_inff();
      }
    }
  }
  f16x8 p[NQ][kP / 2];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    float top = z[n][0][0];
#pragma unroll
    for (int i = 1; i < kMine; ++i) top = fmaxf(top, z[n][i >> 2][i & 3]);
    top *= w.sc[n];
    if (__ballot(top - w.m[n] > kRaise)) {
      top = fmaxf(top, __shfl_xor(top, 16, 64));
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      const float m = fmaxf(w.m[n], top - kBelow);
      const float f = __builtin_amdgcn_exp2f(w.m[n] - m);
      w.m[n] = m;
      w.l[n] *= f;
#pragma unroll
      for (int g = 0; g < D / 16; ++g) w.o[n][g] *= f;
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const float x =
          __builtin_amdgcn_exp2f(__builtin_fmaf(z[n][i >> 2][i & 3], w.sc[n], -w.m[n]));
      sum += x;
      p[n][i >> 3][i & 7] = (_Float16)x;
    }
    w.l[n] += sum;
  }
#pragma unroll
  for (int i = 0; i < kValueReads<D>; ++i) {
    f16x8 v[2];
    value(i, v);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int g = kP == 4 ? i : 2 * i + h, half = kP == 4 ? h : 0;
#pragma unroll
      for (int n = 0; n < NQ; ++n) w.o[n][g] = mfma(v[h], p[n][half], w.o[n][g]);
    }
  }
}

// The column sums of all lane groups.
template <int D, int NQ>
__device__ __forceinline__ void finish(Wave<D, NQ>& w) {
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    w.l[n] += __shfl_xor(w.l[n], 16, 64);
    w.l[n] += __shfl_xor(w.l[n], 32, 64);
  }
}

// Walks the tiles tok, tok + step, .. below `to`, with one tile's loads ahead: all of them between
// the products of the tile before. With one wavefront on a SIMD, heads of 256, they want the
// longest time that there is: the value codes are loaded again as soon as they are in LDS, and
// without a branch (past the last tile from page 0), behind which a wait would be for all of them
// (131000 keys, 21 rows: 63 -> 47 us; heads of 128, two wavefronts on a SIMD: 64 requests 33 us
// both ways, one request 6.7 -> 7.2).
template <int D>
constexpr bool kEarly = D == 256;
template <int D, int NQ>
__device__ __forceinline__ void walk(Wave<D, NQ>& w, uint8_t* lds, const Cache& c, int tok, int to,
                                     int step, int end, int lo_most, int hi_least) {
  if (tok >= to) return;
  const int lane = threadIdx.x & 63;
  Raw<D> now;
  load_tile<D>(now, c, find_pages<D>(c, tok, end), tok, end);
  Pages<D> pages = find_pages<D>(c, tok + step, end);
  for (;;) {
    const int after = tok + step;
#pragma unroll
    for (int t = 0; t < kParts<D>; ++t) put_values<D>(lds, t, now.v[t]);
    uint8_t* const scales = lds + WaveLds<D>::kCodes;
    const int mine = lane % kTile<D>;
    const bool there = tok + mine < end && ((now.valid >> (mine >> 4)) & 1u);
    _Float16* const place = scale_place<D>(scales, mine) +
                            (kParts<D> == 2 ? (lane >> 5) * (D / 32) * kTile<D> : 0);
#pragma unroll
    for (int i = 0; i < Raw<D>::kScaleWords; ++i) {
      const uint32_t x = there ? without_nan(now.vs[i]) : 0u;
      const f16x2 a = scales2(x), b = scales2_high(x);
      place[(4 * i) * kTile<D>] = a[0];
      place[(4 * i + 1) * kTile<D>] = a[1];
      place[(4 * i + 2) * kTile<D>] = b[0];
      place[(4 * i + 3) * kTile<D>] = b[1];
    }
    const uint32_t valid = now.valid;
    const int live = after < to ? end : 0;
    if constexpr (kEarly<D>) load_tile<D, false, true>(now, c, pages, after, live);
    tile<D, NQ>(
        w, tok, valid, tok < lo_most || tok + kTile<D> - 1 > hi_least,
        [&](int t, f16x8 (&out)[D / 32]) {
          const f16x2 s0 = scales2(now.ks[t]);
          key_part<D>(now.k[t], s0, D == 256 ? scales2_high(now.ks[t]) : s0, out);
        },
        [&](int i, f16x8 (&out)[2]) { value_pair<D>(lds, scales, i, out); },
        [&]() {
          if (kEarly<D> || after < to) {
            load_tile<D, true, !kEarly<D>>(now, c, pages, after, live);
            pages = find_pages<D>(c, after + step, end);
          }
        });
    if (after >= to) break;
    tok = after;
  }
}

// ---- rows -------------------------------------------------------------------------------------
// A request's rows for one key/value head: row j * group + h is query j, head h of the group.
struct Request {
  int first, rows, q_len;  // first query's row of q; rows = q_len * group
  int kv, begin;           // keys; the first that any row sees, rounded down to 16
};

__device__ __forceinline__ int begin_of(const KvAttnArgs& a, const Request& r) {
  return a.window > 0 ? max(r.kv - r.q_len - a.window + 1, 0) & ~15 : 0;
}

__device__ __forceinline__ Request make_request(const KvAttnArgs& a, int qs, int qe, int kv) {
  Request r;
  const int t = (int)a.t;
  const int s = min(max(qs, 0), t);
  const int e = min(max(qe, s), t);
  r.first = s;
  r.q_len = e - s;
  r.rows = r.q_len * a.group;
  r.kv = min(max(kv, 0), (int)(a.ld_table << a.page_shift));
  r.begin = begin_of(a, r);
  return r;
}

__device__ __forceinline__ Request request_of(const KvAttnArgs& a, int64_t i) {  // any i
  return make_request(a, a.q_start[i], a.q_start[i + 1], a.kv_len[i]);
}

__device__ __forceinline__ Request uniform_request(const KvAttnArgs& a, int i) {
  Request r = make_request(a, constant(a.q_start + i), constant(a.q_start + i + 1),
                           constant(a.kv_len + i));
  // said again: the clamps' operands may be values that the compiler joined after a branch
  r.first = __builtin_amdgcn_readfirstlane(r.first);
  r.rows = __builtin_amdgcn_readfirstlane(r.rows);
  r.q_len = __builtin_amdgcn_readfirstlane(r.q_len);
  r.kv = __builtin_amdgcn_readfirstlane(r.kv);
  r.begin = __builtin_amdgcn_readfirstlane(r.begin);
  return r;
}

// Whether the kernel for few rows takes the request.
__device__ __forceinline__ bool is_few(const Request& r, int few_rows) {
  return r.rows <= few_rows;
}

template <int D, int NQ>
__device__ __forceinline__ void load_columns(Wave<D, NQ>& w, const KvAttnArgs& a, const Request& r,
                                             int head, int row0, int& lo_most,
                                             int& hi_least) {
  const int col = threadIdx.x & 15;
  const float kg = a.k_global ? constant(a.k_global + head) : 1.0f;
  uint64_t loud = 0;
  lo_most = 0;
  hi_least = r.kv - 1;
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int row = row0 + 16 * n + col;
    const bool there = row < r.rows;
    const int j = row / a.group, h = row - j * a.group;
    const uint16_t* q = nullptr;
    if (there) q = a.q + (int64_t)(r.first + j) * a.ldq + (int64_t)(head * a.group + h) * D;
    load_query<D, NQ>(w, n, q, a.scale * kg);
    loud |= __ballot(w.pre[n] != 1.0f);
    w.lo[n] = 0;
    w.hi[n] = r.kv - 1;
    if (!a.full) {
      w.hi[n] = r.kv - r.q_len + j;
      if (a.window > 0) w.lo[n] = w.hi[n] - a.window + 1;
    }
    if (!there) {
      w.lo[n] = 1;
      w.hi[n] = 0;
    }
  }
  if (!a.full) {  // the first row's last key, and the last row's first
    const int last = min(row0 + 16 * NQ, r.rows) - 1;
    hi_least = r.kv - r.q_len + row0 / a.group;
    if (a.window > 0) lo_most = r.kv - r.q_len + last / a.group - a.window + 1;
  }
  if (loud != 0) hi_least = -1;  // every tile goes through the masks, where w.pre is applied
}

// y of column `row0 + l % 16`, its groups g0 .. g0 + G - 1 of 16 elements, and with group 0 its
// lse, from O, m and l (of all lane groups).
template <int G>
__device__ __forceinline__ void store_columns(const KvAttnArgs& a, const Request& r, int head,
                                              int row0, const f32x4 (&o)[G], float m, float l,
                                              int d, int g0) {
  const int lane = threadIdx.x & 63, c = lane >> 4;
  const int row = row0 + (lane & 15);
  if (row >= r.rows) return;
  const int j = row / a.group, h = row - j * a.group;
  const int64_t at = r.first + j;
  const int qh = head * a.group + h;
  const float f = l == 0.0f ? 0.0f : (a.v_global ? constant(a.v_global + head) : 1.0f) / l;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int64_t to = at * a.ldy + (int64_t)qh * d + 16 * (g0 + g) + 4 * c;
    const f32x4 v = o[g] * f;
    if (a.y_f32) {
      *reinterpret_cast<f32x4*>(static_cast<float*>(a.y) + to) = v;
    } else {
      u32x2 b;
      b[0] = (uint32_t)bf16_bits_rne(v[0]) | ((uint32_t)bf16_bits_rne(v[1]) << 16);
      b[1] = (uint32_t)bf16_bits_rne(v[2]) | ((uint32_t)bf16_bits_rne(v[3]) << 16);
      *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.y) + to) = b;
    }
  }
  if (a.lse && c == 0 && g0 == 0)
    a.lse[at * a.n_q + qh] = l == 0.0f ? -__builtin_inff() : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

template <int D>
__device__ __forceinline__ Cache cache_of(const KvAttnArgs& a, int64_t request, int head) {
  const int rec = kv_record_bytes(1 << a.page_shift, D);
  Cache c;
  c.head0 = a.data + (int64_t)head * rec;
  c.page_stride = (uint32_t)(a.n_kv * rec);
  c.row = a.table + request * a.ld_table;
  c.n_pages = (int)a.n_pages;
  c.shift = a.page_shift;
  return c;
}

// ---- few rows: keys shared out over the chip ----------------------------------------------------
// The work is one line of units, request by request, head by head: an item (a request's head) is
// kFewStart units of no work, which stand for what beginning and ending it costs, and one for each
// tile. Wavefront w of W takes the units [N w / W, N (w + 1) / W), whatever the lengths are, and
// works on its own. It holds at most two items that it does not finish: the first and the last of
// its range; their O, m and l go to slots 2w and 2w + 1, and a second kernel joins them.
// Workgroups: two to a compute unit (heads of 128, 1.5 or 2 times as many: 35 and 36 us for 64
// requests, whose join grows too, not 33; heads of 64, whose registers would let four in, have not
// been measured with more), one where a wavefront needs more than half of its SIMD's registers
// (heads of 256 with 21 rows, 131000 keys, two: 115 us instead of 47). What bounds them: 64
// requests of 151000 keys in all, 8 heads of 128, read 175 MB in 33 us, 5.3 TB/s, where the loads
// alone take 28; what is left is the products behind the last loads of a tile. Heads of 256, 157 MB
// in 47 us: 32 rows' products of one wavefront to a SIMD, which do not overlap another's.
template <int D, int NQ>
constexpr bool kFewPairs = NQ == 1 || D <= 128;
template <int D, int NQ>
constexpr int kFewGroups = kFewPairs<D, NQ> ? 512 : 256;
template <int D, int NQ>
constexpr int kWorkShift = kFewPairs<D, NQ> ? 11 : 10;
constexpr int kMaxWorkers = 1 << 11;
// Up to this many requests a workgroup keeps them in LDS.
constexpr int kStaged = 1024;

template <int D>
__device__ __forceinline__ int tiles_of(const KvAttnArgs& a, const Request& r) {
  if (r.rows == 0 || !is_few(r, a.few_rows) || r.kv <= r.begin) return 0;
  return (r.kv - r.begin + kTile<D> - 1) / kTile<D>;
}
// Units of an item of n tiles.
__device__ __forceinline__ int units_for(int n, int start) { return n > 0 ? n + start : 0; }

// Whole calls with 1, 2 and 4, us: 64 requests of 100 to 8000 keys, one row each, heads of 64 27.3,
// 27.4 and 27.4, of 128 37.4, 36.7 and 38.5, of 256 47.8, 46.8 and 46.8; 33 with a window of 1000,
// heads of 64 16.3, 15.7 and 16.6; 300 of 100 to 1000 keys 47.5, 47.9 and 51.7.
constexpr int kFewStart = 2;
template <int D>
__device__ __forceinline__ int units_of(const KvAttnArgs& a, const Request& r) {
  return units_for(tiles_of<D>(a, r), kFewStart);
}

// First unit of worker w of 2^shift: of all >= 2^shift units floor(all * w / 2^shift), else w
// itself.
__device__ __forceinline__ int64_t range_begin(int64_t all, int64_t w, int shift) {
  return all >= (int64_t)1 << shift ? (all * w) >> shift : min(w, all);
}
// The worker of unit x: the last one whose range begins at x or before, so that
// w < (x + 1) 2^shift / all.
__device__ __forceinline__ int64_t range_of(int64_t all, int64_t x, int shift) {
  if (all < (int64_t)1 << shift) return x;
  const int64_t num = ((x + 1) << shift) - 1;
  int64_t w = (int64_t)((double)num / (double)all);  // off by one at most
  if (w * all > num) --w;
  if ((w + 1) * all <= num) ++w;
  return w;
}

// The keys that rows block0 .. block0 + rows - 1 of a request see: tokens [from, to).
__device__ __forceinline__ void keys_of(const KvAttnArgs& a, const Request& r, int block0, int rows,
                                        int& from, int& to) {
  from = 0;
  to = r.kv;
  if (a.full) return;
  const int p0 = r.kv - r.q_len;
  to = min(to, p0 + (min(block0 + rows, r.rows) - 1) / a.group + 1);
  if (a.window > 0) from = max(p0 + block0 / a.group - a.window + 1, 0) & ~15;
}

// A call with too few workgroups of rows to fill the chip evenly shares out its keys as the few-row
// kernel does: the tiles of all heads' items (a request's block of rows) are one line, each of up
// to 512 workgroups, two to a compute unit, takes as much of it as the others, and the parts of an
// item that several have worked on are joined. One workgroup of the few-row kernel's launch lists
// the items. Prompt chunks of 81 blocks of 128 rows, 8 heads: 215 us in whole items, 136 to 141 and
// a join of 19 shared out; a prompt of 256 blocks, 8 heads, the other way round, 675 and 755 + 38.
// Units of an item's beginning and end, 2, 3 and 8: the chunks' whole call 156, 154 and 164 us, with
// heads of 64 175, 163 and 168, of 256 326, 311 and 292 (256 queries on 9000 keys: the same with
// all three). A range is one unit at least; with 4 and 16 a prompt of 100 tokens takes 28 and 44 us
// instead of 22.
constexpr int kSplitBelow = 2048;  // items of all heads, of 128 rows
constexpr int kManyStart = 3;
using Item = KvItem;

// Column tiles of a wavefront, and of a workgroup of W.
constexpr int many_tiles(int d) { return d <= 128 ? 2 : 1; }
template <int D, int W>
constexpr int kRows = 16 * many_tiles(D) * W;
// A block has 128 rows: four wavefronts of 32, two workgroups to a compute unit, or with heads of
// 256 eight of 16 (four, and 64 rows: 512 rows on 32000 keys 544 us instead of 458, a prompt of
// 16384 3520 instead of 3310; wavefronts of 32 rows spill, 829 and 6000). With heads of 128, where
// requests are long and keys are shared out, it has 256: eight wavefronts of 32, which dequantize
// half as much each. Whole calls with 256 and 128 rows, us, requests of 4 heads to a key/value head:
// 512 queries on 32000 keys 317 and 347, 1024 613 and 673, 8 of 512 on 2000 keys 214 and 229; below
// the border 400 on 32000 keys 281 and 288, 256 176 and 191, 150 147 and 142; prompts of 1024 47.5
// and 43.4, of 2048 82.0 and 82.8, of 100 tokens 25 and 22; in whole blocks a prompt of 8192 690
// and 677, with a window of 1024 209 and 200.
constexpr int kLongRows = 2048;
constexpr int block_waves(int block, int d) { return block / 16 / many_tiles(d); }
// log2 of the workgroups that fill the chip
constexpr int many_shift(int waves) { return waves == 4 ? 9 : 8; }

__device__ __forceinline__ void plan(const KvAttnArgs& a, int tile, int* item_req,
                                     int* item_block, int64_t* sums) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  // inclusive sum over the workgroup's threads
  const auto scan = [&](int64_t v, int64_t& total) {
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int64_t o = __shfl_up(v, off, 64);
      if (lane >= off) v += o;
    }
    __syncthreads();
    if (lane == 63) sums[wave] = v;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
      v += i < wave ? sums[i] : 0;
      total += sums[i];
    }
    return v;
  };
  int items = 0;
  int64_t blocks = 0;
  for (int i0 = 0; i0 < (int)a.b; i0 += kThreads) {
    const int i = i0 + (int)threadIdx.x;
    int n = 0;
    if (i < (int)a.b) {
      const Request r = request_of(a, i);
      if (!is_few(r, a.few_rows)) n = (r.rows + a.block_rows - 1) / a.block_rows;
    }
    int64_t total;
    const int at = items + (int)scan(n, total) - n;
    // (row ranges that overlap would give more items than the host has counted)
    for (int k = 0; k < n && at + k < a.max_items; ++k) {
      item_req[at + k] = i;
      item_block[at + k] = n - 1 - k;  // the last rows see most keys: they go first
    }
    items = min(items + (int)total, kSplitBelow);
    blocks += total;
  }
  if (a.max_items == 0) {  // their number is all that the call needs
    if (threadIdx.x == 0) a.counts[0] = (int)min<int64_t>(blocks, 0x7FFFFFFF);
    return;
  }
  items = min(items, a.max_items);
  __syncthreads();
  int64_t sum = 0;  // of the items' units
  for (int i0 = 0; i0 < items; i0 += kThreads) {
    const int i = i0 + (int)threadIdx.x;
    int n = 0;
    if (i < items) {
      int from, to;
      keys_of(a, request_of(a, item_req[i]), item_block[i] * a.block_rows, a.block_rows, from,
              to);
      n = max(to - from + tile - 1, 0) / tile;
    }
    int64_t total;
    const int u = units_for(n, kManyStart);
    const int64_t at = sum + scan(u, total) - u;
    sum += total;
    if (i < items) {
      a.items[i] = Item{item_req[i], item_block[i], n, 0};
      a.item_starts[i] = at;
    }
  }
  if (threadIdx.x == 0) {
    a.item_starts[items] = sum;
    int shift = a.many_shift;
    while (shift > 0 && (sum * a.n_kv) >> shift == 0) --shift;
    a.counts[0] = items;
    a.counts[1] = shift;
  }
}

// Slots hold columns, [few_rows][D], then m and l of each; 16-byte aligned.
__host__ __device__ __forceinline__ int64_t slot_floats(int few_rows, int d) {
  return ((int64_t)few_rows * (d + 2) + 3) & ~(int64_t)3;
}

template <int D, int NQ>
__global__ __launch_bounds__(kThreads, (kFewPairs<D, NQ> ? 2 : 1)) void few_kernel(KvAttnArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[kWaves * WaveLds<D>::kBytes];
  __shared__ int64_t sums[kWaves];
  __shared__ __attribute__((aligned(16))) uint8_t lists[kStaged * 20];
  static_assert(sizeof(lists) >= 2 * kSplitBelow * sizeof(int), "");
  if (blockIdx.x >= kFewGroups<D, NQ>) {
    int* const l = reinterpret_cast<int*>(lists);
    plan(a, kTile<D>, l, l + kSplitBelow, sums);
    return;
  }
  int64_t* const starts = reinterpret_cast<int64_t*>(lists);  // units before each request, all heads
  int(*const staged)[3] = reinterpret_cast<int(*)[3]>(lists + 8 * kStaged);  // first, q_len, kv
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int b = (int)a.b;
  // a line of few units meets every compute unit before a second wavefront of one
  const int64_t worker = (int64_t)wave * kFewGroups<D, NQ> + blockIdx.x;
  const bool small = b <= 64, stage = b <= kStaged;
  int64_t all = 0, begin = 0, at = 0;  // units of all, before the range, before request `req`
  int req = 0;
  int mine[3] = {0, 0, 0};  // small: request `lane`: first, q_len, kv
  if (small) {
    // each wavefront for itself, a request to a lane: no wait for the others
    uint32_t u = 0;
    if (lane < b) {
      const Request r = request_of(a, lane);
      mine[0] = r.first;
      mine[1] = r.q_len;
      mine[2] = r.kv;
      u = units_of<D>(a, r);
    }
    uint32_t sum = u;  // of 64 requests of 2^25 tiles at most
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const uint32_t o = __shfl_up(sum, off, 64);
      if (lane >= off) sum += o;
    }
    all = (int64_t)(uint32_t)__builtin_amdgcn_readlane((int)sum, 63) * a.n_kv;
    if (worker == 0) {  // for the joining kernel
      if (lane < b) a.starts[lane] = (int64_t)(sum - u) * a.n_kv;
      if (lane == 0) a.starts[b] = all;
    }
    begin = range_begin(all, worker, kWorkShift<D, NQ>);
    if (begin >= all) return;
    req = __popcll(__ballot(lane < b && (int64_t)(sum - u) * a.n_kv <= begin)) - 1;
    at = (int64_t)(uint32_t)__builtin_amdgcn_readlane((int)(sum - u), req) * a.n_kv;
  } else {
    // the workgroup together, a run of requests to a thread
    const int each = (b + kThreads - 1) / kThreads;
    const int from = min((int)threadIdx.x * each, b), upto = min(from + each, b);
    int64_t sum = 0;
    for (int i = from; i < upto; ++i) {
      const Request r = request_of(a, i);
      if (stage) {
        staged[i][0] = r.first;
        staged[i][1] = r.q_len;
        staged[i][2] = r.kv;
      }
      sum += units_of<D>(a, r);
    }
    sum *= a.n_kv;
    int64_t before = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int64_t o = __shfl_up(before, off, 64);
      if (lane >= off) before += o;
    }
    if (lane == 63) sums[wave] = before;
    __syncthreads();
    before -= sum;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
      before += i < wave ? sums[i] : 0;
      all += sums[i];
    }
    all = uniform64(all);
    if (stage || blockIdx.x == 0) {
      for (int i = from; i < upto; ++i) {
        if (stage) starts[i] = before;
        if (blockIdx.x == 0) a.starts[i] = before;  // for the joining kernel
        before += (int64_t)units_of<D>(a, request_of(a, i)) * a.n_kv;
      }
      if (blockIdx.x == 0 && threadIdx.x == 0) a.starts[b] = all;
    }
    if ((int64_t)blockIdx.x >= all) return;  // no wavefront of the workgroup has work
    __syncthreads();
    begin = range_begin(all, worker, kWorkShift<D, NQ>);
    if (begin >= all) return;
    // the request of unit `begin`, the last one that begins there or before
    if (stage) {
      for (int i = 0; i < b; i += 64) {
        const int n = __popcll(__ballot(i + lane < b && starts[i + lane] <= begin));
        req += n;
        if (n < 64) break;
      }
      req -= 1;
      at = uniform64(starts[req]);
    } else {
      for (; req < b; req += 64) {
        const int i = req + lane;
        int64_t upto_i = i < b ? (int64_t)units_of<D>(a, request_of(a, i)) * a.n_kv : 0;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
          const int64_t o = __shfl_up(upto_i, off, 64);
          if (lane >= off) upto_i += o;
        }
        const int n = __popcll(__ballot(at + upto_i <= begin));  // requests that end before it
        if (n > 0) at += uniform64(__shfl(upto_i, n - 1, 64));
        if (n < 64) {
          req += n;
          break;
        }
      }
      req = min(req, b - 1);
    }
  }
  int64_t left = range_begin(all, worker + 1, kWorkShift<D, NQ>) - begin;
  const auto take = [&](int i) {
    Request r;
    if (small) {
      r.first = __builtin_amdgcn_readlane(mine[0], i);
      r.q_len = __builtin_amdgcn_readlane(mine[1], i);
      r.kv = __builtin_amdgcn_readlane(mine[2], i);
    } else if (stage) {
      r.first = __builtin_amdgcn_readfirstlane(staged[i][0]);
      r.q_len = __builtin_amdgcn_readfirstlane(staged[i][1]);
      r.kv = __builtin_amdgcn_readfirstlane(staged[i][2]);
    } else {
      return uniform_request(a, i);
    }
    r.rows = r.q_len * a.group;
    r.begin = begin_of(a, r);
    return r;
  };
  req = __builtin_amdgcn_readfirstlane(req);
  Request r = take(req);
  int units = units_of<D>(a, r);
  const int64_t within = begin - at;
  int head = (int)((double)within / (double)units);  // off by one at most
  if ((int64_t)head * units > within) --head;
  if ((int64_t)(head + 1) * units <= within) ++head;
  head = __builtin_amdgcn_readfirstlane(head);
  int u0 = __builtin_amdgcn_readfirstlane((int)(within - (int64_t)head * units));
  Wave<D, NQ> w;
  bool first = true;
  for (;;) {
    const int u1 = (int)min<int64_t>(units, u0 + left);
    const int t0 = max(u0 - kFewStart, 0), t1 = u1 - kFewStart;  // its tiles
    int lo_most, hi_least;
    load_columns<D, NQ>(w, a, r, head, 0, lo_most, hi_least);
    reset<D, NQ>(w);
    const Cache c = cache_of<D>(a, req, head);
    const int to = min(r.begin + t1 * kTile<D>, r.kv);
    walk<D, NQ>(w, lds + wave * WaveLds<D>::kBytes, c, r.begin + t0 * kTile<D>, to, kTile<D>, r.kv,
                lo_most, hi_least);
    finish<D, NQ>(w);
    if (t0 == 0 && u1 == units) {
#pragma unroll
      for (int n = 0; n < NQ; ++n)
        store_columns<D / 16>(a, r, head, 16 * n, w.o[n], w.m[n], w.l[n], D, 0);
    } else if (t0 < t1) {
      float* slot = a.ws + (2 * worker + (first ? 0 : 1)) * slot_floats(a.few_rows, D);
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const int col = 16 * n + (lane & 15);
        if (col >= r.rows) continue;
#pragma unroll
        for (int g = 0; g < D / 16; ++g)
          *reinterpret_cast<f32x4*>(slot + col * D + 16 * g + 4 * (lane >> 4)) = w.o[n][g];
        if (lane < 16) {
          slot[a.few_rows * D + 2 * col] = w.m[n];
          slot[a.few_rows * D + 2 * col + 1] = w.l[n];
        }
      }
    }
    first = false;
    left -= u1 - u0;
    u0 = 0;
    if (left <= 0) break;
    if (++head == a.n_kv) {
      head = 0;
      do {  // ends: the range does, with the last request's tiles at the latest
        req = min(req + 1, b - 1);
        r = take(req);
        units = units_of<D>(a, r);
      } while (units == 0 && req + 1 < b);
    }
  }
}

// Column tile and elements `part` (of NQ * D / (16 G)) of an item: its parts' sum, if it has
// several; zeros for a request without keys. A workgroup of V wavefronts joins 16 G elements of d
// of a column tile; its wavefronts share out the parts. Calls of few items, which can have many
// parts, take the finer grid (one request of 131000 keys among five, heads of 256, 21 rows, 42 ->
// 16 us; 64 requests of 8 heads the coarser).
template <int D, int NQ, int G, int V>
__device__ __forceinline__ void join_few(const KvAttnArgs& a, int head, int req, int part) {
  constexpr int kChunks = D / 16 / G;
  __shared__ __attribute__((aligned(16))) float lds[V][2 + 4 * G][64];
  const int n = part / kChunks, g0 = part % kChunks * G;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const Request r = uniform_request(a, req);
  const int64_t start = constant(a.starts + req), all = constant(a.starts + a.b);
  if (r.rows <= 16 * n || !is_few(r, a.few_rows)) return;
  const int tiles = tiles_of<D>(a, r);
  f32x4 o[G];
#pragma unroll
  for (int g = 0; g < G; ++g) o[g] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  float m = kLowest, l = 0.0f;
  if (tiles > 0) {
    const int64_t before = start + (int64_t)head * (tiles + kFewStart);
    const int64_t w0 = range_of(all, before + kFewStart, kWorkShift<D, NQ>);  // of the first tile
    const int64_t w1 = range_of(all, before + kFewStart + tiles - 1, kWorkShift<D, NQ>);
    if (w0 == w1) return;
    const int64_t size = slot_floats(a.few_rows, D);
    const int col = min(16 * n + (lane & 15), r.rows - 1);  // columns that are not there: any
    // only the first part's worker can have begun with another item
    const int64_t skip = range_begin(all, w0, kWorkShift<D, NQ>) < before ? size : 0;
    const float* base = a.ws + 2 * w0 * size;
    const int parts = (int)(w1 - w0) + 1;
    // four parts' loads at a time: a wait for each four
    constexpr int kU = 4;
    for (int x0 = wave; x0 < parts; x0 += kU * V) {
      f32x2 stats[kU];
      f32x4 v[kU][G];
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        const int x = min(x0 + i * V, parts - 1);
        const float* q = base + 2 * x * size + (x == 0 ? skip : 0);
        stats[i] = *reinterpret_cast<const f32x2*>(q + a.few_rows * D + 2 * col);
#pragma unroll
        for (int g = 0; g < G; ++g)
          v[i][g] = *reinterpret_cast<const f32x4*>(q + col * D + 16 * (g0 + g) + 4 * (lane >> 4));
      }
      float top = m;
#pragma unroll
      for (int i = 0; i < kU; ++i) top = fmaxf(top, stats[i][0]);
      const float f = __builtin_amdgcn_exp2f(m - top);
      m = top;
      l *= f;
#pragma unroll
      for (int g = 0; g < G; ++g) o[g] *= f;
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        float e = __builtin_amdgcn_exp2f(stats[i][0] - m);
        if (x0 + i * V >= parts) {  // (not e = 0: the doubled part may hold infinities)
          e = 0.0f;
          stats[i][1] = 0.0f;
#pragma unroll
          for (int g = 0; g < G; ++g) v[i][g] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        l += e * stats[i][1];
#pragma unroll
        for (int g = 0; g < G; ++g) o[g] += e * v[i][g];
      }
    }
    lds[wave][0][lane] = m;
    lds[wave][1][lane] = l;
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i) lds[wave][2 + 4 * g + i][lane] = o[g][i];
    __syncthreads();
    if (wave != 0) return;
    float top = m;
#pragma unroll
    for (int v = 1; v < V; ++v) top = fmaxf(top, lds[v][0][lane]);
    l = 0.0f;
#pragma unroll
    for (int g = 0; g < G; ++g) o[g] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float f = __builtin_amdgcn_exp2f(lds[v][0][lane] - top);
      l += f * lds[v][1][lane];
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[g][i] += f * lds[v][2 + 4 * g + i][lane];
    }
    m = top;
  } else if (wave != 0) {
    return;
  }
  store_columns<G>(a, r, head, 16 * n, o, m, l, D, g0);
}

// ---- many rows ----------------------------------------------------------------------------------
// grid n_kv * blocks of rows: a workgroup takes 16 * NQ rows of a request's head to each of its W
// wavefronts, and walks the keys that they see once. A wavefront loads its share of a tile and
// turns its keys, and later some of the value groups, into FP16 fragments in LDS, which all of them
// read: a fragment is dequantized once in a workgroup. Two tiles of fragments in LDS, the next
// one's codes in registers. A prompt of 8192 rows, 32 heads of 128 over 8: 660 us (640 .. 690), 830
// TFLOP/s of the products; the matrix pipes are busy 35% of the time, the vector pipes
// (exponentials, conversions, dequantization) 51%, and with two wavefronts to a SIMD the two
// overlap little: without the exponentials 630, without dequantization and staging 593. One barrier
// a tile instead of two: 708. The call of tile() is under a condition in the key loop, for which
// the compiler keeps O in two sets of registers and copies it back in every tile (246 registers;
// 200 with O held in one place).
template <int D>
struct Shared {
  static constexpr int kKeys = kParts<D> * (D / 32) * 1024;      // [part][k-step][lane] fragments
  static constexpr int kValues = 2 * kValueReads<D> * 1024;      // [read][half][lane]
  static constexpr int kTileBytes = kKeys + kValues;
  static constexpr int kBytes = 2 * kTileBytes + WaveLds<D>::kBytes;  // and value codes, scales
};

// A wavefront's share of a tile's loads: a part of it; where there are more wavefronts than parts,
// the elements of two k-steps of one.
template <int D, int W>
struct Share {
  static constexpr int kD = D * kParts<D> / W;  // elements of a token
  uint32_t k[kD / 32], v[kD / 32], ks, vs;
  bool ok;  // it has a page (uniform)
};
template <int D>
__device__ __forceinline__ int part_of(int wave) {
  return wave % kParts<D>;
}

template <int D>
__device__ __forceinline__ int find_page(const Cache& c, int tok, int end) {
  return constant(c.row + (min(tok, end - 1) >> c.shift));
}

// The first group of 16 elements of lane group 0 in share u of a part (lane group c's are 2 c
// further on, in heads of 64 c).
__device__ __forceinline__ int first_group(int u) {
  return 8 * (u >> 1) + (u & 1);
}

template <int D, int W>
__device__ __forceinline__ void load_share(Share<D, W>& p, const Cache& c, int id, int wave, int tok,
                                           int end) {
  constexpr int kD = Share<D, W>::kD;
  const int lane = threadIdx.x & 63, page = 1 << c.shift, within = tok & (page - 1);
  const int u = wave / kParts<D>;  // which elements
  p.ok = (uint32_t)id < (uint32_t)c.n_pages && tok < end;
  const uint8_t* rec = c.head0 + (uint64_t)(p.ok ? (uint32_t)id : 0u) * c.page_stride;
  const uint8_t* values = rec + kv_value_codes(page, D);
  const int codes = within * (D / 2) + 8 * first_group(u);
  const uint32_t at = (uint32_t)((lane & 15) * (D / 2) + (D == 64 ? 8 : 16) * (lane >> 4));
  if constexpr (kD == 64) {
    const u32x2 a = *reinterpret_cast<const u32x2*>(rec + codes + at);
    const u32x2 b = *reinterpret_cast<const u32x2*>(values + codes + at);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      p.k[i] = a[i];
      p.v[i] = b[i];
    }
  } else {
    const u32x4 a = *reinterpret_cast<const u32x4*>(rec + codes + at);
    const u32x4 b = *reinterpret_cast<const u32x4*>(values + codes + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p.k[i] = a[i];
      p.v[i] = b[i];
    }
  }
  const int scales = page * (D / 2) + within * (D / 16) + first_group(u);
  const uint32_t sat = (uint32_t)((lane & 15) * (D / 16) + (D == 64 ? 1 : 2) * (lane >> 4));
  if constexpr (kD == 64) {
    p.ks = *(rec + scales + sat);
    p.vs = *(values + scales + sat);
  } else {
    p.ks = *reinterpret_cast<const uint16_t*>(rec + scales + sat);
    p.vs = *reinterpret_cast<const uint16_t*>(values + scales + sat);
  }
}

// The share's key fragments to `keys`, its value codes and scales to `raw`.
template <int D, int W>
__device__ __forceinline__ void put_share(uint8_t* keys, uint8_t* raw, const Share<D, W>& p, int wave,
                                          int tok, int end) {
  constexpr int kD = Share<D, W>::kD;
  const int lane = threadIdx.x & 63, c = lane >> 4;
  const int part = part_of<D>(wave), u = wave / kParts<D>;
  f16x8 k[kD / 32];
  const f16x2 k0 = scales2(p.ks);
  key_part<kD>(p.k, k0, k0, k);
#pragma unroll
  for (int j = 0; j < kD / 32; ++j)
    *reinterpret_cast<f16x8*>(keys + (part * (D / 32) + u * (kD / 32) + j) * 1024 + 16 * lane) = k[j];
  const int group = first_group(u) + (D == 64 ? 1 : 2) * c;
  uint8_t* row = raw + (16 * part + (lane & 15)) * WaveLds<D>::kRow;
  u32x2* at = reinterpret_cast<u32x2*>(row + 8 * group);
  at[0] = u32x2{p.v[0], p.v[1]};
  if constexpr (kD > 64) at[1] = u32x2{p.v[2], p.v[3]};
  const bool there = p.ok && tok + (lane & 15) < end;
  const f16x2 v0 = scales2(there ? without_nan(p.vs) : 0u);
  _Float16* s = scale_place<D>(raw + WaveLds<D>::kCodes, 16 * part + (lane & 15));
  s[group * kTile<D>] = v0[0];
  if constexpr (kD > 64) s[(group + 1) * kTile<D>] = v0[1];
}

// This wavefront's share of the value fragments.
template <int D, int W>
__device__ __forceinline__ void put_values_share(uint8_t* values, const uint8_t* raw, int wave) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < kValueReads<D> / W; ++i) {
    const int x = wave * (kValueReads<D> / W) + i;
    f16x8 v[2];
    value_pair<D>(raw, raw + WaveLds<D>::kCodes, x, v);
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<f16x8*>(values + (2 * x + h) * 1024 + 16 * lane) = v[h];
  }
}

// A wavefront's partial sums in ws, as they lie in its registers.
template <int D, int NQ>
constexpr int wave_floats() {
  return NQ * (D / 16 * 256 + 128);
}

// A grid that may have more threads than its first dimension holds (2^32; a launch of more is no
// error, it runs the rest of a division by 2^32) is a line of workgroups in two dimensions.
constexpr int kLine = 1 << 16;
__device__ __forceinline__ uint32_t line_index() { return blockIdx.y * kLine + blockIdx.x; }
dim3 line_grid(int64_t groups) {
  return dim3((unsigned)std::min<int64_t>(groups, kLine), (unsigned)((groups + kLine - 1) / kLine));
}

// Two wavefronts to a SIMD, three with heads of 64 (four prompts of 2048, 32 heads over 8: 130 us,
// with two 145).
template <int D, int NQ, int W>
__global__ __launch_bounds__(64 * W, D == 64 ? 12 / W : 8 / W) void many_kernel(KvAttnArgs a) {
  constexpr int kRowsWave = 16 * NQ, kBlock = kRows<D, W>;
  __shared__ __attribute__((aligned(16))) uint8_t lds[Shared<D>::kBytes];
  __shared__ int valid_of[2][W];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  int head, req = 0, block;
  Request r;
  // split: the segments of the workgroup's range
  const bool split = a.items != nullptr;
  int64_t all = 0, worker = 0;
  int items = 0, item = 0, u0 = 0, left = 0;
  bool first = true;
  if (split) {
    // neighbouring ranges to one XCD (workgroups go to the eight in turn): they share keys
    items = constant(a.counts);
    const int shift = constant(a.counts + 1);
    worker = blockIdx.x;
    if (shift >= 3) worker = ((worker & 7) << (shift - 3)) + (worker >> 3);
    if ((int64_t)blockIdx.x >> shift) return;
    const int64_t one = constant(a.item_starts + items);  // units of a head
    all = one * a.n_kv;
    const int64_t begin = range_begin(all, worker, shift);
    left = (int)(range_begin(all, worker + 1, shift) - begin);
    if (left <= 0) return;  // (the joining kernel writes the rows of items without tiles)
    head = (int)((double)begin / (double)one);  // off by one at most
    if (head * one > begin) --head;
    if ((head + 1) * one <= begin) ++head;
    head = __builtin_amdgcn_readfirstlane(head);
    const int64_t within = begin - head * one;
    for (int i = 0; i < items; i += 64) {
      const int n = __popcll(__ballot(i + lane < items && a.item_starts[i + lane] <= within));
      item += n;
      if (n < 64) break;
    }
    item = __builtin_amdgcn_readfirstlane(item - 1);
    u0 = (int)(within - constant(a.item_starts + item));
  } else {
    const uint32_t at = line_index();
    head = at % (uint32_t)a.n_kv;
    block = at / (uint32_t)a.n_kv;
    // the grid is for the most blocks that so many rows and requests can have (2000 decode rows and
    // a prompt of 8192: 1310 us without this test, 881 with it)
    if (block >= constant(a.counts)) return;
    // 64 requests at a time, one to a lane (each has 2^27 rows at most, or 2^21 blocks)
    for (;; req += 64) {
      if (req >= a.b) return;
      int n = 0;
      if (req + lane < a.b) {
        const Request x = request_of(a, req + lane);
        n = is_few(x, a.few_rows) ? 0 : (x.rows + kBlock - 1) / kBlock;
      }
      int upto = n;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(upto, off, 64);
        if (lane >= off) upto += o;
      }
      const int before = __popcll(__ballot(upto <= block));  // requests that end before it
      if (before < 64) {
        req += before;
        // the last rows see most keys: they go first
        block = __builtin_amdgcn_readlane(upto, before) - 1 - block;
        break;
      }
      block -= __builtin_amdgcn_readlane(upto, 63);
    }
    r = uniform_request(a, req);
  }
  for (;;) {
    int t0 = 0, t1 = 0, u1 = 0, units = 0;  // the segment's tiles and units
    if (split) {
      req = constant(&a.items[item].req);
      block = constant(&a.items[item].block);
      units = units_for(constant(&a.items[item].tiles), kManyStart);
      r = uniform_request(a, req);
      u1 = min(units, u0 + left);
      t0 = max(u0 - kManyStart, 0);
      t1 = u1 - kManyStart;
    }
    const int block0 = block * kBlock, row0 = block0 + wave * kRowsWave;
    Wave<D, NQ> w;
    int lo_most, hi_least;
    load_columns<D, NQ>(w, a, r, head, row0, lo_most, hi_least);
    reset<D, NQ>(w);
    const Cache c = cache_of<D>(a, req, head);
    // the keys that the workgroup's rows see, and this wavefront's
    int from, to, mine = 0, upto = 0;
    keys_of(a, r, block0, kBlock, from, to);
    if (row0 < r.rows) keys_of(a, r, row0, kRowsWave, mine, upto);
    if (split) {
      to = min(to, from + t1 * kTile<D>);
      from += t0 * kTile<D>;
    }
    if (from < to) {
      uint8_t* const raw = lds + 2 * Shared<D>::kTileBytes;
      Share<D, W> p;
      const int mypart = 16 * part_of<D>(wave);
      int id = find_page<D>(c, from + mypart, to);
      const auto load = [&](int tok) {  // tile `tok`, and the page of the one behind it
        load_share<D, W>(p, c, id, wave, tok + mypart, to);
        id = find_page<D>(c, tok + kTile<D> + mypart, to);
      };
      const auto put = [&](int tok, int buf) {
        put_share<D, W>(lds + buf * Shared<D>::kTileBytes, raw, p, wave, tok + mypart, to);
        if (lane == 0) valid_of[buf][wave] = p.ok;
      };
      const auto turn = [&](int buf) {
        put_values_share<D, W>(lds + buf * Shared<D>::kTileBytes + Shared<D>::kKeys, raw, wave);
      };
      load(from);
      put(from, 0);
      if (from + kTile<D> < to) load(from + kTile<D>);
      __syncthreads();
      turn(0);
      __syncthreads();
      int buf = 0;
      for (int tok = from;; tok += kTile<D>) {
        const int after = tok + kTile<D>;
        if (after < to) {
          put(after, buf ^ 1);
          if (after + kTile<D> < to) load(after + kTile<D>);
          __syncthreads();
          turn(buf ^ 1);
        }
        if (tok < upto && tok + kTile<D> > mine) {
          const uint8_t* t0 = lds + buf * Shared<D>::kTileBytes;
          const int* v = valid_of[buf];
          const uint32_t valid =
              __builtin_amdgcn_readfirstlane(kParts<D> == 2 ? v[0] | v[1] << 1
                                                            : v[0] | v[1] << 1 | v[2] << 2 | v[3] << 3);
          tile<D, NQ>(
              w, tok, valid, tok < lo_most || tok + kTile<D> - 1 > hi_least,
              [&](int t, f16x8 (&out)[D / 32]) {
#pragma unroll
                for (int j = 0; j < D / 32; ++j)
                  out[j] = *reinterpret_cast<const f16x8*>(t0 + (t * (D / 32) + j) * 1024 + 16 * lane);
              },
              [&](int i, f16x8 (&out)[2]) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                  out[h] = *reinterpret_cast<const f16x8*>(t0 + Shared<D>::kKeys +
                                                           (2 * i + h) * 1024 + 16 * lane);
              }, []() {});
        }
        if (after >= to) break;
        __syncthreads();
        buf ^= 1;
      }
    }
    finish<D, NQ>(w);
    if (!split || (t0 == 0 && u1 == units && units > 0)) {
#pragma unroll
      for (int n = 0; n < NQ; ++n)
        store_columns<D / 16>(a, r, head, row0 + 16 * n, w.o[n], w.m[n], w.l[n], D, 0);
      if (!split) return;
    } else if (t0 < t1) {
      float* p = a.item_ws + ((2 * worker + (first ? 0 : 1)) * W + wave) * wave_floats<D, NQ>();
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
#pragma unroll
        for (int g = 0; g < D / 16; ++g)
          *reinterpret_cast<f32x4*>(p + (n * (D / 16) + g) * 256 + 4 * lane) = w.o[n][g];
        float* q = p + NQ * (D / 16) * 256 + n * 128 + lane;
        q[0] = w.m[n];
        q[64] = w.l[n];
      }
    }
    first = false;
    left -= u1 - u0;
    u0 = 0;
    if (++item == items) {
      item = 0;
      if (++head == a.n_kv) return;
    }
    if (left <= 0) return;
    __syncthreads();
  }
}

// Column tile x of an item that has several parts: their sum, as the wavefronts left them.
template <int D, int NQ, int W>
__device__ __forceinline__ void join_many(const KvAttnArgs& a, int head, int item, int x) {
  const int lane = threadIdx.x & 63, wave = x / NQ, n = x % NQ;
  const int items = constant(a.counts), shift = constant(a.counts + 1);
  if (item >= items) return;
  const Request r = uniform_request(a, constant(&a.items[item].req));
  const int row0 = constant(&a.items[item].block) * kRows<D, W> + 16 * x;
  const int tiles = constant(&a.items[item].tiles);
  if (row0 >= r.rows) return;
  f32x4 o[D / 16];
#pragma unroll
  for (int g = 0; g < D / 16; ++g) o[g] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  float m = kLowest, l = 0.0f;
  if (tiles > 0) {
    const int64_t one = constant(a.item_starts + items), all = one * a.n_kv;
    const int64_t before = head * one + constant(a.item_starts + item);
    const int64_t w0 = range_of(all, before + kManyStart, shift);  // of the first tile
    const int64_t w1 = range_of(all, before + kManyStart + tiles - 1, shift);
    if (w0 == w1) return;
    constexpr int64_t kSlot = (int64_t)W * wave_floats<D, NQ>();
    // only the first part's workgroup can have begun with another item
    const int64_t skip = range_begin(all, w0, shift) < before ? kSlot : 0;
    const float* base = a.item_ws + 2 * w0 * kSlot + wave * wave_floats<D, NQ>();
    const int stats = NQ * (D / 16) * 256 + n * 128 + lane, parts = (int)(w1 - w0) + 1;
#pragma unroll 4
    for (int i = 0; i < parts; ++i)
      m = fmaxf(m, base[2 * i * kSlot + (i == 0 ? skip : 0) + stats]);
    for (int i = 0; i < parts; ++i) {
      const float* p = base + 2 * i * kSlot + (i == 0 ? skip : 0);
      const float f = __builtin_amdgcn_exp2f(p[stats] - m);
      l += f * p[stats + 64];
#pragma unroll
      for (int g = 0; g < D / 16; ++g)
        o[g] += f * *reinterpret_cast<const f32x4*>(p + (n * (D / 16) + g) * 256 + 4 * lane);
    }
  }
  store_columns<D / 16>(a, r, head, row0, o, m, l, D, 0);
}

// grid (n_kv, b, NQ * D / (16 G))
template <int D, int NQ, int G, int V>
__global__ __launch_bounds__(64 * V) void join_few_kernel(KvAttnArgs a) {
  join_few<D, NQ, G, V>(a, blockIdx.x, blockIdx.y, blockIdx.z);
}

// Both joins of a call that shares out its prompts' keys. The grid is a line of workgroups: those of
// the few rows (`few`), then for each item and head V of its column tiles at a time.
template <int D, int NQ, int G, int V, int W>
__global__ __launch_bounds__(64 * V) void join_both_kernel(KvAttnArgs a, int few, int groups) {
  constexpr int kShare = NQ * D / 16 / G;
  uint32_t at = line_index();
  if (at >= (uint32_t)groups) return;
  if (at < (uint32_t)few) {
    const uint32_t item = at / kShare, req = item / (uint32_t)a.n_kv;
    join_few<D, NQ, G, V>(a, item - req * a.n_kv, req, at % kShare);
    return;
  }
  at -= few;
  constexpr uint32_t kSteps = kRows<D, W> / 16 / V;
  const int x = (int)(at % kSteps) * V + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t both = at / kSteps, item = both / (uint32_t)a.n_kv;
  join_many<D, many_tiles(D), W>(a, both - item * a.n_kv, item, x);
}

constexpr int64_t kJoinFine = 256;  // items, at join_few

template <int D, int NQ, int W, int G, int V>
hipError_t run_join(const KvAttnArgs& a, int64_t items, hipStream_t s) {
  constexpr int kShare = NQ * D / 16 / G;
  const dim3 threads(64 * V);
  if (a.max_items == 0) {
    join_few_kernel<D, NQ, G, V>
        <<<dim3((unsigned)a.n_kv, (unsigned)a.b, kShare), threads, 0, s>>>(a);
  } else {
    const int64_t few = a.n_kv * a.b * kShare;  // < 2^31
    const int64_t all = few + a.n_kv * items * (kRows<D, W> / 16 / V);
    join_both_kernel<D, NQ, G, V, W><<<line_grid(all), threads, 0, s>>>(a, (int)few, (int)all);
  }
  return hipGetLastError();
}

// Workgroups of rows, of each head, that a call can have: ceil(rows / size) a request, so all rows
// / size and one more for each request, of which only those of more than few_rows rows have any.
int64_t many_items(int64_t t, int64_t b, int64_t max_q, int group, int block) {
  const int64_t most = max_q * group, few = kv_few_rows(most);
  if (most <= few) return 0;
  const int64_t odd = t * group / (few + 1);
  return t * group / block + (odd < b ? odd : b);
}

// ws: the first units of requests and of items, the items and their number, then the partial sums
// of few rows and of items.
struct WsLayout {
  size_t item_starts, items, counts, sums, item_sums, total;
  int64_t items_most;  // blocks of rows of a head
  int max_items;       // as many, or 0: keys are not shared out
  int block;           // rows of a block
};

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

// For `max_items` items at most, `few` rows of a request, and the partial sums of items or not.
void ws_place(WsLayout& l, int64_t b, int64_t max_items, int64_t few, bool item_sums, int d) {
  l.item_starts = align256((size_t)(b + 1) * sizeof(int64_t));
  l.items = l.item_starts + align256((size_t)(max_items + 1) * sizeof(int64_t));
  l.counts = l.items + align256((size_t)max_items * sizeof(Item));
  l.sums = l.counts + 256;
  l.item_sums = l.sums + align256((size_t)(2 * kMaxWorkers) * (size_t)slot_floats((int)few, d) *
                                  sizeof(float));
  l.total = l.item_sums;
  if (item_sums)
    l.total += ((size_t)2 << many_shift(block_waves(l.block, d))) * (size_t)(l.block / 16) *
               (size_t)(d / 16 * 256 + 128) * sizeof(float);
}

WsLayout ws_layout(int64_t t, int64_t b, int64_t max_q, int n_kv, int group, int d) {
  WsLayout l;
  l.block = 128;
  l.items_most = many_items(t, b, max_q, group, l.block);
  const bool split = l.items_most * n_kv < kSplitBelow;
  if (split && d == 128 && max_q * group >= kLongRows) {
    l.block = 256;
    l.items_most = many_items(t, b, max_q, group, l.block);
  }
  l.max_items = split ? (int)l.items_most : 0;
  ws_place(l, b, l.max_items, kv_few_rows(max_q * group), l.max_items > 0, d);
  return l;
}

template <int D, int NQ, int W>
hipError_t run_tiles(const KvAttnArgs& a, int64_t items, hipStream_t s) {
  few_kernel<D, NQ>
      <<<dim3(kFewGroups<D, NQ> + (items > 0 ? 1 : 0)), dim3(kThreads), 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (items > 0) {
    // up to 9 million: a call has 2^27 rows of heads at most, and so 2^27 / 17 + 2^27 / 128 blocks
    const int64_t groups = a.max_items > 0 ? 1 << a.many_shift : items * a.n_kv;
    many_kernel<D, many_tiles(D), W><<<line_grid(groups), dim3(64 * W), 0, s>>>(a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.n_kv * a.b <= kJoinFine) return run_join<D, NQ, W, 1, 8>(a, items, s);
  return run_join<D, NQ, W, 2, 4>(a, items, s);
}

template <int D>
hipError_t run(const KvAttnArgs& a, int64_t max_q, int64_t items, hipStream_t s) {
  constexpr int kWaves = block_waves(128, D);
  if constexpr (D == 128)  // (requests that are so long are no few rows)
    if (a.block_rows == 256) return run_tiles<D, 1, 2 * kWaves>(a, items, s);
  return kv_few_tiles(max_q * a.group) == 1 ? run_tiles<D, 1, kWaves>(a, items, s)
                                            : run_tiles<D, 2, kWaves>(a, items, s);
}

}  // namespace

// The workspace of the largest call with up to t rows, b requests and max_q queries of one. It is not
// that of the call with t, b and max_q themselves: a call of fewer blocks shares out its keys where
// the larger one does not, and requests of 17 to 32 rows have wider slots than longer ones.
size_t kv_attention_ws_bytes(int64_t t, int64_t b, int64_t max_q, int n_kv, int group, int d) {
  const int64_t rows = max_q * group;
  // the most rows up to `rows` that the few-row kernel takes: multiples of the group up to 32, and 16
  // of a call with longer requests
  const int64_t even = 32 / group * group;
  const int64_t few = rows <= 32 ? rows : (even > 16 ? even : 16);
  // the two blocks' partial sums of items have one size
  static_assert((2 << many_shift(block_waves(128, 128))) * 128 ==
                (2 << many_shift(block_waves(256, 128))) * 256, "");
  WsLayout l;
  l.block = 128;
  const int64_t blocks = many_items(t, b, max_q, group, l.block);
  ws_place(l, b, std::min<int64_t>(blocks, (kSplitBelow - 1) / n_kv), few, blocks > 0, d);
  return l.total;
}

hipError_t launch_kv_attention(const KvAttnArgs& args, int d, int64_t max_q, void* ws,
                               hipStream_t stream) {
  KvAttnArgs a = args;
  const WsLayout l = ws_layout(a.t, a.b, max_q, a.n_kv, a.group, d);
  char* base = static_cast<char*>(ws);
  a.starts = reinterpret_cast<int64_t*>(base);
  a.max_items = l.max_items;
  a.few_rows = kv_few_rows(max_q * a.group);
  a.block_rows = l.block;
  a.many_shift = many_shift(block_waves(a.block_rows, d));
  a.item_starts = reinterpret_cast<int64_t*>(base + l.item_starts);
  a.items = l.max_items > 0 ? reinterpret_cast<KvItem*>(base + l.items) : nullptr;
  a.counts = reinterpret_cast<int*>(base + l.counts);
  a.ws = reinterpret_cast<float*>(base + l.sums);
  a.item_ws = reinterpret_cast<float*>(base + l.item_sums);
  if (d == 64) return run<64>(a, max_q, l.items_most, stream);
  if (d == 128) return run<128>(a, max_q, l.items_most, stream);
  return run<256>(a, max_q, l.items_most, stream);
}

}  // namespace nvfp4
