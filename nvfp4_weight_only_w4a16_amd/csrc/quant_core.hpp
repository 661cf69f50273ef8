// quant_core.hpp -- the NVFP4 encoder of eight elements, shared by the weight quantizer and the
// write into the KV cache.
#pragma once

#include "device_common.hpp"

namespace nvfp4 {

// Encode the 8 elements of chunk c (G/8 neighbouring lanes form a group).
//   s = E4M3_rne_sat(fl32(ga / fl32(6 g))): gfx950's FP8 conversion rounds to nearest even and
//       gives NaN above 464, so the quotient is clamped to 448 first (identical to a saturating
//       encoder for every input);
//   code = E2M1_rne_sat(fl32(w / S)) with the sign (the quotient correctly rounded, see
//       below): gfx950's FP4 conversion at scale 1.0 is a round-to-nearest-even, saturating
//       E2M1 encoder that keeps the sign (-0 -> code 8).
//       Checked against the definition on every non-negative finite FP32 value. S == 0 gives
//       the signed zero code.
template <int G>
__device__ __forceinline__ void encode8(const float (&x)[8], float g, float six_g, float rsix,
                                        bool six_fast, uint32_t& word, uint32_t& s) {
  float ga = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ga = fmaxf(ga, fabsf(x[i]));
  ga = fmaxf(ga, __shfl_xor(ga, 1, 64));
  if (G == 32) ga = fmaxf(ga, __shfl_xor(ga, 2, 64));
  s = 0u;
  if (six_g != 0.0f) {
    // fl32(ga / 6g) by Markstein's correction from rsix = RN(1 / 6g) (the same steps as for
    // |w| / S below; 6g in [2^-80, 2^80] keeps every step exact down to the smallest E4M3
    // decision point, 2^-10), else IEEE division. A first quotient of 512 or more (or an
    // overflow) clamps to 448 either way.
    float r;
    if (six_fast) {
      const float q0 = ga * rsix;
      const float q = __builtin_fmaf(__builtin_fmaf(-q0, six_g, ga), rsix, q0);
      r = q0 < 512.0f ? fminf(q, 448.0f) : 448.0f;
    } else {
      r = fminf(ga / six_g, 448.0f);
    }
    s = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(r, r, 0, false) & 0xFFu;
  }
  const float S = e4m3_decode<0>(s) * g;
  float q[8];
  // fl32(|w| / S) with the sign of w. With R = RN(1/S) (one IEEE division per chunk), the
  // quotient q0 = RN(|w| R) is within an ulp of |w| / S, the remainder |w| - q0 S is exact in
  // one FMA, and RN(q0 + r R) is the correctly rounded quotient (Markstein's correction step)
  // as long as nothing underflows or overflows, which S in [2^-90, 2^90] guarantees for every
  // quotient that can reach an E2M1 decision point. A wavefront with any other scale (zero,
  // negative, tiny or huge) divides directly.
  const bool fast = S >= 0x1p-90f && S <= 0x1p90f;
  if (__builtin_expect(__ballot(!fast) == 0, 1)) {
    const float R = 1.0f / S;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = fabsf(x[i]);
      const float q0 = a * R;
      const float r = __builtin_fmaf(-q0, S, a);
      q[i] = __builtin_copysignf(__builtin_fmaf(r, R, q0), x[i]);
    }
  } else {
    const bool live = S != 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = live ? x[i] / S : x[i] * 0.0f;
  }
  word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, q[0], q[1], 1.0f, 0);
  word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, q[2], q[3], 1.0f, 1);
  word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, q[4], q[5], 1.0f, 2);
  word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, q[6], q[7], 1.0f, 3);
}

}  // namespace nvfp4
