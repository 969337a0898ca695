// Block scales and element codes of the OCP Microscaling formats, shared by the
// quantisers (mx.hip), the MXFP4 experts' epilogue (mx4.hip) and the norms
// (block_norm.hip).
#pragma once

#include "common.hpp"

namespace moe {

// E8M0 exponent byte of an MX block with largest magnitude amax: floor(log2 amax) -
// emax_elem + 127 (emax_elem 8 for E4M3, 2 for E2M1), in [0, 254]; 127 for a zero block.
__device__ __forceinline__ int mx_scale_exp(float amax, int emax_elem) {
  if (!(amax > 0.0f)) return 127;
  int e2;
  frexpf(amax, &e2);                        // amax = f * 2^e2, f in [0.5, 1)
  const int e = (e2 - 1) - emax_elem + 127;
  return e < 0 ? 0 : (e > 254 ? 254 : e);
}

// Nearest E2M1 code (ties to the even code, saturating at 6; NaN -> 0).
__device__ __forceinline__ uint32_t float_to_fp4e2m1(float v) {
  const float a = fabsf(v);
  uint32_t c;
  if (!(a == a)) return 0u;
  if (a <= 0.25f) c = 0u;
  else if (a < 0.75f) c = 1u;
  else if (a <= 1.25f) c = 2u;
  else if (a < 1.75f) c = 3u;
  else if (a <= 2.5f) c = 4u;
  else if (a < 3.5f) c = 5u;
  else if (a <= 5.0f) c = 6u;
  else c = 7u;
  return (v < 0.0f && c != 0u) ? (c | 8u) : c;
}

// Eight floats at E8M0 scale X = 2^(e - 127): the codes that float_to_fp4e2m1 gives for v / X,
// packed from the low nibble up, by gfx950's scaled conversion (v_cvt_scalef32_pk_fp4_f32: nearest,
// ties to even, saturating; on MI355X its codes equal the comparisons above on 2^20 magnitudes up to
// 8 X, the borders' neighbours, infinity, and scales from 2^-127 to 2^123). It codes -0 as 8 and
// NaN as 7; both become 0 here.
__device__ __forceinline__ uint32_t pk8_fp4e2m1(const float* v, float X) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = v[i] == v[i] ? v[i] : 0.0f;
  uint32_t q = 0u;
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f[0], f[1], X, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f[2], f[3], X, 1);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f[4], f[5], X, 2);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f[6], f[7], X, 3);
  const uint32_t mag = q & 0x77777777u;
  return mag | (q & (mag + 0x77777777u) & 0x88888888u);   // a sign only where there is a magnitude
}

}  // namespace moe
