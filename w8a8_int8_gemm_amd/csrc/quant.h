// quant.h -- the per-token quantizer's arithmetic, shared by the kernels that
// quantize BF16 rows (rowwise.hip) and the ones that quantize a norm's output
// (norm.hip).  Not part of the public ABI (include/w8a8.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w8a8 {

// Per-row constants of the quantizer.  For rows whose scale is a normal
// number the codes come from u = fma(x, 1/s, 128): the reciprocal (one
// IEEE division per row), the product and the sum together stay within
// 2.3e-5 of 128 + RN(x/s) (|x/s| <= 127 + 2^-17; x any binary32 value up
// to the row's maximum, BF16 or not), so when u is farther
// than 2^-14 from a half-integer, rounding u to the nearest integer gives
// exactly 128 + round_half_even(RN(x/s)).  The remaining elements (about
// one in 8000) and rows with a subnormal scale use the division itself.
struct QuantRow {
  float s, r;
  bool fast;
};

__device__ __forceinline__ QuantRow quant_row(float amax) {
  QuantRow q;
  q.s = amax / 127.0f;
  q.fast = q.s >= 0x1p-126f;
  q.r = q.fast ? 1.0f / q.s : 0.0f;
  return q;
}

// Code of one value as the byte (q + 128), q = clamp(rint(x / s)).
__device__ __noinline__ float quant_biased_exact(float x, float s) {
  const float q = fminf(fmaxf(rintf(x / s), -127.0f), 127.0f);
  return q + 128.0f;  // exact small integer
}

// Four values -> four INT8 codes in one dword.  The closeness test runs on
// the four values together; in the rare group where one is close to a
// half-integer (or the row needs the exact path), every code of the group
// comes from the division.
__device__ __forceinline__ uint32_t quant4_f32(const float f[4],
                                               const QuantRow &R) {
  float u[4], d[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    u[e] = fmaf(f[e], R.r, 128.0f);
    d[e] = fabsf(__builtin_amdgcn_fractf(u[e]) - 0.5f);
  }
  const float dmin = fminf(fminf(d[0], d[1]), fminf(d[2], d[3]));
  if (!R.fast || !(dmin > 0x1p-14f)) {
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] = quant_biased_exact(f[e], R.s);
  }
  uint32_t out = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e)  // nearest integer in [0, 255] as byte e
    out = __builtin_amdgcn_cvt_pk_u8_f32(u[e], e, out);
  return out ^ 0x80808080u;  // biased byte -> two's complement code
}

}  // namespace w8a8
