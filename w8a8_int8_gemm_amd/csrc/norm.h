// norm.h -- launcher of the block norms (norm.hip): norm, modulation, gate and
// residual of a transformer block.  Not part of the public ABI
// (include/w8a8.h); arguments are validated by the API layer before.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w8a8 {

// One call.  A null vector is absent (weight 1, bias 0, scale and shift 0,
// gate 1); strides in elements; `row` null: modulation row m * row_step.
struct NormArgs {
  const uint16_t *x, *branch;  // branch null: no residual part
  uint16_t *r, *y;             // y null: none, or codes instead
  int8_t *q;
  float *qs;
  const uint16_t *post_weight, *post_bias, *weight, *bias;
  const uint16_t *scale, *shift, *gate;
  int64_t scale_stride, shift_stride, gate_stride;
  const int32_t *row;
  int64_t M;
  int rows, row_step, H;
  int post_kind, kind;  // w8a8_norm_kind_t
  float post_eps, eps, residual_scale;
};

hipError_t launch_norm(const NormArgs &a, hipStream_t stream);

}  // namespace w8a8
