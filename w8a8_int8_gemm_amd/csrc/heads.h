// heads.h -- launchers of what stands between a block's Q, K, V and its output
// projection: rotary table, head norms with rotation (heads.hip), attention
// (attention.hip).  Not part of the public ABI (include/w8a8.h); arguments are
// validated by the API layer before.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "w8a8.h"

namespace w8a8 {

// Quarter turns a position of every pair (in 64 bits), and the axis it reads.
struct RopeArgs {
  const void *pos;  // [T, axes], int32 or binary32
  float *table;     // [T, 2, pairs]
  int64_t T;
  int pos_type, axes, pairs;
  float amplitude;
  uint8_t axis[W8A8_ROPE_MAX_PAIRS];
  double quarters[W8A8_ROPE_MAX_PAIRS];
};

hipError_t launch_rope_table(const RopeArgs &a, hipStream_t stream);

// One side (queries or keys): strides in elements, w_step 0 (one weight for
// all heads) or D.  heads 0: no such side.
struct HeadSide {
  const uint16_t *x;
  uint16_t *y;
  const uint16_t *weight, *bias;
  int64_t x_stride, y_stride;
  int heads, kind, w_step;
  float eps;
};

// table null: no rotation.  row null: table row m * row_step.
struct HeadArgs {
  HeadSide side[2];
  const float *table;
  const int32_t *row;
  int64_t M;
  int rows, row_step, D, pairs, interleaved;
};

// Work-items of a launch (the API layer refuses 2^32 and more).
int64_t head_norm_items(const HeadArgs &a);
hipError_t launch_head_norm(const HeadArgs &a, hipStream_t stream);

// Offsets null: B equal sequences.  Strides in elements; a head's values are
// contiguous, the next head's follow.
struct AttnArgs {
  const uint16_t *q, *k, *v;
  uint16_t *out;
  int64_t q_stride, k_stride, v_stride, out_stride;
  const int32_t *q_offsets, *k_offsets, *k_lens;
  int Tq, Tk, B, Hq, Hk, D;
  float scale_log2;  // scale * log2(e)
  void *workspace;
  int G;  // query heads that share a key head
};

// How a call is cut: queries (times the heads that share keys) a tile, tiles
// over all sequences (an upper bound where offsets say where they end), and
// parts that the keys are split into.
struct AttnPlan {
  int config;
  int64_t tiles;
  int splits;
  size_t workspace;  // bytes of partial results (0 without a split)
};

AttnPlan plan_attention(int64_t Tq, int64_t Tk, int64_t B, bool packed,
                        int64_t Hq, int64_t Hk, int64_t D);
// Whether the launches fit the hardware's grid limits.
bool attention_launchable(const AttnPlan &plan, int64_t Hk);
hipError_t launch_attention(const AttnArgs &a, const AttnPlan &plan,
                            hipStream_t stream);

}  // namespace w8a8
