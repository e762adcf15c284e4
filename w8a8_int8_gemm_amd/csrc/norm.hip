// norm.hip -- the block norms for gfx950: RMS or layer norm of a row with
// modulation, and the post-norm, gate and residual sum in front of it, to
// BF16 rows or to INT8 codes with per-token scales (the formulas are in
// include/w8a8.h).
//
// Bound by HBM: 4 bytes a value for a norm to BF16, 3 to codes, 8 and 7 with
// the residual part; a dozen binary32 operations a value.  A row is read once
// and stays in registers through all of its reductions.
#include "internal.h"
#include "norm.h"
#include "quant.h"
#include "w8a8.h"

namespace w8a8 {
namespace {

typedef unsigned v4u __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

enum NormOut : int { OUT_NONE = 0, OUT_ROW = 1, OUT_CODES = 2 };

struct F8 {
  float v[8];
};

__device__ __forceinline__ F8 unpack8(v4u c) {
  F8 f;
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f.v[2 * e] = __uint_as_float(w[e] << 16);
    f.v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
  }
  return f;
}

__device__ __forceinline__ v4u pack8(const F8 &f) {
  return v4u{pack_bf16x2(f.v[0], f.v[1]), pack_bf16x2(f.v[2], f.v[3]),
             pack_bf16x2(f.v[4], f.v[5]), pack_bf16x2(f.v[6], f.v[7])};
}

// Chunk j (8 values) of a vector, or eight times `absent`.
__device__ __forceinline__ F8 vec8(const uint16_t *p, int j, float absent) {
  if (p) return unpack8(reinterpret_cast<const v4u *>(p)[j]);
  F8 f;
#pragma unroll
  for (int e = 0; e < 8; ++e) f.v[e] = absent;
  return f;
}

template <bool MAX>
__device__ __forceinline__ float join(float a, float b) {
  return MAX ? fmaxf(a, b) : a + b;
}

// Sum or maximum over the work group; `part` holds kWaves values and is free
// for the next call after the barrier at its start.
template <bool MAX>
__device__ __forceinline__ float block_reduce(float v, float *part) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1)
    v = join<MAX>(v, __shfl_xor(v, off, 64));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  v = part[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) v = join<MAX>(v, part[w]);
  return v;
}

// Normalizes the row held in v in place, without weight and bias: the mean
// first, then the squares of the differences, so that a large mean costs the
// variance no digits.  Values past the row's end are zero and stay unused.
template <int CH>
__device__ __forceinline__ void normalize(F8 (&v)[CH], int kind, float eps,
                                          int H, float *part) {
  const int chunks = H >> 3;
  if (kind == W8A8_NORM_NONE) return;
  if (kind == W8A8_NORM_LAYER) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += v[i].v[e];
    const float mean = block_reduce<false>(sum, part) / (float)H;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const bool ok = i * kThreads + (int)threadIdx.x < chunks;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i].v[e] = ok ? v[i].v[e] - mean : 0.0f;
    }
  }
  float sq = 0.0f;
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) sq = fmaf(v[i].v[e], v[i].v[e], sq);
  const float rs =
      rsqrtf(block_reduce<false>(sq, part) / (float)H + eps);
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i].v[e] *= rs;
}

template <int CH, bool RES, int OUT>
__global__ __launch_bounds__(kThreads) void norm_kernel(NormArgs a) {
  __shared__ float part[kWaves];
  const int64_t m = blockIdx.x;
  const int t = threadIdx.x;
  const int chunks = a.H >> 3;
  const int64_t at = m * (int64_t)a.H;
  const v4u *xr = reinterpret_cast<const v4u *>(a.x + at);
  const int64_t mr = a.row ? (int64_t)a.row[m] : m * a.row_step;

  if (mr < 0 || mr >= a.rows) {  // padding: r = x, the rest zero
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int j = i * kThreads + t;
      if (j >= chunks) continue;
      if (RES && a.r != a.x) reinterpret_cast<v4u *>(a.r + at)[j] = xr[j];
      if (OUT == OUT_ROW) reinterpret_cast<v4u *>(a.y + at)[j] = v4u{0, 0, 0, 0};
      if (OUT == OUT_CODES)
        reinterpret_cast<uint2 *>(a.q + at)[j] = make_uint2(0, 0);
    }
    if (OUT == OUT_CODES && t == 0) a.qs[m] = 0.0f;
    return;
  }

  F8 v[CH];
  if (RES) {
    const v4u *br = reinterpret_cast<const v4u *>(a.branch + at);
    const uint16_t *gate = a.gate ? a.gate + mr * a.gate_stride : nullptr;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int j = i * kThreads + t;
      v[i] = unpack8(j < chunks ? br[j] : v4u{0, 0, 0, 0});
    }
    normalize<CH>(v, a.post_kind, a.post_eps, a.H, part);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int j = i * kThreads + t;
      if (j >= chunks) continue;
      const F8 x = unpack8(xr[j]);
      const F8 w = vec8(a.post_weight, j, 1.0f);
      const F8 b = vec8(a.post_bias, j, 0.0f);
      const F8 g = vec8(gate, j, 1.0f);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[i].v[e] = fmaf(g.v[e], fmaf(v[i].v[e], w.v[e], b.v[e]),
                         a.residual_scale * x.v[e]);
      reinterpret_cast<v4u *>(a.r + at)[j] = pack8(v[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int j = i * kThreads + t;
      v[i] = unpack8(j < chunks ? xr[j] : v4u{0, 0, 0, 0});
    }
  }
  if (OUT == OUT_NONE) return;

  normalize<CH>(v, a.kind, a.eps, a.H, part);
  const uint16_t *scale = a.scale ? a.scale + mr * a.scale_stride : nullptr;
  const uint16_t *shift = a.shift ? a.shift + mr * a.shift_stride : nullptr;
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int j = i * kThreads + t;
    if (j >= chunks) continue;
    const F8 w = vec8(a.weight, j, 1.0f);
    const F8 b = vec8(a.bias, j, 0.0f);
    const F8 sc = vec8(scale, j, 0.0f);
    const F8 sh = vec8(shift, j, 0.0f);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float n = fmaf(v[i].v[e], w.v[e], b.v[e]);
      v[i].v[e] = fmaf(n, 1.0f + sc.v[e], sh.v[e]);
      amax = fmaxf(amax, fabsf(v[i].v[e]));
    }
    if (OUT == OUT_ROW) reinterpret_cast<v4u *>(a.y + at)[j] = pack8(v[i]);
  }
  if (OUT != OUT_CODES) return;
  const QuantRow R = quant_row(block_reduce<true>(amax, part));
  if (t == 0) a.qs[m] = R.s;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int j = i * kThreads + t;
    if (j >= chunks) continue;
    uint2 o = make_uint2(0, 0);
    if (R.s != 0.0f)
      o = make_uint2(quant4_f32(v[i].v, R), quant4_f32(v[i].v + 4, R));
    reinterpret_cast<uint2 *>(a.q + at)[j] = o;
  }
}

template <int CH>
void launch_ch(const NormArgs &a, hipStream_t stream) {
  const dim3 grid((unsigned)a.M), block(kThreads);
  if (a.branch) {
    if (a.q)
      hipLaunchKernelGGL((norm_kernel<CH, true, OUT_CODES>), grid, block, 0,
                         stream, a);
    else if (a.y)
      hipLaunchKernelGGL((norm_kernel<CH, true, OUT_ROW>), grid, block, 0,
                         stream, a);
    else
      hipLaunchKernelGGL((norm_kernel<CH, true, OUT_NONE>), grid, block, 0,
                         stream, a);
  } else if (a.q) {
    hipLaunchKernelGGL((norm_kernel<CH, false, OUT_CODES>), grid, block, 0,
                       stream, a);
  } else {
    hipLaunchKernelGGL((norm_kernel<CH, false, OUT_ROW>), grid, block, 0,
                       stream, a);
  }
}

}  // namespace

hipError_t launch_norm(const NormArgs &a, hipStream_t stream) {
  const int ch = (a.H / 8 + kThreads - 1) / kThreads;  // 16 at the largest H
  if (ch <= 1) launch_ch<1>(a, stream);
  else if (ch <= 2) launch_ch<2>(a, stream);
  else if (ch <= 4) launch_ch<4>(a, stream);
  else if (ch <= 8) launch_ch<8>(a, stream);
  else if (ch <= 16) launch_ch<16>(a, stream);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

}  // namespace w8a8
