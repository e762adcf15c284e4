// w4.hip -- linear over few tokens with packed 4-bit weights and group scales,
// and the converters that write the packed layout (include/w8a8.h).
//
// y[m,n] = sum_g s[n,g] * sum_{k in g} x[m,k] * (u[n,k] - 8) + bias[n].
//
// Bound by HBM: half a byte a weight (plus 2 / group), read once; x and y are
// small.  The products run on v_mfma_f32_16x16x32_bf16, tokens as the A
// operand and channels as B, so a lane's results belong to one channel and
// take one scale.
#include "internal.h"
#include "w4.h"
#include "w8a8.h"

namespace w8a8 {
namespace {

typedef unsigned v4u __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

// A packed block: 16 channels x 128 inputs, 16 bytes a lane.
constexpr int kBlockN = 16, kBlockK = 128, kBlockBytes = 1024;

// ---------------------------------------------------------------------------
// converters: one wave per block, each lane writing its own 16 bytes
// ---------------------------------------------------------------------------

constexpr int kPackThreads = 256;

// The input whose code lies in the low half of byte b of lane quarter q; the
// high half holds the input 4 further.
__device__ __forceinline__ int packed_k(int q, int b) {
  return 32 * (b >> 2) + 8 * q + (b & 3);
}

__global__ __launch_bounds__(kPackThreads) void w4_pack_kernel(
    const int8_t *codes, const uint16_t *scales, int64_t blocks, int kblocks,
    int group, uint8_t *w4, uint16_t *scale) {
  const int64_t blk =
      (int64_t)blockIdx.x * (kPackThreads / 64) + (threadIdx.x >> 6);
  if (blk >= blocks) return;
  const int lane = threadIdx.x & 63, q = lane >> 4;
  const int64_t K = (int64_t)kblocks * kBlockK;
  const int64_t n = blk / kblocks * kBlockN + (lane & 15);
  const int64_t k0 = blk % kblocks * kBlockK;
  const int8_t *row = codes + n * K + k0;
  uint32_t out[4];
  for (int d = 0; d < 4; ++d) {
    uint32_t w = 0;
    for (int b = 0; b < 4; ++b) {
      const int k = packed_k(q, 4 * d + b);
      const int lo = min(max((int)row[k], -8), 7) + 8;
      const int hi = min(max((int)row[k + 4], -8), 7) + 8;
      w |= (uint32_t)(lo | hi << 4) << (8 * b);
    }
    out[d] = w;
  }
  reinterpret_cast<v4u *>(w4 + blk * kBlockBytes)[lane] =
      v4u{out[0], out[1], out[2], out[3]};
  const int groups = kBlockK / group;
  if (q < groups)
    scale[(blk * kBlockN + (lane & 15)) * groups + q] =
        scales[n * (K / group) + k0 / group + q];
}

__global__ __launch_bounds__(kPackThreads) void w4_quantize_kernel(
    const uint16_t *w, int64_t blocks, int kblocks, int group, uint8_t *w4,
    uint16_t *scale) {
  const int64_t blk =
      (int64_t)blockIdx.x * (kPackThreads / 64) + (threadIdx.x >> 6);
  if (blk >= blocks) return;
  const int lane = threadIdx.x & 63, q = lane >> 4;
  const int64_t K = (int64_t)kblocks * kBlockK;
  const int64_t n = blk / kblocks * kBlockN + (lane & 15);
  const int64_t k0 = blk % kblocks * kBlockK;
  // chunk d of a lane: 8 inputs from 32 d + 8 q on, so a group of 32 is chunk
  // d of the four lanes of a channel
  const v4u *row = reinterpret_cast<const v4u *>(w + n * K + k0);
  v4u c[4];
  float amax[4];
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    c[d] = row[4 * d + q];
    float a = 0.0f;
    const uint32_t p[4] = {c[d].x, c[d].y, c[d].z, c[d].w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      a = fmaxf(a, fmaxf(fabsf(bf16_to_f32(p[e] & 0xFFFFu)),
                         fabsf(bf16_to_f32(p[e] >> 16))));
    a = fmaxf(a, __shfl_xor(a, 16, 64));
    amax[d] = fmaxf(a, __shfl_xor(a, 32, 64));
  }
  if (group >= 64) {
    amax[0] = amax[1] = fmaxf(amax[0], amax[1]);
    amax[2] = amax[3] = fmaxf(amax[2], amax[3]);
  }
  if (group == 128)
    amax[0] = amax[1] = amax[2] = amax[3] = fmaxf(amax[0], amax[2]);
  uint32_t out[4];
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    // the scale is rounded to BF16 before the codes are taken from it; a
    // group too small for that rounding takes the smallest BF16 above zero
    uint32_t s16 = amax[d] == 0.0f ? 0x3F80u : f32_to_bf16_rne(amax[d] / 7.0f);
    s16 = s16 == 0 ? 1u : s16;
    const float s = bf16_to_f32(s16);
    const uint32_t p[4] = {c[d].x, c[d].y, c[d].z, c[d].w};
    uint32_t r = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float f = bf16_to_f32(e & 1 ? p[e / 2] >> 16 : p[e / 2] & 0xFFFFu);
      const int u = (int)fminf(fmaxf(rintf(f / s), -7.0f), 7.0f) + 8;
      r |= (uint32_t)u << (8 * (e & 3) + (e & 4));
    }
    out[d] = r;
    const int groups = kBlockK / group;
    if (q == 0 && d % (group / 32) == 0)
      scale[(blk * kBlockN + (lane & 15)) * groups + d / (group / 32)] =
          (uint16_t)s16;
  }
  reinterpret_cast<v4u *>(w4 + blk * kBlockBytes)[lane] =
      v4u{out[0], out[1], out[2], out[3]};
}

// ---------------------------------------------------------------------------
// the product
// ---------------------------------------------------------------------------

// Eight codes -> eight BF16 values u.  A byte u in 0..15 is the e4m3 number
// u * 2^-9 (its subnormals and first binade are linear in the byte), so the
// FP8 conversion with a factor of 2^9 gives u exactly.  Bytes 0..3 hold inputs
// 0..3 in their low halves and inputs 4..7 in their high ones.
__device__ __forceinline__ v8bf codes8(uint32_t v) {
  const uint32_t lo = v & 0x0F0F0F0Fu, hi = (v >> 4) & 0x0F0F0F0Fu;
  union {
    bf2v p[4];
    v8bf v;
  } u;
  u.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, false);
  u.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, true);
  u.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, false);
  u.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, true);
  return u.v;
}

__device__ __forceinline__ v4f mfma(v4u a, v8bf b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(
      __builtin_bit_cast(v8bf, a), b, c, 0, 0, 0);
}

// A work group owns 16 T channels and up to 16 F tokens; its W waves take the
// K blocks in turn and join their sums through LDS.  Lane (r, q) of a fragment
// holds token r (A) or channel r (B) at inputs 8 q .. 8 q + 7 of 32, and
// results i = 0..3 of token 4 q + i and channel r.
//
// The -8 of every code: its products with x do not depend on the channel, so
// per group they are summed once (B = -8) and are where each channel's sum
// starts.
template <int F, int T, int W, int G>
__global__ __launch_bounds__(W * 64) void w4_linear_kernel(
    const uint16_t *x, const uint8_t *w4, const uint16_t *scale,
    const uint16_t *bias, uint16_t *y, int64_t M, int tiles, int kblocks) {
  constexpr int GPB = kBlockK / G;  // groups a block
  __shared__ v4f red[W][F][T][64];
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tile0 = blockIdx.x * T;
  const int64_t m0 = (int64_t)blockIdx.y * (16 * F);
  const int64_t K = (int64_t)kblocks * kBlockK, N = (int64_t)tiles * kBlockN;

  v8bf minus8;
#pragma unroll
  for (int e = 0; e < 8; ++e) minus8[e] = (__bf16)-8.0f;
  v4f acc[F][T];
#pragma unroll
  for (int f = 0; f < F; ++f)
#pragma unroll
    for (int t = 0; t < T; ++t) acc[f][t] = v4f{0, 0, 0, 0};

  for (int b = wave; b < kblocks; b += W) {
    v4u wv[T];
    float sc[T][GPB];
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const int64_t blk = (int64_t)min(tile0 + t, tiles - 1) * kblocks + b;
      wv[t] = reinterpret_cast<const v4u *>(w4 + blk * kBlockBytes)[lane];
#pragma unroll
      for (int g = 0; g < GPB; ++g)
        sc[t][g] = bf16_to_f32(scale[(blk * kBlockN + r) * GPB + g]);
    }
    v4u xa[F][4];
#pragma unroll
    for (int f = 0; f < F; ++f) {
      const int64_t m = m0 + 16 * f + r;
      const v4u *xr = reinterpret_cast<const v4u *>(x + m * K + b * kBlockK);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        xa[f][j] = m < M ? xr[4 * j + q] : v4u{0, 0, 0, 0};
    }
#pragma unroll
    for (int g = 0; g < GPB; ++g) {
      v4f start[F];
#pragma unroll
      for (int f = 0; f < F; ++f) {
        start[f] = v4f{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 4 / GPB; ++j)
          start[f] = mfma(xa[f][g * (4 / GPB) + j], minus8, start[f]);
      }
#pragma unroll
      for (int t = 0; t < T; ++t) {
        v8bf wb[4 / GPB];
#pragma unroll
        for (int j = 0; j < 4 / GPB; ++j)
          wb[j] = codes8(wv[t][g * (4 / GPB) + j]);
#pragma unroll
        for (int f = 0; f < F; ++f) {
          v4f s = start[f];
#pragma unroll
          for (int j = 0; j < 4 / GPB; ++j)
            s = mfma(xa[f][g * (4 / GPB) + j], wb[j], s);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[f][t][i] = fmaf(s[i], sc[t][g], acc[f][t][i]);
        }
      }
    }
  }

#pragma unroll
  for (int f = 0; f < F; ++f)
#pragma unroll
    for (int t = 0; t < T; ++t) red[wave][f][t][lane] = acc[f][t];
  __syncthreads();
  // A thread finishes four tokens of one channel.
  for (int o = threadIdx.x; o < F * T * 64; o += W * 64) {
    const int f = o / (64 * T), t = o / 64 % T, l = o & 63;
    v4f s = red[0][f][t][l];
#pragma unroll
    for (int w = 1; w < W; ++w) s += red[w][f][t][l];
    if (tile0 + t >= tiles) continue;
    const int64_t n = (int64_t)(tile0 + t) * kBlockN + (l & 15);
    const float b = bias ? bf16_to_f32(bias[n]) : 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t m = m0 + 16 * f + 4 * (l >> 4) + i;
      if (m < M) y[m * N + n] = (uint16_t)pack_bf16x2(s[i] + b, 0.0f);
    }
  }
}

template <int F, int T, int W>
hipError_t launch_linear(const uint16_t *x, const uint8_t *w4,
                         const uint16_t *scale, const uint16_t *bias,
                         uint16_t *y, int64_t M, int tiles, int kblocks,
                         int group, hipStream_t stream) {
  const dim3 grid((unsigned)((tiles + T - 1) / T),
                  (unsigned)((M + 16 * F - 1) / (16 * F)));
#define W8A8_W4_LAUNCH(G)                                                   \
  hipLaunchKernelGGL((w4_linear_kernel<F, T, W, G>), grid, dim3(W * 64), 0, \
                     stream, x, w4, scale, bias, y, M, tiles, kblocks)
  if (group == 32)
    W8A8_W4_LAUNCH(32);
  else if (group == 64)
    W8A8_W4_LAUNCH(64);
  else
    W8A8_W4_LAUNCH(128);
#undef W8A8_W4_LAUNCH
  return hipGetLastError();
}

dim3 pack_grid(int64_t blocks) {
  constexpr int per = kPackThreads / 64;
  return dim3((unsigned)((blocks + per - 1) / per));
}

}  // namespace

hipError_t launch_w4_quantize(const uint16_t *w, int64_t N, int64_t K,
                              int group, uint8_t *w4, uint16_t *scale,
                              hipStream_t stream) {
  const int kblocks = (int)(K / kBlockK);
  const int64_t blocks = N / kBlockN * kblocks;
  hipLaunchKernelGGL(w4_quantize_kernel, pack_grid(blocks), dim3(kPackThreads),
                     0, stream, w, blocks, kblocks, group, w4, scale);
  return hipGetLastError();
}

hipError_t launch_w4_pack(const int8_t *codes, const uint16_t *scales,
                          int64_t N, int64_t K, int group, uint8_t *w4,
                          uint16_t *scale, hipStream_t stream) {
  const int kblocks = (int)(K / kBlockK);
  const int64_t blocks = N / kBlockN * kblocks;
  hipLaunchKernelGGL(w4_pack_kernel, pack_grid(blocks), dim3(kPackThreads), 0,
                     stream, codes, scales, blocks, kblocks, group, w4, scale);
  return hipGetLastError();
}

hipError_t launch_w4_linear(const uint16_t *x, const uint8_t *w4,
                            const uint16_t *scale, const uint16_t *bias,
                            uint16_t *y, int64_t M, int64_t N, int64_t K,
                            int group, hipStream_t stream) {
  const int tiles = (int)(N / kBlockN), kblocks = (int)(K / kBlockK);
  if (M <= 16)
    return launch_linear<1, 1, 8>(x, w4, scale, bias, y, M, tiles, kblocks,
                                  group, stream);
  return launch_linear<4, 2, 8>(x, w4, scale, bias, y, M, tiles, kblocks,
                                group, stream);
}

}  // namespace w8a8
