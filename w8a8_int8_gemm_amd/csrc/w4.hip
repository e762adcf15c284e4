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
constexpr int kCUs = 256;

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

// The larger value, NaN if either is: fmaxf would drop the NaN, and its weight
// would become a code under an ordinary scale.
__device__ __forceinline__ float larger(float a, float b) {
  return __builtin_elementwise_maximum(a, b);
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
      a = larger(a, larger(fabsf(bf16_to_f32(p[e] & 0xFFFFu)),
                           fabsf(bf16_to_f32(p[e] >> 16))));
    a = larger(a, __shfl_xor(a, 16, 64));
    amax[d] = larger(a, __shfl_xor(a, 32, 64));
  }
  if (group >= 64) {
    amax[0] = amax[1] = larger(amax[0], amax[1]);
    amax[2] = amax[3] = larger(amax[2], amax[3]);
  }
  if (group == 128)
    amax[0] = amax[1] = amax[2] = amax[3] = larger(amax[0], amax[2]);
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

// Eight codes -> eight BF16 values u / 16.  A byte u in 0..15 is the e4m3
// number u * 2^-9 (its subnormals and first binade are linear in the byte), so
// the FP8 conversion with a factor of 2^5 gives u / 16 exactly: below 1, so that
// no product with a finite x overflows.  Bytes 0..3 hold inputs 0..3 in their
// low halves and inputs 4..7 in their high ones.
constexpr float kUnit = 32.0f;

__device__ __forceinline__ v8bf codes8(uint32_t v) {
  const uint32_t lo = v & 0x0F0F0F0Fu, hi = (v >> 4) & 0x0F0F0F0Fu;
  union {
    bf2v p[4];
    v8bf v;
  } u;
  u.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, kUnit, false);
  u.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, kUnit, true);
  u.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, kUnit, false);
  u.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, kUnit, true);
  return u.v;
}

__device__ __forceinline__ v4f mfma(v4u a, v8bf b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(
      __builtin_bit_cast(v8bf, a), b, c, 0, 0, 0);
}

// The scales of a channel's groups in a block: 128 / G BF16 values.
template <int G>
struct Scales;
template <>
struct Scales<128> {
  typedef uint16_t raw;
  static __device__ __forceinline__ float get(raw r, int) {
    return bf16_to_f32(r);
  }
};
template <>
struct Scales<64> {
  typedef uint32_t raw;
  static __device__ __forceinline__ float get(raw r, int g) {
    return g ? __uint_as_float(r & 0xFFFF0000u) : __uint_as_float(r << 16);
  }
};
template <>
struct Scales<32> {
  typedef uint2 raw;
  static __device__ __forceinline__ float get(raw r, int g) {
    return Scales<64>::get(g < 2 ? r.x : r.y, g & 1);
  }
};

// A work group owns 16 T channels and up to 16 F tokens; its waves take the K
// blocks in turn and join their sums through LDS, so that a launch has waves
// enough for the weight stream where N is small, and nothing leaves the group.
// Lane (r, q) of a fragment holds token r (A) or channel r (B) at inputs
// 8 q .. 8 q + 7 of 32, and results i = 0..3 of token 4 q + i and channel r.
//
// The -8 of every code: its products with x do not depend on the channel, so
// per group they are summed once (B = -8 / 16) and are where each channel's sum
// starts.  The sum so rounds by magnitudes of |x| (|u - 8| + 16); unpacking to
// u - 8 itself, by v_cvt_off_f32_i4 or sign and magnitude, is exact at a code of
// 8 but takes twice the operations and 20% more time (1 x 5376 x 5376 6.2 us
// against 5.2, 8 x 21504 x 5376 19.8 against 16.4).  The factor 16 comes back in
// the last step.
//
// x costs more than the weights here: every group reads all of it, and a
// fragment is 16 rows of 64 bytes.  Taken as fragments from memory it held up
// the weights (8 tokens, 21504 x 5376: 19.3 us, without x 14.2); as whole rows
// of 256 bytes turned in LDS, and over T channels' tiles, 15.9 us.
struct LinearArgs {
  const uint16_t *x;
  const uint8_t *w4;
  const uint16_t *scale, *bias;
  uint16_t *y;
  int64_t M;
  int tiles, kblocks;
};

// A wave's LDS accesses run in order; this keeps the compiler from moving them
// past each other where lanes exchange values.
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// XR: loads of four rows that x takes (4 F, or fewer where the tokens are).
template <int F, int XR, int T, int WMAX, int G>
__global__ __launch_bounds__(WMAX * 64) void w4_linear_kernel(LinearArgs p) {
  constexpr int GPB = kBlockK / G;  // groups a block
  constexpr int J = 4 / GPB;        // matrix steps a group
  constexpr int kWaveLds = F * (T > 4 ? T : 4) * 64;  // 16-byte units a wave
  __shared__ v4f smem[WMAX * kWaveLds];
  __shared__ float bias_of[16 * T];
  const int W = blockDim.x >> 6;
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tile0 = blockIdx.x * T;
  const int64_t m0 = (int64_t)blockIdx.y * (16 * F);
  const int M = (int)min(p.M - m0, (int64_t)(16 * F));
  const int64_t K = (int64_t)p.kblocks * kBlockK;
  const int64_t N = (int64_t)p.tiles * kBlockN;

  // Uniform bases and 32-bit lane offsets.
  const uint8_t *wp[T];
  const uint16_t *sp[T];
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const int64_t blk = (int64_t)min(tile0 + t, p.tiles - 1) * p.kblocks;
    wp[t] = p.w4 + blk * kBlockBytes;
    sp[t] = p.scale + blk * (kBlockN * GPB);
  }
  // x of a block comes as whole rows of 256 bytes, four rows an instruction
  // (lane l: row l / 16, chunk l % 16), and turns into fragments through this
  // wave's own piece of LDS: row r keeps chunk c at c ^ r, so that the reads of
  // 16 rows meet no bank twice.  Rows past the last token read it again or are
  // zero; their results are not written.
  v4f *mine = smem + wave * kWaveLds;
  v4u *xs = reinterpret_cast<v4u *>(mine);
  uint32_t xo[XR];
#pragma unroll
  for (int i = 0; i < XR; ++i)
    xo[i] = (uint32_t)(min(4 * i + q, M - 1) * K) * 2 + 16 * r;
  struct Block {
    v4u w[T];
    typename Scales<G>::raw s[T];
    v4u x[XR];
  };
  auto load = [&](Block &k, int b) {
#pragma unroll
    for (int t = 0; t < T; ++t) {
      k.w[t] = *reinterpret_cast<const v4u *>(
          wp[t] + (int64_t)b * kBlockBytes + (uint32_t)lane * 16);
      k.s[t] = *(reinterpret_cast<const typename Scales<G>::raw *>(
                     sp[t] + (int64_t)b * (kBlockN * GPB)) +
                 (uint32_t)r);
    }
    const char *xb =
        reinterpret_cast<const char *>(p.x + m0 * K + (int64_t)b * kBlockK);
#pragma unroll
    for (int i = 0; i < XR; ++i)
      k.x[i] = *reinterpret_cast<const v4u *>(xb + xo[i]);
  };

  v8bf offset;
#pragma unroll
  for (int e = 0; e < 8; ++e) offset[e] = (__bf16)-0.5f;
  v4f acc[F][T];
#pragma unroll
  for (int f = 0; f < F; ++f)
#pragma unroll
    for (int t = 0; t < T; ++t) acc[f][t] = v4f{0, 0, 0, 0};
  auto multiply = [&](const Block &k) {
#pragma unroll
    for (int i = 0; i < XR; ++i)
      xs[(4 * i + q) * 16 + ((r ^ (4 * i + q)) & 15)] = k.x[i];
    wave_order();
#pragma unroll
    for (int g = 0; g < GPB; ++g) {
      v4u x[F][J];
      v4f start[F];
#pragma unroll
      for (int f = 0; f < F; ++f) {
#pragma unroll
        for (int j = 0; j < J; ++j)
          x[f][j] = xs[(16 * f + r) * 16 + ((4 * (g * J + j) + q) ^ r)];
        start[f] = v4f{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < J; ++j) start[f] = mfma(x[f][j], offset, start[f]);
      }
#pragma unroll
      for (int t = 0; t < T; ++t) {
        v4f s[F];
#pragma unroll
        for (int f = 0; f < F; ++f) s[f] = start[f];
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const v8bf w = codes8(k.w[t][g * J + j]);
#pragma unroll
          for (int f = 0; f < F; ++f) s[f] = mfma(x[f][j], w, s[f]);
        }
        const float sc = Scales<G>::get(k.s[t], g);
#pragma unroll
        for (int f = 0; f < F; ++f)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[f][t][i] = fmaf(s[f][i], sc, acc[f][t][i]);
      }
    }
    wave_order();
  };

  // A block's loads are issued once the block before is done, x last, and x is
  // stored to LDS first, so that a wave waits for all of them before a product
  // and only the waves beside it hide a load.  Two or three blocks on their way
  // at a time measured no faster in this order and cost the registers.
  Block blk;
  load(blk, wave);
  for (int i = threadIdx.x; i < 16 * T; i += (int)blockDim.x) {
    const int64_t c = (int64_t)tile0 * kBlockN + i;
    bias_of[i] = p.bias && c < N ? bf16_to_f32(p.bias[c]) : 0.0f;
  }
#pragma unroll
  for (int i = XR; i < 4 * F; ++i) xs[i * 64 + lane] = v4u{0, 0, 0, 0};
  for (int b = wave; b < p.kblocks; b += W) {
    multiply(blk);
    load(blk, min(b + W, p.kblocks - 1));
  }

#pragma unroll
  for (int f = 0; f < F; ++f)
#pragma unroll
    for (int t = 0; t < T; ++t) mine[(f * T + t) * 64 + lane] = acc[f][t];
  __syncthreads();
  // A thread finishes four tokens of one channel.
  for (int o = threadIdx.x; o < F * T * 64; o += (int)blockDim.x) {
    const int f = o / (64 * T), t = o / 64 % T, l = o & 63;
    v4f s = smem[o];
    for (int w = 1; w < W; ++w) s += smem[w * kWaveLds + o];
    if (tile0 + t >= p.tiles) continue;
    const int64_t c = (int64_t)(tile0 + t) * kBlockN + (l & 15);
    const float b = bias_of[16 * t + (l & 15)];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = 16 * f + 4 * (l >> 4) + i;
      if (m < M)
        p.y[(m0 + m) * N + c] =
            (uint16_t)pack_bf16x2(fmaf(s[i], 16.0f, b), 0.0f);
    }
  }
}

template <int F, int XR, int T, int WMAX>
hipError_t launch_linear(const LinearArgs &p, int group, hipStream_t stream) {
  const dim3 grid((unsigned)((p.tiles + T - 1) / T),
                  (unsigned)((p.M + 16 * F - 1) / (16 * F)));
  const int waves = p.kblocks < WMAX ? p.kblocks : WMAX;
  const dim3 block(64 * waves);
#define W8A8_W4_LAUNCH(G)                                                   \
  hipLaunchKernelGGL((w4_linear_kernel<F, XR, T, WMAX, G>), grid, block, 0,   \
                     stream, p)
  if (group == 32)
    W8A8_W4_LAUNCH(32);
  else if (group == 64)
    W8A8_W4_LAUNCH(64);
  else
    W8A8_W4_LAUNCH(128);
#undef W8A8_W4_LAUNCH
  return hipGetLastError();
}

// 16 tokens a group, XR by the tokens; T so that the groups (of `all` tiles,
// counted once for every 16 tokens) are about one a CU.
template <int XR>
hipError_t launch_16(const LinearArgs &p, int64_t all, int group,
                     hipStream_t stream) {
  if (all <= kCUs) return launch_linear<1, XR, 1, 16>(p, group, stream);
  if (all <= 2 * kCUs) return launch_linear<1, XR, 2, 16>(p, group, stream);
  if (all <= 3 * kCUs) return launch_linear<1, XR, 3, 12>(p, group, stream);
  if (all <= 4 * kCUs) return launch_linear<1, XR, 4, 8>(p, group, stream);
  if (all <= 6 * kCUs) return launch_linear<1, XR, 6, 8>(p, group, stream);
  return launch_linear<1, XR, 7, 8>(p, group, stream);
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

// Groups of about one a CU read x least often for the CUs they fill; the widest
// outputs take as many rounds as they need.  Measured at one token unless said
// (us; tiles of 16 channels), widths between not at all; T goes from 3 to 6 in
// one step for 32 tokens, where half the CUs hold a group.
//    336 tiles, K  5376: T 2, 16 waves 5.1; T 1 5.6, T 4 6.5
//   1344 tiles, K  5376: (8 tokens) T 6, 8 waves 15.9; T 3 17.4, T 4 19.2
//   1792 tiles, K  5376: T 7 17.6; T 4 17.9, T 2 18.7
// From 17 tokens on a group takes 32 of them: 64 tokens through 336 tiles,
// K 5376, 9.7 us, as four times 16 tokens 10.7; 32 tokens through 1344 tiles
// 20.0 and 24.9.  But where 16 at a time still make one group a CU of at most
// three tiles, that is faster: 32 tokens through 336 tiles 7.0 us against 8.3,
// with K 21504 26.9 against 31.
hipError_t launch_w4_linear(const uint16_t *x, const uint8_t *w4,
                            const uint16_t *scale, const uint16_t *bias,
                            uint16_t *y, int64_t M, int64_t N, int64_t K,
                            int group, hipStream_t stream) {
  const LinearArgs p{x, w4, scale, bias, y, M, (int)(N / kBlockN),
                     (int)(K / kBlockK)};
  if (M <= 4) return launch_16<1>(p, p.tiles, group, stream);
  if (M <= 8) return launch_16<2>(p, p.tiles, group, stream);
  if (M <= 16) return launch_16<4>(p, p.tiles, group, stream);
  if (M <= 32 && 2 * p.tiles <= 3 * kCUs)
    return launch_16<4>(p, 2 * p.tiles, group, stream);
  const int64_t all = p.tiles * ((M + 31) / 32);
  if (all <= kCUs) return launch_linear<2, 8, 1, 8>(p, group, stream);
  if (all <= 2 * kCUs) return launch_linear<2, 8, 2, 8>(p, group, stream);
  if (all <= 3 * kCUs) return launch_linear<2, 8, 3, 8>(p, group, stream);
  if (all <= 6 * kCUs) return launch_linear<2, 8, 6, 8>(p, group, stream);
  return launch_linear<2, 8, 8, 8>(p, group, stream);
}

}  // namespace w8a8
