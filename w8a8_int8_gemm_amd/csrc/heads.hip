// heads.hip -- rotary tables, and the norms of queries and keys for each head
// with the rotation in the same pass, for gfx950 (the formulas are in
// include/w8a8.h).
//
// Both are streams: the table writes 8 bytes a token and pair, the head norms
// read and write every value once (4 bytes), and the table's row once a token.
// Times are a call's GPU time in a captured graph whose calls take three sets of
// inputs in turn, both sides of a comparison on one card; 56 + 56 heads of 128.
#include <type_traits>

#include "heads.h"
#include "internal.h"
#include "w8a8.h"

namespace w8a8 {
namespace {

typedef unsigned v4u __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------------------
// rotary table
// ---------------------------------------------------------------------------

// sin and cos of t quarter turns, |t| <= 1/2: Taylor's series about 0 in
// x = t pi/2, |x| <= pi/4, ended where the next term is below 2^-28 of the sum
// (x^11/11! < 2^-28 x, x^12/12! < 2^-32).
struct SinCos {
  float s, c;
};

__device__ __forceinline__ SinCos quarter_sincos(float t) {
  const float x = t * 1.57079632679489662f, z = x * x;
  float s = fmaf(z, 2.75573192e-6f, -1.98412698e-4f);
  s = fmaf(z, s, 8.33333333e-3f);
  s = fmaf(z, s, -1.66666667e-1f);
  float c = fmaf(z, -2.75573192e-7f, 2.48015873e-5f);
  c = fmaf(z, c, -1.38888889e-3f);
  c = fmaf(z, c, 4.16666667e-2f);
  c = fmaf(z, c, -0.5f);
  return SinCos{fmaf(x * z, s, x), fmaf(z, c, 1.0f)};
}

constexpr int kTableThreads = 256;
constexpr int kTablePer = 4;  // tokens a thread

// Position times frequency in quarter turns, in 64 bits: at position 10^6 the
// angle of the fastest pair is off by 2^-33 of a radian, where 32 bits would
// leave 2^-4.  The nearest whole number of quarters picks the quadrant, what is
// left has its own digits in 32 bits.  A thread keeps one pair, so that its
// frequency is read once and nothing is divided for a token.
// Bound by its operations as much as by its stores: 37503 tokens of 64 pairs
// (19 MB) 7.3 us, without the stores 6.0.
template <class Pos>
__global__ __launch_bounds__(kTableThreads) void rope_table_kernel(RopeArgs a) {
  const int P = a.pairs, at_once = kTableThreads / P;
  const int first = threadIdx.x / P, p = threadIdx.x - first * P;
  if (first >= at_once) return;
  const double quarters = a.quarters[p];
  const Pos *pos = static_cast<const Pos *>(a.pos) + a.axis[p];
  int64_t t = (int64_t)blockIdx.x * (at_once * kTablePer) + first;
#pragma unroll 4
  for (int i = 0; i < kTablePer; ++i, t += at_once) {
    if (t >= a.T) return;
    const double turns = (double)pos[t * a.axes] * quarters;
    const double whole = __builtin_rint(turns);
    const SinCos sc = quarter_sincos((float)(turns - whole));
    // The quadrant, whole mod 4.  No pair turns faster than one radian a
    // position, so INT32 positions stay below 2^31 quarters; the others may lie
    // anywhere.
    const int quad = std::is_integral<Pos>::value
                         ? (int)whole & 3
                         : (int)(whole - 4.0 * __builtin_floor(whole * 0.25));
    float c = (quad & 1) ? sc.s : sc.c, s = (quad & 1) ? sc.c : sc.s;
    c = quad == 1 || quad == 2 ? -c : c;
    s = quad & 2 ? -s : s;
    float *to = a.table + 2 * t * P + p;
    to[0] = c * a.amplitude;
    to[P] = s * a.amplitude;
  }
}

// ---------------------------------------------------------------------------
// head norms with rotation
// ---------------------------------------------------------------------------

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

template <int CTRL>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(
                 0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}

// Sum over the L lanes of a head (L a power of two, heads side by side).
template <int L>
__device__ __forceinline__ float head_sum(float v) {
  if (L >= 2) v = add_dpp<0xB1>(v);    // lane ^ 1
  if (L >= 4) v = add_dpp<0x4E>(v);    // lane ^ 2
  if (L >= 8) v = add_dpp<0x141>(v);   // mirrored within 8
  if (L >= 16) v = add_dpp<0x140>(v);  // mirrored within 16
  if (L >= 32) v += __shfl_xor(v, 16);
  return v;
}

constexpr int kHeadPasses = 8;  // at most, a wave's rounds over its lanes

struct HeadShape {
  int lanes;      // of a head: 8 values each
  int passes[2];  // a wave takes passes * 64 / lanes heads of a side
  int chunks[2];  // waves a token and side
};

HeadShape head_shape(const HeadArgs &a) {
  HeadShape s;
  s.lanes = 1;
  while (s.lanes * 8 < a.D) s.lanes *= 2;
  for (int i = 0; i < 2; ++i) {
    const int64_t rounds = ((int64_t)a.side[i].heads * s.lanes + 63) / 64;
    // A wave's table row and weights serve all its rounds, so many are better,
    // as long as there are waves for every place on the chip (19077 tokens: 208
    // us with up to 8 rounds, 225 with 4, 251 with 2; 14 spill).
    int64_t most = a.M * rounds / 8192;
    most = most < 1 ? 1 : most > kHeadPasses ? kHeadPasses : most;
    const int64_t chunks = rounds ? (rounds + most - 1) / most : 0;
    s.chunks[i] = (int)chunks;
    s.passes[i] = chunks ? (int)((rounds + chunks - 1) / chunks) : 0;
  }
  return s;
}

// L lanes a head.  A wave owns one token's heads of one side: it asks for all
// of them, then for the token's table row and the weights, and turns and stores
// them one after the other.  Waves share nothing.
//
// STREAM: values go past the caches.  Where they all fit the L2s (32 MB) they stay
// for the attention behind this (the norms themselves take as long either way: 64
// tokens 3.6 us); beyond that they would only push each other out (2000 tokens 28
// us, through the caches 30; 19077 208 and 225).
//
// Told to leave room for five waves a SIMD the compiler keeps them without moving
// its loads apart (19077 tokens 208 us; untold 213, for six 256, for seven it spills:
// 354).
template <int L, bool HALF, bool STREAM>
__global__ __launch_bounds__(256, 5) void head_norm_kernel(HeadArgs a,
                                                           HeadShape shape) {
  constexpr int HEADS = 64 / L;  // a round's
  const int lane = threadIdx.x & 63;
  const int64_t wave =
      (int64_t)blockIdx.x * 4 +
      __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int per = shape.chunks[0] + shape.chunks[1];
  const int64_t m = wave / per;
  if (m >= a.M) return;
  int chunk = (int)(wave - m * per);
  const int which = chunk >= shape.chunks[0];
  if (which) chunk -= shape.chunks[0];
  const HeadSide &s = a.side[which];
  const int passes = shape.passes[which];

  const int sub = lane & (L - 1);           // chunk of 8 values in the head
  const bool live = 8 * sub < a.D;
  const int head0 = chunk * passes * HEADS + lane / L;

  // The token's row of the table; none: padding, whose outputs are zero.
  int64_t row = a.row ? (int64_t)a.row[m] : m * a.row_step;
  const bool pad = row < 0 || row >= a.rows;
  if (pad) row = 0;

  v4u raw[kHeadPasses];
#pragma unroll
  for (int u = 0; u < kHeadPasses; ++u) {
    const int h = head0 + u * HEADS;
    raw[u] = v4u{0, 0, 0, 0};
    if (u < passes && live && h < s.heads && !pad) {
      const v4u *from = reinterpret_cast<const v4u *>(
          s.x + m * s.x_stride + (int64_t)h * a.D + 8 * sub);
      raw[u] = STREAM ? __builtin_nontemporal_load(from) : *from;
    }
  }

  // Cosines and sines of this lane's values, and which of its halves turn at
  // all (the others stay as they are, whatever their partners' places hold).
  // Interleaved: 4 pairs, both values here.  Halves: value e of the first half
  // turns with the one `pairs` further; sines carry the sign.
  const int P = a.pairs;
  F8 c, d;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    c.v[e] = 1.0f;
    d.v[e] = 0.0f;
  }
  int from[2] = {lane, lane};  // HALF: the lane that holds the partners
  bool turned[2] = {false, false};
  if (P > 0 && live && !pad) {
    const float *t = a.table + row * 2 * P;
    if (HALF) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int e0 = 8 * sub + 4 * h;
        if (e0 >= 2 * P) continue;
        const bool second = e0 >= P;
        const int p0 = second ? e0 - P : e0;
        const v4f tc = *reinterpret_cast<const v4f *>(t + p0);
        const v4f td = *reinterpret_cast<const v4f *>(t + P + p0);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          c.v[4 * h + e] = tc[e];
          d.v[4 * h + e] = second ? td[e] : -td[e];
        }
        from[h] = lane - sub + (second ? p0 : e0 + P) / 8;
        turned[h] = true;
      }
    } else if (4 * sub < P) {
      const v4f tc = *reinterpret_cast<const v4f *>(t + 4 * sub);
      const v4f td = *reinterpret_cast<const v4f *>(t + P + 4 * sub);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        c.v[2 * e] = c.v[2 * e + 1] = tc[e];
        d.v[2 * e] = -td[e];
        d.v[2 * e + 1] = td[e];
      }
      turned[0] = turned[1] = true;
    }
  }
  // Partners lie in the same half of 4 values where pairs % 8 == 0, else in
  // the other one.
  const bool odd = (P & 4) != 0;
  // Two halves of 64: the partners lie 8 lanes on in the row of 16, which a lane
  // permutation reaches without a trip through LDS (19077 tokens 208 us either way:
  // the trips are covered).
  const bool across = L == 16 && P == 64;

  const float width = (float)a.D;
  F8 w, b;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    w.v[e] = 1.0f;
    b.v[e] = 0.0f;
  }
  if (live && s.w_step == 0) {
    if (s.weight)
      w = unpack8(*reinterpret_cast<const v4u *>(s.weight + 8 * sub));
    if (s.bias) b = unpack8(*reinterpret_cast<const v4u *>(s.bias + 8 * sub));
  }

#pragma unroll
  for (int u = 0; u < kHeadPasses; ++u) {
    if (u >= passes) break;
    const int h = head0 + u * HEADS;
    const bool here = live && h < s.heads;
    F8 x = unpack8(raw[u]);
    if (s.kind != W8A8_NORM_NONE) {
      float mean = 0.0f, sq = 0.0f;
      if (s.kind == W8A8_NORM_LAYER) {
#pragma unroll
        for (int e = 0; e < 8; ++e) mean += x.v[e];
        mean = head_sum<L>(mean) / width;
      }
      const float mi = live ? mean : 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x.v[e] -= mi;
        sq = fmaf(x.v[e], x.v[e], sq);
      }
      const float ms = head_sum<L>(sq) / width + s.eps;
      // A sum of squares that is not finite makes the whole head NaN.
      const float f =
          ms < __builtin_inff() ? rsqrtf(ms) : __builtin_nanf("");
      if (s.w_step != 0 && here) {
        if (s.weight)
          w = unpack8(*reinterpret_cast<const v4u *>(
              s.weight + (int64_t)h * s.w_step + 8 * sub));
        if (s.bias)
          b = unpack8(*reinterpret_cast<const v4u *>(
              s.bias + (int64_t)h * s.w_step + 8 * sub));
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) x.v[e] = fmaf(x.v[e] * f, w.v[e], b.v[e]);
    }
    F8 y;
    if (HALF) {
#pragma unroll
      for (int h2 = 0; h2 < 2; ++h2)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = 4 * h2 + e;
          const float mine = odd ? x.v[4 * (1 - h2) + e] : x.v[i];
          const float o =
              across ? __int_as_float(__builtin_amdgcn_update_dpp(
                           0, __float_as_int(mine), 0x128, 0xF, 0xF, true))
                     : __shfl(mine, from[h2]);
          y.v[i] = turned[h2] ? fmaf(x.v[i], c.v[i], o * d.v[i]) : x.v[i];
        }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        y.v[e] = turned[0] ? fmaf(x.v[e], c.v[e], x.v[e ^ 1] * d.v[e])
                           : x.v[e];
    }
    if (here) {
      // A padding token's zeros are written as such: NaN in a weight or bias
      // does not reach it.
      const v4u packed = pad ? v4u{0, 0, 0, 0} : pack8(y);
      v4u *to = reinterpret_cast<v4u *>(s.y + m * s.y_stride +
                                        (int64_t)h * a.D + 8 * sub);
      if (STREAM)
        __builtin_nontemporal_store(packed, to);
      else
        *to = packed;
    }
  }
}

constexpr int64_t kStreamBytes = int64_t(32) << 20;

template <int L>
void launch_lanes(const HeadArgs &a, const HeadShape &s, unsigned blocks,
                  hipStream_t stream) {
  const bool half = !a.interleaved && a.pairs > 0;
  const bool past =
      4 * a.M * (a.side[0].heads + a.side[1].heads) * a.D > kStreamBytes;
  if (half && past)
    head_norm_kernel<L, true, true><<<blocks, 256, 0, stream>>>(a, s);
  else if (half)
    head_norm_kernel<L, true, false><<<blocks, 256, 0, stream>>>(a, s);
  else if (past)
    head_norm_kernel<L, false, true><<<blocks, 256, 0, stream>>>(a, s);
  else
    head_norm_kernel<L, false, false><<<blocks, 256, 0, stream>>>(a, s);
}

}  // namespace

hipError_t launch_rope_table(const RopeArgs &a, hipStream_t stream) {
  const int64_t per = kTableThreads / a.pairs * kTablePer;
  const unsigned blocks = (unsigned)((a.T + per - 1) / per);
  if (a.pos_type == W8A8_POSITIONS_I32)
    rope_table_kernel<int32_t><<<blocks, kTableThreads, 0, stream>>>(a);
  else
    rope_table_kernel<float><<<blocks, kTableThreads, 0, stream>>>(a);
  return hipGetLastError();
}

int64_t head_norm_items(const HeadArgs &a) {
  const HeadShape s = head_shape(a);
  return (a.M * (s.chunks[0] + s.chunks[1]) + 3) / 4 * 256;
}

hipError_t launch_head_norm(const HeadArgs &a, hipStream_t stream) {
  const HeadShape s = head_shape(a);
  const unsigned blocks = (unsigned)(head_norm_items(a) / 256);
  switch (s.lanes) {
    case 1: launch_lanes<1>(a, s, blocks, stream); break;
    case 2: launch_lanes<2>(a, s, blocks, stream); break;
    case 4: launch_lanes<4>(a, s, blocks, stream); break;
    case 8: launch_lanes<8>(a, s, blocks, stream); break;
    case 16: launch_lanes<16>(a, s, blocks, stream); break;
    default: launch_lanes<32>(a, s, blocks, stream); break;
  }
  return hipGetLastError();
}

}  // namespace w8a8
