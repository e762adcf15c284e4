// norm.hip -- the block norms for gfx950: RMS or layer norm of a row with
// modulation, and the post-norm, gate and residual sum in front of it, to
// BF16 rows or to INT8 codes with per-token scales (the formulas are in
// include/w8a8.h).
//
// Bound by HBM: 4 bytes a value for a norm to BF16, 3 to codes, 8 and 7 with
// the residual part; a dozen binary32 operations a value.  A row is read once
// and stays in registers through all of its reductions.
//
// A work group owns R consecutive rows, so that the vectors of a modulation row
// that they share are read, unpacked and joined once.
#include "internal.h"
#include "norm.h"
#include "w8a8.h"

namespace w8a8 {
namespace {

typedef unsigned v4u __attribute__((ext_vector_type(4)));

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

// Keeps the compiler from holding a packed row's 32-bit values from one pass
// over it to the next: twice the registers, where unpacking again costs one
// operation a value.
template <int CH>
__device__ __forceinline__ void forget(v4u (&c)[CH]) {
#pragma unroll
  for (int i = 0; i < CH; ++i) asm volatile("" : "+v"(c[i]));
}

__device__ __forceinline__ v4u pack8(const F8 &f) {
  return v4u{pack_bf16x2(f.v[0], f.v[1]), pack_bf16x2(f.v[2], f.v[3]),
             pack_bf16x2(f.v[4], f.v[5]), pack_bf16x2(f.v[6], f.v[7])};
}

// The larger of m and |v|, NaN if either is (fmaxf would drop it).  Held where
// it stands: several at once would keep the values before them in registers.
__device__ __forceinline__ float max_mag(float m, float v) {
  m = __builtin_elementwise_maximum(m, fabsf(v));
  asm volatile("" : "+v"(m));
  return m;
}

// Chunk j (8 values) of a vector; where there is none, pairs of `absent`.
constexpr uint32_t kZeros = 0, kOnes = 0x3F803F80u;

__device__ __forceinline__ v4u vec8(const uint16_t *p, uint32_t j,
                                    uint32_t absent) {
  return p ? reinterpret_cast<const v4u *>(p)[j]
           : v4u{absent, absent, absent, absent};
}

// Sum, or the larger of two magnitudes.  Those order as their bits do, with
// every NaN above Inf: one NaN makes a row's maximum NaN.
template <bool MAX>
__device__ __forceinline__ float join(float a, float b) {
  return MAX ? __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)))
             : a + b;
}

template <bool MAX, int CTRL>
__device__ __forceinline__ float join_dpp(float v) {
  const int o = __builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF,
                                            0xF, true);
  return join<MAX>(v, __int_as_float(o));
}

// Sum or maximum over a row of 16 lanes: within quads, halves and the row by
// lane permutations of the adder's own operand.
template <bool MAX>
__device__ __forceinline__ float row16_reduce(float v) {
  v = join_dpp<MAX, 0xB1>(v);      // lane ^ 1
  v = join_dpp<MAX, 0x4E>(v);      // lane ^ 2
  v = join_dpp<MAX, 0x141>(v);     // mirrored within 8
  return join_dpp<MAX, 0x140>(v);  // mirrored within 16
}

template <bool MAX>
__device__ __forceinline__ float wave_reduce(float v) {
  const int b = __float_as_int(row16_reduce<MAX>(v));
  const float r0 = __int_as_float(__builtin_amdgcn_readlane(b, 0)),
              r1 = __int_as_float(__builtin_amdgcn_readlane(b, 16)),
              r2 = __int_as_float(__builtin_amdgcn_readlane(b, 32)),
              r3 = __int_as_float(__builtin_amdgcn_readlane(b, 48));
  return join<MAX>(join<MAX>(r0, r1), join<MAX>(r2, r3));
}

// Sums or maxima (of values >= 0) of R rows over the waves of a work group.
// Two slots are used in turn: a slot is written again only after every wave
// has passed the barrier of the reduction between, and so has read it.  Places
// of waves that the group does not have hold zero.
constexpr int kMaxWaves = 16;

template <int R>
struct Reducer {
  float (*part)[R][kMaxWaves];
  int slot;

  __device__ __forceinline__ void clear() {
    float *p = &part[0][0][0];
    for (int i = threadIdx.x; i < 2 * R * kMaxWaves; i += blockDim.x)
      p[i] = 0.0f;
    __syncthreads();
  }

  template <bool MAX>
  __device__ __forceinline__ void reduce(float (&v)[R]) {
#pragma unroll
    for (int r = 0; r < R; ++r) v[r] = wave_reduce<MAX>(v[r]);
    if (blockDim.x == 64) return;
    float(*p)[kMaxWaves] = part[slot];
    slot ^= 1;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int r = 0; r < R; ++r) p[r][threadIdx.x >> 6] = v[r];
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r)
      v[r] = row16_reduce<MAX>(p[r][threadIdx.x & 15]);
  }
};

// A row's statistics: it is normalized by (v - mean) * f, f =
// 1 / sqrt(mean square + eps), the mean 0 but for a layer norm.  The mean
// first, then the squares of the differences, so that a large mean costs the
// variance no digits.  Where the sum of squares is not finite (Inf or NaN in
// the row, or squares beyond the range) f is NaN, and with it the whole row: 0
// would take the row's values out of the result without a trace.
struct Stats {
  float f, mean;
};

// `Row` gives chunk i of row r (CH chunks a thread, thread t of `step`; places
// past the row's end are zero) as 8 values, `squares` adds those of chunk i,
// `again` stands between two passes.
template <int R, int CH, class Row, class Squares, class Again>
__device__ __forceinline__ void row_stats(Stats (&st)[R], int kind, float eps,
                                          int t, int step, int chunks,
                                          float width, Reducer<R> &red,
                                          Row row, Squares squares,
                                          Again again) {
  float sq[R], mean[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    st[r] = Stats{1.0f, 0.0f};
    sq[r] = mean[r] = 0.0f;
  }
  if (kind == W8A8_NORM_NONE) return;
  if (kind == W8A8_NORM_LAYER) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const F8 v = row(r, i);
#pragma unroll
        for (int e = 0; e < 8; ++e) mean[r] += v.v[e];
      }
    red.template reduce<false>(mean);
    again();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] /= width;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const F8 v = row(r, i);
        const float mi = i * step + t < chunks ? mean[r] : 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float d = v.v[e] - mi;
          sq[r] = fmaf(d, d, sq[r]);
        }
      }
    }
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < CH; ++i) sq[r] = squares(r, i, sq[r]);
  }
  red.template reduce<false>(sq);
  again();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float ms = sq[r] / width + eps;
    st[r].f = ms < __builtin_inff() ? rsqrtf(ms) : __builtin_nanf("");
    st[r].mean = mean[r];
  }
}

// sq plus the squares of 8 packed values: products exact, two to an addition.
__device__ __forceinline__ float squares8(v4u c, float sq) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const bf2v p = __builtin_bit_cast(bf2v, w[e]);
    sq = __builtin_amdgcn_fdot2_f32_bf16(p, p, sq, false);
  }
  return sq;
}

__device__ __forceinline__ float squares8(const F8 &v, float sq) {
#pragma unroll
  for (int e = 0; e < 8; ++e) sq = fmaf(v.v[e], v.v[e], sq);
  return sq;
}

// The map n -> n * a + b of a normalized value, for 8 channels.
struct Affine {
  F8 a, b;
};

// What a map is made of, for a chunk: the vectors of modulation row mr and the
// norm's weight.  The bias, which few norms have, is read where it is used.
struct PostVecs {
  v4u gate, weight;
};

__device__ __forceinline__ PostVecs post_vecs(const NormArgs &a, int64_t mr,
                                              uint32_t j) {
  return PostVecs{
      vec8(a.gate ? a.gate + mr * a.gate_stride : nullptr, j, kOnes),
      vec8(a.post_weight, j, kOnes)};
}

// gate behind the post-norm's weight and bias.
__device__ __forceinline__ Affine post_map(const NormArgs &a,
                                           const PostVecs &p, uint32_t j) {
  const F8 g = unpack8(p.gate), w = unpack8(p.weight);
  Affine f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    f.a.v[e] = g.v[e] * w.v[e];
    f.b.v[e] = 0.0f;
  }
  if (a.post_bias) {
    const F8 b = unpack8(vec8(a.post_bias, j, kZeros));
#pragma unroll
    for (int e = 0; e < 8; ++e) f.b.v[e] = g.v[e] * b.v[e];
  }
  return f;
}

struct PreVecs {
  v4u scale, shift, weight;
};

__device__ __forceinline__ PreVecs pre_vecs(const NormArgs &a, int64_t mr,
                                            uint32_t j) {
  return PreVecs{
      vec8(a.scale ? a.scale + mr * a.scale_stride : nullptr, j, kZeros),
      vec8(a.shift ? a.shift + mr * a.shift_stride : nullptr, j, kZeros),
      vec8(a.weight, j, kOnes)};
}

// 1 + scale and shift behind the norm's weight and bias.
__device__ __forceinline__ Affine pre_map(const NormArgs &a, const PreVecs &p,
                                          uint32_t j) {
  const F8 s = unpack8(p.scale), w = unpack8(p.weight);
  Affine f;
  f.b = unpack8(p.shift);
#pragma unroll
  for (int e = 0; e < 8; ++e)
    f.a.v[e] = fmaf(w.v[e], s.v[e], w.v[e]);  // w (1 + s), rounded once
  if (a.bias) {
    const F8 b = unpack8(vec8(a.bias, j, kZeros));
#pragma unroll
    for (int e = 0; e < 8; ++e)
      f.b.v[e] += fmaf(b.v[e], s.v[e], b.v[e]);
  }
  return f;
}

// Scale and reciprocal of a row whose largest magnitude is amax.  The codes
// are the integers nearest to y * (1 / s), rounded once: those of y / s but
// where that lies within 2^-16 of a half, since the reciprocal is off by a
// little over 2^-24 of at most 127 (y itself is known no better).
struct CodeRow {
  float s, r;
};

// At a scale below 2^-100 the reciprocal could overflow: row and scale are
// then taken 2^64 times larger.
constexpr float kSmallScale = 0x1p-100f, kLift = 0x1p64f;

// A NaN in the row is in amax, and so in its scale; the codes mean nothing then.
__device__ __forceinline__ CodeRow code_row(float amax) {
  const float s = amax / 127.0f;
  const float d = s < kSmallScale ? s * kLift : s;
  float r = __builtin_amdgcn_rcpf(d);
  r = fmaf(fmaf(-d, r, 1.0f), r, r);  // Newton's step: to within half a step
  // the same in every lane: keep it in scalar registers
  return CodeRow{
      __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(s))),
      __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(r)))};
}

// Codes of 8 values.  At 1.5 * 2^23 a binary32 step is 1, so one fused
// multiply-add rounds y * r to the nearest integer, ties to even, and leaves
// its two's complement in the low byte.  A subnormal scale is so coarse that
// y / s may pass 127 and is clamped.
template <bool SMALL>
__device__ __forceinline__ uint2 codes8(const F8 &y, float r) {
  uint32_t c[8], o[2];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float v =
        SMALL ? fminf(fmaxf(y.v[e] * kLift * r, -127.0f), 127.0f) : y.v[e];
    c[e] = __float_as_uint(fmaf(v, SMALL ? 1.0f : r, 0x1.8p23f));
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __builtin_amdgcn_perm(c[4 * h + 1], c[4 * h],
                                              0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(c[4 * h + 3], c[4 * h + 2],
                                              0x04000C0Cu);
    o[h] = lo | hi;
  }
  return make_uint2(o[0], o[1]);
}

__device__ __forceinline__ uint2 codes8(const F8 &y, const CodeRow &c) {
  if (c.s >= kSmallScale) return codes8<false>(y, c.r);
  if (c.s == 0.0f) return make_uint2(0, 0);
  return codes8<true>(y, c.r);
}

// The R rows from blockIdx.x * R on; a thread holds chunks t, t + step, ... of
// each.  Registers set the pace once memory does not: a form that walks a long
// run of rows with the vectors kept and the next rows loaded ahead holds more
// of them and ran 14 to 50% slower; one wave a row without barriers spilled.
template <int R, int CH, bool RES, int OUT>
__global__ __launch_bounds__(64 * kMaxWaves) void norm_kernel(NormArgs a) {
  __shared__ float part[2][R][kMaxWaves];
  Reducer<R> red{part, 0};
  const int t = threadIdx.x, step = blockDim.x;
  const int chunks = a.H >> 3;
  const float width = (float)a.H;
  const int64_t m0 = (int64_t)blockIdx.x * R;
  // chunk j of row m0 + r
  auto chunk = [&](const void *p, int r, uint32_t j) {
    return reinterpret_cast<const v4u *>(p) + (m0 + r) * (int64_t)chunks + j;
  };

  // Many rows pass by once and would push the vectors, and what the next
  // kernel reads, out of the caches (norm to BF16 of 19077 x 5376 85 us, 79
  // with nontemporal loads; both with codes 143 us, 131 with r stored so too);
  // a few were written just before and are read soon.
  auto fetch = [](const v4u *p) {
    return R > 1 ? __builtin_nontemporal_load(p) : *p;
  };
  // Rows past the last one read it again and write nothing.
  v4u x[R][CH], b[R][CH];
  int64_t mr[R];
  bool live[R], same = true;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int rr = (int)min((int64_t)r, a.M - 1 - m0);
    mr[r] = a.row ? (int64_t)a.row[m0 + rr] : (m0 + rr) * a.row_step;
    live[r] = mr[r] >= 0 && mr[r] < a.rows;
    same = same && live[r] && mr[r] == mr[0];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int j = i * step + t;
      x[r][i] = j < chunks ? fetch(chunk(a.x, rr, j)) : v4u{0, 0, 0, 0};
      if (RES)
        b[r][i] = j < chunks ? fetch(chunk(a.branch, rr, j)) : v4u{0, 0, 0, 0};
    }
  }
  red.clear();
  auto forget = [&](v4u (&c)[R][CH]) {
#pragma unroll
    for (int r = 0; r < R; ++r) w8a8::forget<CH>(c[r]);
  };
  auto in_range = [&](int r) { return R == 1 || m0 + r < a.M; };

  // The vectors of the maps are asked for ahead of a reduction, not behind it
  // (norm to codes of 37503 x 5376: behind it 150 us, so 128).  Each stands
  // under a test of its pointer, so that the reduction's wait for the row is a
  // wait for them as well.
  F8 v[R][CH];  // the residual rows, or the output on its way to codes
  Stats st[R];
  PreVecs pv[CH];
  auto load_pre = [&]() {
#pragma unroll
    for (int i = 0; i < CH; ++i)
      if (same && i * step + t < chunks)
        pv[i] = pre_vecs(a, mr[0], i * step + t);
  };
  if (RES) {
    PostVecs gv[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i)
      if (same && i * step + t < chunks)
        gv[i] = post_vecs(a, mr[0], i * step + t);
    row_stats<R, CH>(
        st, a.post_kind, a.post_eps, t, step, chunks, width, red,
        [&](int r, int i) { return unpack8(b[r][i]); },
        [&](int r, int i, float sq) { return squares8(b[r][i], sq); },
        [&]() { forget(b); });
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int j = i * step + t;
#pragma unroll
      for (int r = 0; r < R; ++r) v[r][i] = unpack8(v4u{0, 0, 0, 0});
      if (j >= chunks) continue;
      Affine g;
      if (same) g = post_map(a, gv[i], j);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        v4u o = x[r][i];
        if (live[r]) {
          if (!same) g = post_map(a, post_vecs(a, mr[r], j), j);
          const F8 xi = unpack8(x[r][i]), bi = unpack8(b[r][i]);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            v[r][i].v[e] = fmaf((bi.v[e] - st[r].mean) * st[r].f, g.a.v[e],
                                fmaf(a.residual_scale, xi.v[e], g.b.v[e]));
          o = pack8(v[r][i]);
        }
        v4u *to = const_cast<v4u *>(chunk(a.r, r, j));
        if (R > 1 && in_range(r))
          __builtin_nontemporal_store(o, to);
        else if (in_range(r))
          *to = o;
      }
    }
  }
  if (OUT == OUT_NONE) return;
  load_pre();
  row_stats<R, CH>(
      st, a.kind, a.eps, t, step, chunks, width, red,
      [&](int r, int i) { return RES ? v[r][i] : unpack8(x[r][i]); },
      [&](int r, int i, float sq) {
        return RES ? squares8(v[r][i], sq) : squares8(x[r][i], sq);
      },
      [&]() {
        if (!RES) forget(x);
      });
  float amax[R];
#pragma unroll
  for (int r = 0; r < R; ++r) amax[r] = 0.0f;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int j = i * step + t;
    if (j >= chunks) continue;
    Affine g;
    if (same) g = pre_map(a, pv[i], j);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      F8 y = unpack8(v4u{0, 0, 0, 0});
      if (live[r]) {
        if (!same) g = pre_map(a, pre_vecs(a, mr[r], j), j);
        if (!RES) v[r][i] = unpack8(x[r][i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          y.v[e] = fmaf((v[r][i].v[e] - st[r].mean) * st[r].f, g.a.v[e],
                        g.b.v[e]);
          if (OUT == OUT_CODES) amax[r] = max_mag(amax[r], y.v[e]);
        }
      }
      if (OUT == OUT_CODES) v[r][i] = y;
      if (OUT == OUT_ROW && in_range(r))
        *const_cast<v4u *>(chunk(a.y, r, j)) = pack8(y);
    }
  }
  if (OUT != OUT_CODES) return;
  red.template reduce<true>(amax);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (!in_range(r)) continue;
    const CodeRow Q = code_row(amax[r]);
    if (t == 0) a.qs[m0 + r] = Q.s;
    uint2 *q = reinterpret_cast<uint2 *>(a.q) + (m0 + r) * (int64_t)chunks;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const uint32_t j = i * step + t;
      if (j < (uint32_t)chunks) q[j] = codes8(v[r][i], Q);
    }
  }
}

template <int R, int CH>
void launch_rows(const NormArgs &a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.M + R - 1) / R));
  const dim3 block(64 * ((a.H / 8 + 64 * CH - 1) / (64 * CH)));
#define W8A8_NORM_LAUNCH(RES, OUT)                                            \
  hipLaunchKernelGGL((norm_kernel<R, CH, RES, OUT>), grid, block, 0, stream, a)
  if (a.branch) {
    if (a.q)
      W8A8_NORM_LAUNCH(true, OUT_CODES);
    else if (a.y)
      W8A8_NORM_LAUNCH(true, OUT_ROW);
    else
      W8A8_NORM_LAUNCH(true, OUT_NONE);
  } else if (a.q) {
    W8A8_NORM_LAUNCH(false, OUT_CODES);
  } else {
    W8A8_NORM_LAUNCH(false, OUT_ROW);
  }
#undef W8A8_NORM_LAUNCH
}

}  // namespace

// R rows a work group, CH chunks a thread, by the values of the call (M * H):
//  * below 2M values a launch is latency: one chunk a thread (5376 wide, norm
//    to BF16 and both norms to codes: 64 rows 2.6 and 4.9 us, with three
//    chunks 3.1 and 5.7; 256 rows 3.7 and 6.2 against 4.1 and 7.1);
//  * below 6M two chunks, so that a wave's own instructions (addresses,
//    reductions) weigh less (1024 rows 7.0 and 12.4 us; one chunk 7.6 and
//    15.1, three and two rows 7.4 and 12.5);
//  * above, three chunks and two rows that share their vectors (8192 rows 35.0
//    and 66.6 us; one row 36.5 and 75.7, one chunk 45.9 and 100);
//  * modulation rows that are each read once have nothing to share: one row
//    (16384 rows, layer norm to codes 120 us, two rows 133).
// Waves are as few as that allows, and then the chunks as few as those waves
// need.  Rows wider than 24576 take four chunks and one row.
hipError_t launch_norm(const NormArgs &a, hipStream_t stream) {
  const int chunks = a.H / 8;
  const int64_t values = a.M * a.H;
  const bool many = values >= 6000000;
  const bool share = !(a.row == nullptr && a.row_step == 1);
  const int want = values < 2000000 ? 1 : many ? 3 : 2;
  int waves = (chunks + 64 * want - 1) / (64 * want);
  if (waves > kMaxWaves) waves = kMaxWaves;
  const int ch = (chunks + 64 * waves - 1) / (64 * waves);
  const bool two = many && share;
  if (ch == 1 && two) launch_rows<2, 1>(a, stream);
  else if (ch == 1) launch_rows<1, 1>(a, stream);
  else if (ch == 2 && two) launch_rows<2, 2>(a, stream);
  else if (ch == 2) launch_rows<1, 2>(a, stream);
  else if (ch == 3 && two) launch_rows<2, 3>(a, stream);
  else if (ch == 3) launch_rows<1, 3>(a, stream);
  else if (ch == 4) launch_rows<1, 4>(a, stream);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

}  // namespace w8a8
