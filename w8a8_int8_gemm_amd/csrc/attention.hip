// attention.hip -- attention of queries to keys and values of another length
// for gfx950 (the formulas are in include/w8a8.h).
//
// out = softmax(scale q k^T) v per head, in one pass over the keys with each
// row's running maximum m and sum l.  Both products run on
// v_mfma_f32_32x32x16_bf16 with their roles turned round: S^T = K Q^T puts one
// query's scores into one lane (and the lane 32 further), so that maximum, exp
// and sum need no exchange between lanes, and the lane's scores, rounded to
// BF16 in the order in which they lie, are the operand of O^T = V^T P^T.  That
// product sums over keys in any order, so V's fragments are read (transposed,
// from LDS) in the same order.
//
// Weights p = 2^(c s - c m) (c: scale log2 e) are rounded to BF16 for the matrix
// unit; l sums the rounded ones, so that each row's weights still sum to one.  m
// lags: it moves (and O and l with it) only where a row's scores pass it by more
// than 2^8, so p stays near 2^8 at most and the sums far inside binary32.
// c m is rounded, which costs a row's weights a common factor of up to
// 2^(2^-24 |c m|); from |c m| = 2^31 on that would leave binary32.  So where |c m| is
// large (kFar) the difference s - m is taken first.
//
// Times here and below are a call's GPU time in a captured graph whose calls take
// three sets of inputs in turn, both sides of a comparison on one card.
// Bound by power where there are many rows: 19077 tokens to themselves, 56 heads
// of 128, 9.2 ms (1.13 PFLOP/s; 9.1 to 9.7 on other cards; the library's BF16
// product of 8192^3 1.16, of 16384^3 1.40; inputs of zeros 1.5).  By memory where few
// rows read many keys: 64 queries to 37503 keys 220 us, 5.0 TB/s while it reads.
// Small calls by their chain of trips: one query to 512 keys 10.7 us.
#include "heads.h"
#include "internal.h"
#include "w8a8.h"

namespace w8a8 {
namespace {

typedef unsigned v4u __attribute__((ext_vector_type(4)));
typedef unsigned v2u __attribute__((ext_vector_type(2)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) v4s lds_v4s;

constexpr int kXcds = 8;
constexpr float kInf = __builtin_inff();
// How far scores may pass m, in powers of two: weights keep their relative
// precision at any size, so it only has to stay far from the range's end.
constexpr float kLag = 8.0f;
// |c m| from which on weights are taken of s - m, in the branch that moves m, which
// a wave with such a row then takes at every stage.  Below it c m is off by 2^-15 at
// most, so weights of before and behind a move of m, or of waves and parts that
// are joined, agree to 2^-15.
constexpr float kFar = 1024.0f;

// A tile of TM query rows and the keys of a stage.  WQ waves along the rows (32
// each) times WK along the keys of a stage, whose results are joined at the
// end.  DP: head width, rounded up to 32.
template <int WQ_, int WK_, int KT_, int DP_>
struct Cfg {
  static constexpr int WQ = WQ_, WK = WK_, KT = KT_, DP = DP_;
  static constexpr int WAVES = WQ * WK, THREADS = 64 * WAVES, TM = 32 * WQ;
  static constexpr int DL = DP > 64 ? 128 : DP;  // values of a row in LDS
  static constexpr int RB = 2 * DL;              // its bytes
  static constexpr int CPR = RB / 16;            // its 16-byte chunks
  static constexpr int KW = KT / WK;             // a wave's keys of a stage
  static constexpr int NS = KW / 32;             // its score tiles
  static constexpr int KS = DP / 16;             // steps of q k^T
  static constexpr int NO = DP / 32;             // output tiles
  static constexpr int SIDE = KT * RB;           // bytes of a stage's K (or V)
  static constexpr int STAGE = 2 * SIDE;
  // 16-byte loads of K a thread and stage
  static constexpr int LOADS = (SIDE / 16 + THREADS - 1) / THREADS;
  static constexpr int OROW = DP + 4;            // floats of a joined row
  static constexpr int JOIN =
      WK > 1 ? WK * TM * OROW * 4 + 2 * WK * TM * 4 : TM * OROW * 2;
  // Q comes in whole rows, behind the first stage, where it needs little more
  // than the second one's place.
  static constexpr int QSIZE = TM * RB;
  static constexpr bool THROUGH = TM <= 128;
  static constexpr int BUFS =
      THROUGH && QSIZE > STAGE ? STAGE + QSIZE : 2 * STAGE;
  static constexpr int LDS = BUFS > JOIN ? BUFS : JOIN;
  // Work groups a compute unit has registers for, and how many fragments of K
  // are read ahead of their products (4, 6 or 8: 965, 968, 972 us at 8192 tokens, 32
  // heads of 128; 3 keep three work groups' registers).
  static constexpr int GROUPS = WAVES == 8 ? 1 : KT == 32 ? 3 : 2;
  static constexpr int AHEAD = KS * NS < 4 ? 2 : GROUPS == 3 ? 3 : 4;
  static constexpr int WAVES_PER_SIMD = GROUPS * WAVES / 4;
  static_assert(LDS <= 160 * 1024, "");
};

// Where chunk c of row r lies in its row.  LDS gives 256 bytes a cycle if their
// places differ by 256: to 16 lanes a chunk of consecutive rows each (K), to 32
// lanes half a chunk each, 4 chunks side by side of 4 rows (V).
template <int CPR>
__device__ __forceinline__ int swz_k(int r, int c) {
  return c ^ ((r / (16 / CPR)) & (CPR - 1));
}

template <int CPR>
__device__ __forceinline__ int swz_v(int r, int c) {
  return c ^ ((r & 3) / (16 / CPR) * 4);
}

__device__ __forceinline__ int xcd_remap(int bid, int T) {
  const int xcd = bid % kXcds;
  const int local = bid / kXcds;
  const int per = T / kXcds, rem = T % kXcds;
  return xcd * per + min(xcd, rem) + local;
}

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// This wave's reads of LDS are done.  The builtin, which the compiler's own
// counting of waits sees (vmcnt and expcnt stay unlimited: bits [15:14] and [3:0],
// [6:4]; lgkmcnt 0: [11:8]).
__device__ __forceinline__ void wait_lgkm() {
  __builtin_amdgcn_s_waitcnt(0xC07F);
}

// Barrier without the fences of __syncthreads, which would wait for direct
// loads on their way; the waits are written out where they are due.
__device__ __forceinline__ void block_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Uniform 64-bit address -> raw buffer resource of `bytes` bytes: reads past
// them give zeros, in LDS too.
__device__ __forceinline__ v4u rsrc(uint64_t at, uint32_t bytes) {
  return v4u{(uint32_t)at, (uint32_t)(at >> 32) & 0xFFFFu, bytes, 0x00020000u};
}

__device__ __forceinline__ uint64_t uniform64(uint64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(v >> 32));
  return (uint64_t)hi << 32 | lo;
}

// 16 bytes per lane from buffer `r` at byte voff into LDS at `l` (lane i's bytes
// at l + 16 i).  Written out because the compiler, which knows only that the
// builtin writes LDS, waits for every such load before the next transposing
// read; the waits here are the kernel's own.
__device__ __forceinline__ void load_lds16(v4u r, int voff, uint32_t l) {
  asm volatile(
      "s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
      :
      : "s"(l), "v"(voff), "s"(r)
      : "memory", "m0");
}

// A uniform place in LDS, as a number.  Worked out on the spot: the places of all
// loads of a loop, held over it, would take the scalar registers that the
// scheduler needs.
__device__ __forceinline__ uint32_t lds_at(const char *l) {
  uint32_t v = __builtin_amdgcn_readfirstlane(
      (int)(uint32_t)(uintptr_t)(lds_void *)l);
  asm volatile("" : "+s"(v));
  return v;
}

// Of a block of 4 rows x 16 values (a lane's 8 bytes at `l`: 4 values of row
// lane % 16 / 4), the lane's column: one value of each row.
__device__ __forceinline__ v4s read_turned(const char *l) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)l);
}

__device__ __forceinline__ v16f mfma(v8bf a, v8bf b, v16f c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// A tile's sequence: query rows (times the G heads that share keys) from row0
// on, keys from key0 on.
struct Tile {
  int q0, nq, key0, keys;
  int row0;  // of the nq * G rows
};

__device__ __forceinline__ int clamped(int v, int lo, int hi) {
  return min(max(v, lo), hi);
}

__device__ __forceinline__ Tile tile_of(const AttnArgs &a, int b, int q0,
                                        int nq, int row0) {
  int key0 = 0, keys = a.Tk;
  if (a.k_offsets) {
    key0 = clamped(a.k_offsets[b], 0, a.Tk);
    keys = clamped(a.k_offsets[b + 1], key0, a.Tk) - key0;
  } else if (a.B > 1) {
    keys = (uint32_t)a.Tk / (uint32_t)a.B;
    key0 = b * keys;
  }
  if (a.k_lens) keys = clamped(a.k_lens[b], 0, keys);
  return Tile{q0, nq, key0, keys, row0};
}

// Tile `i` of all sequences, TM rows each; nq 0 where there is none.  Offsets are
// clamped to the rows there are, so no content of theirs leads outside.
// Packed sequence b has the tiles from S(b) = floor(rows before it / TM) + b on:
// up to S(b + 1) there are as many as it needs at least, and all of them below
// rows / TM + B, without a sum over the sequences.  S rises with b, so 64 lanes
// find a tile's sequence in as many steps as B has digits of 64.
template <int TM>
__device__ __forceinline__ Tile find_tile(const AttnArgs &a, uint32_t i) {
  const uint32_t G = a.G;
  if (!a.q_offsets) {
    uint32_t b = 0, nq = a.Tq;
    if (a.B > 1) {
      nq = (uint32_t)a.Tq / (uint32_t)a.B;
      const uint32_t per = (nq * G + TM - 1) / TM;
      b = i / per;
      i -= b * per;
    }
    return tile_of(a, b, b * nq, nq, i * TM);
  }
  auto first_tile = [&](int b) {
    return (uint32_t)clamped(a.q_offsets[b], 0, a.Tq) * G / TM + (uint32_t)b;
  };
  const int lane = threadIdx.x & 63;
  int lo = 0, len = a.B;
  for (;;) {
    const int step = (len + 63) / 64, b = lo + lane * step;
    const uint64_t at_or_before =
        __ballot(lane * step < len && first_tile(b) <= i);
    const int n = __builtin_popcountll(at_or_before);
    if (n == 0) return Tile{0, 0, 0, 0, 0};
    lo += (n - 1) * step;
    if (step == 1) break;
    len = min(step, len - (n - 1) * step);
  }
  lo = __builtin_amdgcn_readfirstlane(lo);
  const int q0 = clamped(a.q_offsets[lo], 0, a.Tq);
  const int nq = clamped(a.q_offsets[lo + 1], q0, a.Tq) - q0;
  const uint32_t row0 = (i - first_tile(lo)) * TM;
  if (row0 >= nq * G) return Tile{0, 0, 0, 0, 0};
  return tile_of(a, lo, q0, nq, row0);
}

// Row r of a tile (r below 2^9): its token and its head among the G that share
// keys.  x = row0 mod G + r is below 2^20 (G is, by the strides' limit), and (x +
// 1/2) / G lies 1 / (2 G) or more off every whole number, further than two
// binary32 roundings of it.
struct RowMap {
  int tok0, rem, G;
  float inv;

  __device__ __forceinline__ RowMap(const Tile &t, int G_) : G(G_) {
    tok0 = t.q0 + (G == 1 ? t.row0 : t.row0 / G);
    rem = G == 1 ? 0 : t.row0 % G;
    inv = 1.0f / (float)G;
  }
  __device__ __forceinline__ int past(int r) const {  // tokens past tok0
    return (int)(((float)(rem + r) + 0.5f) * inv);
  }
  __device__ __forceinline__ int head(int r, int past) const {
    return rem + r - past * G;
  }
};

// The larger / the sum of a lane's value and that of the lane 32 further.
__device__ __forceinline__ float max_halves(float v) {
  const v2u r = __builtin_amdgcn_permlane32_swap(
      __float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r.x), __uint_as_float(r.y));
}

__device__ __forceinline__ float add_halves(float v) {
  const v2u r = __builtin_amdgcn_permlane32_swap(
      __float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r.x) + __uint_as_float(r.y);
}

__device__ __forceinline__ float sum2(uint32_t p, float l) {
  const bf2v one = __builtin_bit_cast(bf2v, 0x3F803F80u);
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf2v, p), one, l,
                                         false);
}

// Partial results of a split: per part and query row O (D values), then per
// part and row m and l.
__device__ __forceinline__ float *part_o(const AttnArgs &a, int split) {
  return static_cast<float *>(a.workspace) +
         (int64_t)split * a.Tq * a.Hq * a.D;
}

__device__ __forceinline__ float2 *part_ml(const AttnArgs &a, int splits,
                                           int split) {
  return reinterpret_cast<float2 *>(static_cast<float *>(a.workspace) +
                                    (int64_t)splits * a.Tq * a.Hq * a.D) +
         (int64_t)split * a.Tq * a.Hq;
}

// What a wave holds of its 32 query rows (a lane's row: lane % 32, the lane 32
// further the same), and a stage's work on them.
template <class C>
struct Rows {
  v8bf fq[C::KS];    // Q^T as the right operand: 8 values a step
  int ak[C::KS / 2]; // places of the fragments of K and of V^T in a stage
  int av[C::NO];
  v16f o[C::NO];
  // m (0 until a score sets it), the score that moves it, and l.
  float m, limit, l;
  bool far;  // any of the wave's rows is

  // `wk`: which of the stage's keys are this wave's.
  __device__ __forceinline__ void places(int lane, int wk) {
    const int half = lane >> 5;
    // Key (lane & 31) of a score tile.  The swizzle is an exclusive or, so an
    // odd step's place is one bit off the even one's.
    const int r = lane & 31;
#pragma unroll
    for (int s = 0; s < C::KS / 2; ++s)
      ak[s] = (wk * C::KW + r) * C::RB + swz_k<C::CPR>(r, 4 * s + half) * 16;
    // Of 16 keys a lane needs those that its scores stand for (4 half .. + 3 and
    // 8 further), of value (lane & 31) of an output tile; a transposing read
    // gives 16 lanes 4 keys of 16 values.
    const int i = lane & 15, rv = 4 * half + i / 4;
#pragma unroll
    for (int n = 0; n < C::NO; ++n) {
      const int c = 4 * n + 2 * ((lane >> 4) & 1) + (i & 3) / 2;
      av[n] = C::SIDE + (wk * C::KW + rv) * C::RB + swz_v<C::CPR>(rv, c) * 16 +
              (i & 1) * 8;
    }
  }

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int n = 0; n < C::NO; ++n)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[n][e] = 0.0f;
    m = l = 0.0f;
    limit = -kInf;
    far = false;
  }

  // A stage at `base`; `left` keys of it, from this wave's first on, count.
  __device__ __forceinline__ void step(const char *base, int left, float c,
                                       int half) {
    // Ahead of the other wave's powers on the same SIMD: 0.3% (8192 tokens, 32 heads
    // of 128 965 us beside 967-968).
    __builtin_amdgcn_s_setprio(1);
    v16f s[C::NS];
#pragma unroll
    for (int n = 0; n < C::NS; ++n)
#pragma unroll
      for (int e = 0; e < 16; ++e) s[n][e] = 0.0f;
#pragma unroll
    for (int k = 0; k < C::KS; ++k)
#pragma unroll
      for (int n = 0; n < C::NS; ++n)
        s[n] = mfma(*reinterpret_cast<const v8bf *>(
                        base + (ak[k / 2] ^ (k & 1) * 32) + n * 32 * C::RB),
                    fq[k], s[n]);
    // Fragments are read a few matrix instructions ahead.
    __builtin_amdgcn_sched_group_barrier(0x100, C::AHEAD, 0);
#pragma unroll
    for (int i = 0; i < C::KS * C::NS - C::AHEAD; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, C::AHEAD, 0);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(0);
    // Keys past the end (their rows of LDS are zeros, whatever memory holds).
    if (left < C::KW) {
#pragma unroll
      for (int n = 0; n < C::NS; ++n)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (32 * n + 8 * (e / 4) + 4 * half + e % 4 >= left) s[n][e] = -kInf;
    }
    float top = s[0][0];
#pragma unroll
    for (int n = 0; n < C::NS; ++n)
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, s[n][e]);
    if (far || __any(top > limit)) {
      const float now = max_halves(top);
      const bool unset = limit == -kInf;
      const float nm = unset ? (now == -kInf ? 0.0f : now) : fmaxf(m, now);
      const float f = unset ? 0.0f : __builtin_amdgcn_exp2f((m - nm) * c);
      m = nm;
      limit = unset && now == -kInf ? -kInf : nm + kLag / c;
      far = __any(fabsf(m * c) > kFar);
      l *= f;
#pragma unroll
      for (int n = 0; n < C::NO; ++n)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[n][e] *= f;
      const float sub = far ? m : 0.0f;
#pragma unroll
      for (int n = 0; n < C::NS; ++n)
#pragma unroll
        for (int e = 0; e < 16; ++e) s[n][e] -= sub;
    }
    const float cm = m * (far ? 0.0f : c);
    v4u p[C::NS][2];
#pragma unroll
    for (int n = 0; n < C::NS; ++n)
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        const uint32_t two =
            pack_bf16x2(__builtin_amdgcn_exp2f(fmaf(s[n][e], c, -cm)),
                        __builtin_amdgcn_exp2f(fmaf(s[n][e + 1], c, -cm)));
        l = sum2(two, l);
        p[n][e / 8][(e % 8) / 2] = two;
      }
#pragma unroll
    for (int n = 0; n < C::NS; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int d = 0; d < C::NO; ++d) {
          union {
            v4s h[2];
            v8bf f;
          } fv;
#pragma unroll
          for (int x = 0; x < 2; ++x)
            fv.h[x] =
                read_turned(base + av[d] + (32 * n + 16 * j + 8 * x) * C::RB);
          o[d] = mfma(fv.f, __builtin_bit_cast(v8bf, p[n][j]), o[d]);
        }
  }
};

constexpr int kNowhere = 0x7FFFFFF0;  // past every buffer: reads zeros

// The stages of a tile's keys and values, asked for one after the other.
template <class C>
struct Stages {
  int ok[C::LOADS], ov[C::LOADS];  // what lands in this thread's 16 bytes
  int ks2, vs2, D2, wave;
  uint64_t kat, vat;               // the next stage's first row,
  int left;                        // and the keys from it on

  __device__ __forceinline__ void places(const AttnArgs &a, int wave_,
                                         int lane) {
    wave = wave_;
    ks2 = (int)(a.k_stride * 2);
    vs2 = (int)(a.v_stride * 2);
    D2 = 2 * a.D;
#pragma unroll
    for (int j = 0; j < C::LOADS; ++j) {
      const int slot = (j * C::WAVES + wave) * 64 + lane;
      const int r = slot / C::CPR, s = slot % C::CPR;
      const int ck = swz_k<C::CPR>(r, s), cv = swz_v<C::CPR>(r, s);
      ok[j] = 16 * ck < D2 ? r * ks2 + ck * 16 : kNowhere;
      ov[j] = 16 * cv < D2 ? r * vs2 + cv * 16 : kNowhere;
    }
  }

  __device__ __forceinline__ void begin(const AttnArgs &a, int kvh, int key0,
                                        int keys, int stage) {
    const int64_t key = (int64_t)key0 + (int64_t)stage * C::KT;
    kat = uniform64(reinterpret_cast<uint64_t>(
        a.k + (int64_t)kvh * a.D + key * a.k_stride));
    vat = uniform64(reinterpret_cast<uint64_t>(
        a.v + (int64_t)kvh * a.D + key * a.v_stride));
    left = keys - stage * C::KT;
  }

  // Without keys the stage is zeros and nothing is read.
  __device__ __forceinline__ void ask(char *to) {
    const int n = min(left, C::KT) - 1;
    const v4u rk = rsrc(kat, n < 0 ? 0 : n * ks2 + D2);
    const v4u rv = rsrc(vat, n < 0 ? 0 : n * vs2 + D2);
    const uint32_t at = lds_at(to + wave * 1024);
#pragma unroll
    for (int j = 0; j < C::LOADS; ++j)
      if ((j * C::WAVES + wave) * 1024 < C::SIDE)
        load_lds16(rk, ok[j], at + j * C::WAVES * 1024);
#pragma unroll
    for (int j = 0; j < C::LOADS; ++j)
      if ((j * C::WAVES + wave) * 1024 < C::SIDE)
        load_lds16(rv, ov[j], at + C::SIDE + j * C::WAVES * 1024);
    kat += (uint64_t)C::KT * ks2;
    vat += (uint64_t)C::KT * vs2;
    left -= C::KT;
  }
};

template <class C>
__global__
__launch_bounds__(C::THREADS, C::WAVES_PER_SIMD) void attention_kernel(
    AttnArgs a, uint32_t per_head, int splits) {
  __shared__ __attribute__((aligned(1024))) char smem[C::LDS];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wq = wave / C::WK, wk = wave % C::WK;
  const int half = lane >> 5;

  // Work groups of one head run on one XCD, whose L2 then holds its keys.
  const uint32_t id = xcd_remap(blockIdx.x, gridDim.x);
  const int kvh = id / per_head;
  uint32_t tile = id - kvh * per_head;
  int split = 0;
  if (splits > 1) {
    split = tile % (uint32_t)splits;
    tile /= (uint32_t)splits;
  }
  const Tile t = find_tile<C::TM>(a, tile);
  if (t.nq == 0) return;
  const int G = a.G;
  const int rows = min(t.nq * G - t.row0, C::TM);
  const int stages_all = ((uint32_t)t.keys + C::KT - 1) / C::KT;
  int st0 = 0, st1 = stages_all;
  if (splits > 1) {
    // at most 2^25 stages and 2^6 parts: within 32 bits
    st0 = (uint32_t)split * (uint32_t)stages_all / (uint32_t)splits;
    st1 = (uint32_t)(split + 1) * (uint32_t)stages_all / (uint32_t)splits;
  }

  const RowMap map(t, G);
  auto token = [&](int r) { return map.tok0 + map.past(r); };
  auto head = [&](int r) { return kvh * G + map.head(r, map.past(r)); };

  Stages<C> ahead;
  ahead.places(a, wave, lane);
  ahead.begin(a, kvh, t.key0, t.keys, st0);
  if (st0 < st1) ahead.ask(smem);

  // Read as fragments, each of Q's lines would be asked for four times.
  Rows<C> w;
  if (C::THROUGH) {
    constexpr int QLOADS = (C::QSIZE / 16 + C::THREADS - 1) / C::THREADS;
    const v4u rq = rsrc(uniform64(reinterpret_cast<uint64_t>(
                            a.q + (int64_t)map.tok0 * a.q_stride +
                            (int64_t)kvh * G * a.D)),
                        0x70000000u);
    const uint32_t at = lds_at(smem + C::STAGE + wave * 1024);
    const int qs2 = (int)(a.q_stride * 2);
#pragma unroll
    for (int j = 0; j < QLOADS; ++j) {
      const int slot = (j * C::WAVES + wave) * 64 + lane;
      const int r = slot / C::CPR, ch = swz_k<C::CPR>(r, slot % C::CPR);
      const int past = map.past(r);
      const int off = past * qs2 + map.head(r, past) * 2 * a.D + ch * 16;
      if ((j * C::WAVES + wave) * 1024 < C::QSIZE)
        load_lds16(rq, r < rows && 8 * ch < a.D ? off : kNowhere,
                   at + j * C::WAVES * 1024);
    }
  } else {
    const int r = min(wq * 32 + (lane & 31), rows - 1);
    const uint16_t *q =
        a.q + (int64_t)token(r) * a.q_stride + (int64_t)head(r) * a.D;
#pragma unroll
    for (int s = 0; s < C::KS; ++s) {
      const int d = 16 * s + 8 * half;
      v4u v = {0, 0, 0, 0};
      if (d < a.D) v = *reinterpret_cast<const v4u *>(q + d);
      w.fq[s] = __builtin_bit_cast(v8bf, v);
    }
  }
  w.places(lane, wk);
  w.clear();
  if (C::THROUGH) {
    wait_vmcnt<0>();
    block_barrier();
    const int r = wq * 32 + (lane & 31);
#pragma unroll
    for (int s = 0; s < C::KS; ++s)
      w.fq[s] = *reinterpret_cast<const v8bf *>(
          smem + C::STAGE + r * C::RB +
          swz_k<C::CPR>(r, 2 * s + half) * 16);
  }
  // Q is there before the loop: a wait for it within would be one for the
  // stages on their way.
#pragma unroll
  for (int s = 0; s < C::KS; ++s) asm volatile("" : "+v"(w.fq[s]));
  wait_vmcnt<0>();
  block_barrier();
  for (int st = st0; st < st1; ++st) {
    const int buf = (st - st0) & 1;
    if (st + 1 < st1) ahead.ask(smem + (buf ^ 1) * C::STAGE);
    w.step(smem + buf * C::STAGE, t.keys - st * C::KT - wk * C::KW,
           a.scale_log2, half);
    // The reads of this stage are done (the compiler leaves its last products, and
    // the waits for their operands, to behind the barrier, where another wave
    // may fill the stage's place, or write its results over it), and the next
    // stage has landed.
    wait_lgkm();
    wait_vmcnt<0>();
    block_barrier();
  }
  v16f(&o)[C::NO] = w.o;
  const float m = w.m, c = a.scale_log2;
  const float l = add_halves(w.l);

  // Join the waves that share rows, and bring O into rows: through LDS, which
  // no wave reads keys from any more.
  const int my_row = wq * 32 + (lane & 31);
  float top = m, sum = l, f = 1.0f;
  if (C::WK > 1) {
    float *ml = reinterpret_cast<float *>(
        smem + C::JOIN - 2 * C::WK * C::TM * 4);  // [WK][TM] of m, then of l
    if (half == 0) {
      ml[wk * C::TM + my_row] = m;
      ml[(C::WK + wk) * C::TM + my_row] = l;
    }
    __syncthreads();
    top = -kInf;
    sum = 0.0f;
#pragma unroll
    for (int w = 0; w < C::WK; ++w) {
      const float lw = ml[(C::WK + w) * C::TM + my_row];
      if (lw != 0.0f) top = fmaxf(top, ml[w * C::TM + my_row]);
    }
#pragma unroll
    for (int w = 0; w < C::WK; ++w) {
      const float lw = ml[(C::WK + w) * C::TM + my_row];
      const float fw =
          lw == 0.0f ? 0.0f
                     : __builtin_amdgcn_exp2f((ml[w * C::TM + my_row] - top) * c);
      if (w == wk) f = fw;
      sum += lw * fw;
    }
  }
  const bool whole = splits == 1;
  // A row that no key has a finite score for is 0 / 0; one without keys is 0.
  if (whole) f *= t.keys == 0 ? 0.0f : 1.0f / sum;
  if (C::WK == 1) {
    // one wave a row: normalized (or not, for a part) and written
    if (!whole) {
      if (half == 0 && my_row < rows) {
        const int64_t at = (int64_t)token(my_row) * a.Hq + head(my_row);
        part_ml(a, splits, split)[at] = make_float2(top, sum);
      }
      if (my_row < rows) {
        float *po = part_o(a, split) +
                    ((int64_t)token(my_row) * a.Hq + head(my_row)) * a.D;
#pragma unroll
        for (int n = 0; n < C::NO; ++n)
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const int d = 32 * n + 2 * e + 4 * half;
            if (d < a.D)
              *reinterpret_cast<float4 *>(po + d) =
                  make_float4(o[n][e] * f, o[n][e + 1] * f, o[n][e + 2] * f,
                              o[n][e + 3] * f);
          }
      }
      return;
    }
    uint16_t *lo = reinterpret_cast<uint16_t *>(smem);
#pragma unroll
    for (int n = 0; n < C::NO; ++n)
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        const v2u two = {pack_bf16x2(o[n][e] * f, o[n][e + 1] * f),
                         pack_bf16x2(o[n][e + 2] * f, o[n][e + 3] * f)};
        *reinterpret_cast<v2u *>(lo + my_row * C::OROW + 32 * n + 2 * e +
                                 4 * half) = two;
      }
    __syncthreads();
    const int per = a.D / 8, step = C::THREADS / per;
    int r = tid / per;
    const int d = 8 * (tid - r * per);
    if (r >= step) r = rows;
    for (; r < rows; r += step) {
      const v2u *src = reinterpret_cast<const v2u *>(lo + r * C::OROW + d);
      const v2u x = src[0], y = src[1];
      *reinterpret_cast<v4u *>(a.out + (int64_t)token(r) * a.out_stride +
                               (int64_t)head(r) * a.D + d) =
          v4u{x.x, x.y, y.x, y.y};
    }
  } else {
    float *lo = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int n = 0; n < C::NO; ++n)
#pragma unroll
      for (int e = 0; e < 16; e += 4)
        *reinterpret_cast<float4 *>(lo + (wk * C::TM + my_row) * C::OROW +
                                    32 * n + 2 * e + 4 * half) =
            make_float4(o[n][e] * f, o[n][e + 1] * f, o[n][e + 2] * f,
                        o[n][e + 3] * f);
    if (!whole && wk == 0 && half == 0 && my_row < rows) {
      const int64_t at = (int64_t)token(my_row) * a.Hq + head(my_row);
      part_ml(a, splits, split)[at] = make_float2(top, sum);
    }
    __syncthreads();
    const int per = a.D / 4, step = C::THREADS / per;
    int r = tid / per;
    const int d = 4 * (tid - r * per);
    if (r >= step) r = rows;
    for (; r < rows; r += step) {
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < C::WK; ++w) {
        const float4 x = *reinterpret_cast<const float4 *>(
            lo + (w * C::TM + r) * C::OROW + d);
        v = make_float4(v.x + x.x, v.y + x.y, v.z + x.z, v.w + x.w);
      }
      const int tok = token(r), hd = head(r);
      if (whole)
        *reinterpret_cast<v2u *>(a.out + (int64_t)tok * a.out_stride +
                                 (int64_t)hd * a.D + d) =
            v2u{pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w)};
      else
        *reinterpret_cast<float4 *>(
            part_o(a, split) + ((int64_t)tok * a.Hq + hd) * a.D + d) = v;
    }
  }
}

// Joins the parts of a split: a row's largest m, its parts' sums and values
// scaled to that.  A part without keys has l 0 and its O is not read.  A thread
// takes 4 values of a row; few rows a work group, so that all parts of a call of
// few rows are on their way at once.
constexpr int kJoinThreads = 256;
constexpr int kJoinRows = 8;
constexpr int kMaxSplits = 64;

__global__ __launch_bounds__(kJoinThreads) void attention_join_kernel(
    AttnArgs a, uint32_t per_head, int splits) {
  __shared__ float2 parts[kJoinRows][kMaxSplits];  // l and the factor of a part
  const int kvh = blockIdx.x / per_head;
  const Tile t = find_tile<kJoinRows>(a, blockIdx.x - kvh * per_head);
  if (t.nq == 0) return;
  const int G = a.G;
  const int rows = min(t.nq * G - t.row0, kJoinRows);
  const RowMap map(t, G);
  auto row_at = [&](int r) {
    const int past = map.past(r);
    return (int64_t)(map.tok0 + past) * a.Hq + kvh * G + map.head(r, past);
  };
  const int lane = threadIdx.x & 63;
  for (int r = threadIdx.x >> 6; r < rows; r += kJoinThreads / 64) {
    float2 ml = make_float2(-kInf, 0.0f);
    if (lane < splits) ml = part_ml(a, splits, lane)[row_at(r)];
    float top = ml.y != 0.0f ? ml.x : -kInf;
#pragma unroll
    for (int s = 32; s > 0; s /= 2) top = fmaxf(top, __shfl_xor(top, s));
    parts[r][lane] = make_float2(
        ml.y, ml.y == 0.0f
                  ? 0.0f
                  : __builtin_amdgcn_exp2f((ml.x - top) * a.scale_log2));
  }
  __syncthreads();
  const int per = a.D / 4;
  for (int i = threadIdx.x; i < rows * per; i += kJoinThreads) {
    const int r = i / per, d = 4 * (i - r * per);
    const int64_t at = row_at(r);
    float sum = 0.0f;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
      const float2 p = parts[r][s];
      float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (p.x != 0.0f)
        x = *reinterpret_cast<const float4 *>(part_o(a, s) + at * a.D + d);
      sum = fmaf(p.x, p.y, sum);
      v = make_float4(fmaf(x.x, p.y, v.x), fmaf(x.y, p.y, v.y),
                      fmaf(x.z, p.y, v.z), fmaf(x.w, p.y, v.w));
    }
    const float f = t.keys == 0 ? 0.0f : 1.0f / sum;
    const int past = map.past(r);
    *reinterpret_cast<v2u *>(a.out + (int64_t)(map.tok0 + past) * a.out_stride +
                             (int64_t)(kvh * G + map.head(r, past)) * a.D + d) =
        v2u{pack_bf16x2(v.x * f, v.y * f), pack_bf16x2(v.z * f, v.w * f)};
  }
}

enum Config : int { kFew, kSome, kMid, kShort, kMany };
constexpr int kTileRows[5] = {32, 64, 128, 128, 256};
constexpr int kThreads[5] = {256, 512, 256, 256, 512};

template <class C>
hipError_t launch_cfg(const AttnArgs &a, const AttnPlan &plan,
                      hipStream_t stream) {
  const unsigned blocks = (unsigned)(plan.tiles * a.Hk * plan.splits);
  attention_kernel<C><<<blocks, C::THREADS, 0, stream>>>(
      a, (uint32_t)(plan.tiles * plan.splits), plan.splits);
  return hipGetLastError();
}

template <int DP>
hipError_t launch_width(const AttnArgs &a, const AttnPlan &plan,
                        hipStream_t stream) {
  switch (plan.config) {
    case kFew: return launch_cfg<Cfg<1, 4, 128, DP>>(a, plan, stream);
    case kSome: return launch_cfg<Cfg<2, 4, 128, DP>>(a, plan, stream);
    case kMid: return launch_cfg<Cfg<4, 1, 64, DP>>(a, plan, stream);
    case kShort: return launch_cfg<Cfg<4, 1, 32, DP>>(a, plan, stream);
    default: return launch_cfg<Cfg<8, 1, 64, DP>>(a, plan, stream);
  }
}


int64_t count_tiles(int64_t Tq, int64_t B, bool packed, int64_t G, int rows) {
  return packed ? Tq * G / rows + B : B * ((Tq / B * G + rows - 1) / rows);
}

}  // namespace

AttnPlan plan_attention(int64_t Tq, int64_t Tk, int64_t B, bool packed,
                        int64_t Hq, int64_t Hk, int64_t D) {
  AttnPlan p{};
  const int64_t G = Hq / Hk;
  const int64_t rows = (Tq + B - 1) / B * G;  // of a sequence, on average
  const int64_t keys = Tk / B;
  // Up to 32 and 64 rows, the tile that holds them, so that keys are read once (64
  // queries to 37503 keys: 221 us in one tile of 64 rows, 334 in two of 32).
  // Tiles of 256 rows (kMany) share a stage of keys among the most rows.  With
  // few keys two work groups of 128 rows a compute unit (kMid) do better: one's
  // loads of Q and stores of O go on beside the other's products (19077 tokens, 56
  // heads of 128: to 512 keys 342 us beside 368, to 2000 1065 beside 1063; 4096 to
  // 4096, 42 heads 373 beside 344); and where there are tiles for it, three with
  // stages of 32 keys (kShort beside kMid: 19077 to 77 keys 147 us and 160, to 310 244
  // and 252, to 1000 588 and 587, to 2000 1078 and 1065; 300 to 300, 13.5 and 11.2).
  // Where tiles of 256 are fewer than a quarter of the compute units, tiles of 64
  // rows, whose waves split a stage's keys (kSome beside kMany: 8 heads, 300 queries
  // to 8192 keys 27 us and 32; 56 heads, 300 to 300, 112 tiles: 18 and 15).  All at
  // width 128; no other width was measured.
  const int64_t large = count_tiles(Tq, B, packed, G, kTileRows[kMany]) * Hk;
  p.config = rows <= 32                    ? kFew
             : rows <= 64 || large < 64    ? kSome
             : keys > 2048                 ? kMany
             : keys > 1024 || large <= 512 ? kMid
                                           : kShort;
  p.tiles = count_tiles(Tq, B, packed, G, kTileRows[p.config]);
  // Keys are split where the tiles leave compute units idle, into a part a unit.
  // The join behind it costs as much as three or four stages (one query, 56
  // heads: 512 keys 10.6 us whole, 11.4 in 4 parts; 2048 keys 27 and 18).
  const int64_t groups = p.tiles * Hk;
  const int64_t stages = (keys + 127) / 128;
  int64_t splits = groups >= 256 ? 1 : 256 / groups;
  if (splits > stages) splits = stages;
  if (splits > kMaxSplits) splits = kMaxSplits;
  if (splits < 1 || stages - (stages + splits - 1) / splits < 4) splits = 1;
  p.splits = (int)splits;
  if (p.splits > 1)
    p.workspace = (size_t)p.splits * Tq * Hq * (D * 4 + 8);
  return p;
}

bool attention_launchable(const AttnPlan &plan, int64_t Hk) {
  return plan.tiles * Hk * plan.splits <
         (int64_t(1) << 32) / kThreads[plan.config];
}

hipError_t launch_attention(const AttnArgs &a, const AttnPlan &plan,
                            hipStream_t stream) {
  hipError_t e;
  if (a.D <= 32) e = launch_width<32>(a, plan, stream);
  else if (a.D <= 64) e = launch_width<64>(a, plan, stream);
  else if (a.D <= 96) e = launch_width<96>(a, plan, stream);
  else e = launch_width<128>(a, plan, stream);
  if (e != hipSuccess || plan.splits == 1) return e;
  const int64_t tiles =
      count_tiles(a.Tq, a.B, a.q_offsets != nullptr, a.Hq / a.Hk, kJoinRows);
  attention_join_kernel<<<(unsigned)(tiles * a.Hk), kJoinThreads, 0, stream>>>(
      a, (uint32_t)tiles, plan.splits);
  return hipGetLastError();
}

}  // namespace w8a8
