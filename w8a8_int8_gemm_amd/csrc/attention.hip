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
// Weights p = 2^(c s - c m) are rounded to BF16 for the matrix unit; l sums the
// rounded ones, so that each row's weights still sum to one.  m lags: it moves
// (and O and l with it) only where a row's scores pass it by more than 2^8, so
// p stays below 2^8 and the sums far inside binary32.
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
constexpr float kLag = 8.0f;  // how far scores may pass m, in powers of two

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
  static constexpr int LOADS = SIDE / 16 / THREADS;  // of K a thread and stage
  static constexpr int OROW = DP + 4;            // floats of a joined row
  static constexpr int JOIN = (WK > 1 ? WK * TM * OROW * 4 : TM * OROW * 2) +
                              2 * WK * TM * 4;
  static constexpr int LDS = 2 * STAGE > JOIN ? 2 * STAGE : JOIN;
  static_assert(LDS <= 160 * 1024 && SIDE % (16 * THREADS) == 0, "");
};

// Where chunk c of row r lies in its row: fragments are read by 8 lanes a cycle
// from consecutive rows (K), or as pairs of chunks of 4 consecutive rows (V),
// which must fall into different parts of 128 bytes.
template <int CPR>
__device__ __forceinline__ int swz_k(int r, int c) {
  return CPR == 4 ? c ^ ((r >> 1) & 3) : c ^ (r & (CPR - 1));
}

template <int CPR>
__device__ __forceinline__ int swz_v(int r, int c) {
  return CPR == 4 ? c ^ (((r >> 1) & 1) * 2) : c ^ ((r & (CPR / 2 - 1)) * 2);
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

// Barrier without the fences of __syncthreads, which would wait for direct
// loads on their way; the waits are written out where they are due.
__device__ __forceinline__ void block_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Uniform 64-bit address -> buffer resource of `bytes` bytes: reads past them
// give zeros, in LDS too.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void *p,
                                                       uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  const uint64_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)a);
  const uint64_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(a >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(
      (void *)(uintptr_t)((hi << 32) | lo), 0,
      __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000);
}

// 16 bytes per lane from buffer `r` at byte voff into LDS at `l` (lane i's bytes
// at l + 16 i).
__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t r, int voff,
                                           char *l) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)l, 16, voff, 0, 0, 0);
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

__device__ __forceinline__ void keys_of(const AttnArgs &a, int b, Tile &t) {
  if (a.k_offsets) {
    t.key0 = clamped(a.k_offsets[b], 0, a.Tk);
    t.keys = clamped(a.k_offsets[b + 1], t.key0, a.Tk) - t.key0;
  } else {
    t.keys = a.Tk / a.B;
    t.key0 = b * t.keys;
  }
  if (a.k_lens) t.keys = clamped(a.k_lens[b], 0, t.keys);
}

// Tile `i` of all sequences, TM rows each; false past the last.  Offsets are
// clamped to the rows there are, so no content of theirs leads outside.
template <int TM>
__device__ __forceinline__ bool find_tile(const AttnArgs &a, int64_t i,
                                          Tile &t) {
  const int G = a.Hq / a.Hk;
  if (!a.q_offsets) {
    t.nq = a.Tq / a.B;
    const int64_t per = ((int64_t)t.nq * G + TM - 1) / TM;
    const int b = (int)(i / per);
    t.q0 = b * t.nq;
    t.row0 = (int)(i - b * per) * TM;
    if (b >= a.B) return false;
    keys_of(a, b, t);
    return true;
  }
  // 64 sequences at a time: their tile counts summed over the lanes.
  const int lane = threadIdx.x & 63;
  for (int b0 = 0; b0 < a.B; b0 += 64) {
    const int b = b0 + lane;
    int q0 = 0, nq = 0;
    if (b < a.B) {
      q0 = clamped(a.q_offsets[b], 0, a.Tq);
      nq = clamped(a.q_offsets[b + 1], q0, a.Tq) - q0;
    }
    const int mine = (int)(((int64_t)nq * G + TM - 1) / TM);
    int upto = mine;
#pragma unroll
    for (int s = 1; s < 64; s *= 2) {
      const int o = __shfl_up(upto, s);
      if (lane >= s) upto += o;
    }
    const int total = __builtin_amdgcn_readlane(upto, 63);
    if (i < total) {
      const uint64_t past = __ballot(upto > (int)i);
      const int at = __builtin_ctzll(past);
      t.q0 = __builtin_amdgcn_readlane(q0, at);
      t.nq = __builtin_amdgcn_readlane(nq, at);
      t.row0 = ((int)i - (__builtin_amdgcn_readlane(upto, at) -
                          __builtin_amdgcn_readlane(mine, at))) * TM;
      keys_of(a, b0 + at, t);
      return true;
    }
    i -= total;
  }
  return false;
}

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
// part and row c m and l.
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

template <class C>
__global__ __launch_bounds__(C::THREADS) void attention_kernel(AttnArgs a,
                                                               int splits) {
  __shared__ __attribute__((aligned(1024))) char smem[C::LDS];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wq = wave / C::WK, wk = wave % C::WK;
  const int half = lane >> 5;

  // Work groups of one head run on one XCD, whose L2 then holds its keys.
  const int64_t id = xcd_remap(blockIdx.x, gridDim.x);
  const int64_t per_head = gridDim.x / a.Hk;
  const int kvh = (int)(id / per_head);
  const int64_t rest = id - kvh * per_head;
  const int split = (int)(rest % splits);
  Tile t;
  if (!find_tile<C::TM>(a, rest / splits, t)) return;
  const int G = a.Hq / a.Hk;
  const int rows = min((int64_t)t.nq * G - t.row0, (int64_t)C::TM);
  const int stages_all = (t.keys + C::KT - 1) / C::KT;
  const int st0 = (int)((int64_t)split * stages_all / splits);
  const int st1 = (int)((int64_t)(split + 1) * stages_all / splits);

  // Query row r of the tile: token and head of its sequence's row.
  auto token = [&](int r) { return t.q0 + (t.row0 + r) / G; };
  auto head = [&](int r) { return kvh * G + (t.row0 + r) % G; };

  // Q^T as the right operand: lane's query, 8 values a step.
  v8bf fq[C::KS];
  {
    const int r = min(wq * 32 + (lane & 31), rows - 1);
    const uint16_t *q =
        a.q + (int64_t)token(r) * a.q_stride + (int64_t)head(r) * a.D;
#pragma unroll
    for (int s = 0; s < C::KS; ++s) {
      const int d = 16 * s + 8 * half;
      v4u v = {0, 0, 0, 0};
      if (d < a.D) v = *reinterpret_cast<const v4u *>(q + d);
      fq[s] = __builtin_bit_cast(v8bf, v);
    }
  }

  // Direct loads: what lands in this thread's 16 bytes of a stage.
  int ok[C::LOADS], ov[C::LOADS];
  const int ks2 = (int)(a.k_stride * 2), vs2 = (int)(a.v_stride * 2);
  constexpr int kNowhere = 0x7FFFFFF0;
#pragma unroll
  for (int j = 0; j < C::LOADS; ++j) {
    const int slot = (j * C::WAVES + wave) * 64 + lane;
    const int r = slot / C::CPR, s = slot % C::CPR;
    const int ck = swz_k<C::CPR>(r, s), cv = swz_v<C::CPR>(r, s);
    ok[j] = 8 * ck < a.D ? r * ks2 + ck * 16 : kNowhere;
    ov[j] = 8 * cv < a.D ? r * vs2 + cv * 16 : kNowhere;
  }
  const uint16_t *kb = a.k + (int64_t)kvh * a.D, *vb = a.v + (int64_t)kvh * a.D;
  auto issue = [&](int buf, int st) {
    const int64_t key = (int64_t)t.key0 + (int64_t)st * C::KT;
    const int left = min(t.keys - st * C::KT, C::KT);
    const auto rk = rsrc(kb + key * a.k_stride,
                         (uint32_t)(left - 1) * ks2 + 2 * a.D);
    const auto rv = rsrc(vb + key * a.v_stride,
                         (uint32_t)(left - 1) * vs2 + 2 * a.D);
    char *base = smem + buf * C::STAGE + wave * 1024;
#pragma unroll
    for (int j = 0; j < C::LOADS; ++j)
      load_lds16(rk, ok[j], base + j * C::WAVES * 1024);
#pragma unroll
    for (int j = 0; j < C::LOADS; ++j)
      load_lds16(rv, ov[j], base + C::SIDE + j * C::WAVES * 1024);
  };

  // Fragments of K: key (lane & 31) of a score tile, 8 values a step.
  int ak[C::KS];
  {
    const int r = lane & 31;
#pragma unroll
    for (int s = 0; s < C::KS; ++s)
      ak[s] = (wk * C::KW + r) * C::RB + swz_k<C::CPR>(r, 2 * s + half) * 16;
  }
  // Fragments of V^T: of 16 keys a lane needs those that its scores stand for
  // (4 half .. + 3 and 8 further), of value (lane & 31) of an output tile; a
  // transposing read gives 16 lanes 4 keys of 16 values.
  int av[C::NO];
  {
    const int i = lane & 15, r = 4 * half + i / 4;
#pragma unroll
    for (int n = 0; n < C::NO; ++n) {
      const int c = 4 * n + 2 * ((lane >> 4) & 1) + (i & 3) / 2;
      av[n] = C::SIDE + (wk * C::KW + r) * C::RB + swz_v<C::CPR>(r, c) * 16 +
              (i & 1) * 8;
    }
  }

  v16f o[C::NO];
#pragma unroll
  for (int n = 0; n < C::NO; ++n)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[n][e] = 0.0f;
  float m = -kInf, cm = 0.0f, l = 0.0f;
  const float c = a.scale_log2;

  if (st0 < st1) issue(0, st0);
  wait_vmcnt<0>();
  block_barrier();
  for (int st = st0; st < st1; ++st) {
    const int buf = (st - st0) & 1;
    if (st + 1 < st1) issue(buf ^ 1, st + 1);
    const char *base = smem + buf * C::STAGE;

    v16f s[C::NS];
#pragma unroll
    for (int n = 0; n < C::NS; ++n) {
#pragma unroll
      for (int e = 0; e < 16; ++e) s[n][e] = 0.0f;
#pragma unroll
      for (int k = 0; k < C::KS; ++k) {
        const v8bf fk = *reinterpret_cast<const v8bf *>(
            base + ak[k] + n * 32 * C::RB);
        s[n] = mfma(fk, fq[k], s[n]);
      }
    }
    // Keys past the end (their rows of LDS are zeros, whatever memory holds).
    const int left = t.keys - st * C::KT - wk * C::KW;
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
    if (__any(fmaf(top, c, -cm) > kLag || (m == -kInf && top > m))) {
      const float now = fmaxf(m, max_halves(top));
      const float was = m;
      m = now;
      const float ncm = now == -kInf ? 0.0f : now * c;
      const float f =
          was == -kInf ? 0.0f : __builtin_amdgcn_exp2f(cm - ncm);
      cm = ncm;
      l *= f;
#pragma unroll
      for (int n = 0; n < C::NO; ++n)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[n][e] *= f;
    }
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
    wait_vmcnt<0>();
    block_barrier();
  }
  l = add_halves(l);

  // Join the waves that share rows, and bring O into rows: through LDS, which
  // no wave reads keys from any more.
  float *ml = reinterpret_cast<float *>(
      smem + C::JOIN - 2 * C::WK * C::TM * 4);  // [WK][TM] of c m, then of l
  const int my_row = wq * 32 + (lane & 31);
  if (half == 0) {
    ml[wk * C::TM + my_row] = cm;
    ml[(C::WK + wk) * C::TM + my_row] = l;
  }
  __syncthreads();
  float top = -kInf, sum = 0.0f, f = 1.0f;
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
                   : __builtin_amdgcn_exp2f(ml[w * C::TM + my_row] - top);
    if (w == wk) f = fw;
    sum += lw * fw;
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
    const int per = a.D / 8;
    for (int i = tid; i < rows * per; i += C::THREADS) {
      const int r = i / per, d = 8 * (i - r * per);
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
    const int per = a.D / 4;
    for (int i = tid; i < rows * per; i += C::THREADS) {
      const int r = i / per, d = 4 * (i - r * per);
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

// Joins the parts of a split: a row's largest c m, its parts' sums and values
// scaled to that.  A part without keys has l 0 and its O is not read.
constexpr int kJoinThreads = 256;
constexpr int kJoinRows = 32;

__global__ __launch_bounds__(kJoinThreads) void attention_join_kernel(
    AttnArgs a, int splits) {
  const int64_t per_head = gridDim.x / a.Hk;
  const int kvh = (int)(blockIdx.x / per_head);
  Tile t;
  if (!find_tile<kJoinRows>(a, blockIdx.x - kvh * per_head, t)) return;
  const int G = a.Hq / a.Hk;
  const int rows = min((int64_t)t.nq * G - t.row0, (int64_t)kJoinRows);
  const int per = a.D / 4;
  for (int i = threadIdx.x; i < rows * per; i += kJoinThreads) {
    const int r = i / per, d = 4 * (i - r * per);
    const int tok = t.q0 + (t.row0 + r) / G, hd = kvh * G + (t.row0 + r) % G;
    const int64_t at = (int64_t)tok * a.Hq + hd;
    float top = -kInf;
    for (int s = 0; s < splits; ++s) {
      const float2 ml = part_ml(a, splits, s)[at];
      if (ml.y != 0.0f) top = fmaxf(top, ml.x);
    }
    float sum = 0.0f;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int s = 0; s < splits; ++s) {
      const float2 ml = part_ml(a, splits, s)[at];
      if (ml.y == 0.0f) continue;
      const float f = __builtin_amdgcn_exp2f(ml.x - top);
      sum += ml.y * f;
      const float4 x =
          *reinterpret_cast<const float4 *>(part_o(a, s) + at * a.D + d);
      v = make_float4(fmaf(x.x, f, v.x), fmaf(x.y, f, v.y), fmaf(x.z, f, v.z),
                      fmaf(x.w, f, v.w));
    }
    const float f = t.keys == 0 ? 0.0f : 1.0f / sum;
    *reinterpret_cast<v2u *>(a.out + (int64_t)tok * a.out_stride +
                             (int64_t)hd * a.D + d) =
        v2u{pack_bf16x2(v.x * f, v.y * f), pack_bf16x2(v.z * f, v.w * f)};
  }
}

template <class C>
hipError_t launch_cfg(const AttnArgs &a, const AttnPlan &plan,
                      hipStream_t stream) {
  const unsigned blocks = (unsigned)(plan.tiles * a.Hk * plan.splits);
  attention_kernel<C><<<blocks, C::THREADS, 0, stream>>>(a, plan.splits);
  return hipGetLastError();
}

template <int DP>
hipError_t launch_width(const AttnArgs &a, const AttnPlan &plan,
                        hipStream_t stream) {
  switch (plan.config) {
    case 0: return launch_cfg<Cfg<1, 4, 128, DP>>(a, plan, stream);
    case 1: return launch_cfg<Cfg<2, 4, 128, DP>>(a, plan, stream);
    default:
      return launch_cfg<Cfg<8, 1, DP == 32 ? 128 : 64, DP>>(a, plan, stream);
  }
}

constexpr int kTileRows[3] = {32, 64, 256};

int64_t count_tiles(int64_t Tq, int64_t B, bool packed, int64_t G, int rows) {
  return packed ? Tq * G / rows + B : B * ((Tq / B * G + rows - 1) / rows);
}

}  // namespace

AttnPlan plan_attention(int64_t Tq, int64_t Tk, int64_t B, bool packed,
                        int64_t Hq, int64_t Hk, int64_t D) {
  AttnPlan p{};
  const int64_t G = Hq / Hk;
  const int64_t rows = (Tq + B - 1) / B * G;  // of a sequence, on average
  p.config = rows <= 32 ? 0 : rows <= 64 ? 1 : 2;
  p.tiles = count_tiles(Tq, B, packed, G, kTileRows[p.config]);
  // Keys are split where the tiles leave compute units idle.
  const int64_t groups = p.tiles * Hk;
  const int64_t stages = (Tk / B + 127) / 128;
  int64_t splits = groups >= 256 ? 1 : 512 / groups;
  if (splits > stages / 2) splits = stages / 2;
  if (splits > 64) splits = 64;
  p.splits = splits < 1 ? 1 : (int)splits;
  if (p.splits > 1)
    p.workspace = (size_t)p.splits * Tq * Hq * (D * 4 + 8);
  return p;
}

bool attention_launchable(const AttnPlan &plan, int64_t Hk) {
  const int threads[3] = {256, 512, 512};
  return plan.tiles * Hk * plan.splits <
         (int64_t(1) << 32) / threads[plan.config];
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
      a, plan.splits);
  return hipGetLastError();
}

}  // namespace w8a8
