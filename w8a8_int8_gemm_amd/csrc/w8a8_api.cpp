// w8a8_api.cpp -- the C ABI declared in include/w8a8.h.
//
// Every entry point validates its arguments on the host first (pointers,
// shape contract, alignment, overlap, workspace size, device) and launches
// nothing when a check fails; only then does it enqueue kernels on the
// caller's stream.  The library allocates nothing and never synchronizes.
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstring>
#include <mutex>
#include <unordered_map>

#include "heads.h"
#include "internal.h"
#include "norm.h"
#include "rope.h"
#include "rowwise.h"
#include "w4.h"
#include "w8a8.h"

namespace {

using w8a8::GemmArgs;
using w8a8::GemmPlan;

// Largest K the register-resident row kernels cover (44 chunks of 8 BF16
// per lane x 4 waves x 64 lanes): the glue kernels (SiLU, renormalization)
// and the fused quantizers.  The plain quantizers (activations, weights)
// take longer rows, up to W8A8_MAX_K, through a kernel that reads each row
// twice.
constexpr int64_t kGlueMaxK = 44 * 8 * 4 * 64;
constexpr int64_t kQuantMaxK = W8A8_MAX_K;
constexpr int64_t kMaxRows = 0x7FFFFFFF;
// Rows of the per-token kernels: their launches hold up to 256 work-items
// per row, and a launch holds fewer than 2^32 work-items.
constexpr int64_t kMaxTokenRows = (int64_t(1) << 24) - 1;

thread_local int g_last_hip_error = 0;

inline bool aligned(const void *p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};

inline Range range_of(const void *p, int64_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Range{lo, lo + (uintptr_t)(bytes > 0 ? bytes : 0)};
}

inline bool overlap(Range a, Range b) {
  return a.lo < b.hi && b.lo < a.hi && a.hi > a.lo && b.hi > b.lo;
}

inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// The current device must be gfx950; checked once per device and cached.
int check_device() {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return W8A8_ERR_DEVICE;
  static std::mutex mu;
  static std::unordered_map<int, int> checked;
  std::lock_guard<std::mutex> lock(mu);
  auto it = checked.find(dev);
  if (it != checked.end()) return it->second;
  hipDeviceProp_t prop;
  int status = W8A8_ERR_DEVICE;
  if (hipGetDeviceProperties(&prop, dev) == hipSuccess &&
      std::strncmp(prop.gcnArchName, "gfx950", 6) == 0)
    status = W8A8_OK;
  // Set-up on the first call on a gfx950 device, with it current: the
  // address of this device's copy of the allocation-free entry point's
  // scratch (a failure is reported by that entry point, which retries).
  if (status == W8A8_OK) (void)w8a8::resolve_scratch(dev);
  checked[dev] = status;
  return status;
}

inline int hip_status(hipError_t e) {
  if (e == hipSuccess) return W8A8_OK;
  g_last_hip_error = (int)e;
  return W8A8_ERR_HIP;
}

bool gemm_shape_ok(int64_t M, int64_t N, int64_t K) {
  return M >= 1 && M <= kMaxRows && N >= 128 && N % 128 == 0 &&
         N <= kMaxRows && K >= 128 && K % 128 == 0 && K <= W8A8_MAX_K;
}

int validate_quant(const uint16_t *x, int64_t M, int64_t K, const int8_t *q,
                   const float *sa, int64_t max_k = kQuantMaxK) {
  if (!x || !q || !sa) return W8A8_ERR_NULL;
  if (M < 1 || M > kMaxTokenRows || K < 8 || K % 8 != 0 || K > max_k)
    return W8A8_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(q, 8) || !aligned(sa, 4))
    return W8A8_ERR_ALIGN;
  const Range rx = range_of(x, M * K * 2), rq = range_of(q, M * K),
              rs = range_of(sa, M * 4);
  if (overlap(rx, rq) || overlap(rx, rs) || overlap(rq, rs))
    return W8A8_ERR_ALIAS;
  return W8A8_OK;
}

int out_elem_bytes(int out_dtype) {
  switch (out_dtype) {
    case W8A8_OUT_BF16: return 2;
    case W8A8_OUT_FP32: return 4;
    case W8A8_OUT_I32: return 4;
    default: return 0;
  }
}

// Everything w8a8_gemm checks except its workspace: pointers, shape,
// output type, alignment, a launchable plan and overlaps between the
// output and the inputs.
int validate_gemm_args(const int8_t *a_q, const float *a_scale,
                       const int8_t *w_q, const float *w_scale,
                       const uint16_t *bias, const void *out, int out_dtype,
                       int64_t M, int64_t N, int64_t K, GemmPlan *plan) {
  if (!a_q || !a_scale || !w_q || !w_scale || !out) return W8A8_ERR_NULL;
  if (!gemm_shape_ok(M, N, K)) return W8A8_ERR_SHAPE;
  const int eb = out_elem_bytes(out_dtype);
  if (eb == 0) return W8A8_ERR_OUT_DTYPE;
  if (!aligned(a_q, 16) || !aligned(w_q, 16) || !aligned(out, 16) ||
      !aligned(w_scale, 4) || !aligned(a_scale, 4) ||
      (bias && !aligned(bias, 2)))
    return W8A8_ERR_ALIGN;
  *plan = w8a8::plan_gemm(M, N, K);
  if (!w8a8::plan_launchable(*plan)) return W8A8_ERR_SHAPE;
  const Range ro = range_of(out, M * N * eb);
  const Range ins[] = {range_of(a_q, M * K), range_of(a_scale, M * 4),
                       range_of(w_q, N * K), range_of(w_scale, N * 4),
                       range_of(bias, bias ? N * 2 : 0)};
  for (const Range &r : ins)
    if (overlap(ro, r)) return W8A8_ERR_ALIAS;
  return W8A8_OK;
}

// The partial-sum buffer of a plan against the call's other buffers.
int scratch_alias(const void *buf, const GemmPlan &plan, const int8_t *a_q,
                  const float *a_scale, const int8_t *w_q,
                  const float *w_scale, const uint16_t *bias,
                  const void *out, int out_dtype, int64_t M, int64_t N,
                  int64_t K) {
  if (plan.workspace == 0) return W8A8_OK;
  const Range rw = range_of(buf, (int64_t)plan.workspace);
  const Range all[] = {range_of(out, M * N * out_elem_bytes(out_dtype)),
                       range_of(a_q, M * K), range_of(a_scale, M * 4),
                       range_of(w_q, N * K), range_of(w_scale, N * 4),
                       range_of(bias, bias ? N * 2 : 0)};
  for (const Range &r : all)
    if (overlap(rw, r)) return W8A8_ERR_ALIAS;
  return W8A8_OK;
}

int validate_gemm(const int8_t *a_q, const float *a_scale, const int8_t *w_q,
                  const float *w_scale, const uint16_t *bias, const void *out,
                  int out_dtype, int64_t M, int64_t N, int64_t K,
                  const void *workspace, size_t workspace_bytes,
                  GemmPlan *plan) {
  int st = validate_gemm_args(a_q, a_scale, w_q, w_scale, bias, out,
                              out_dtype, M, N, K, plan);
  if (st != W8A8_OK) return st;
  if (plan->workspace > 0) {
    if (!workspace || workspace_bytes < plan->workspace)
      return W8A8_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return W8A8_ERR_ALIGN;
  }
  return scratch_alias(workspace, *plan, a_q, a_scale, w_q, w_scale, bias,
                       out, out_dtype, M, N, K);
}

// One norm of a block-norm call: its kind and constants.
int validate_norm(const w8a8_norm_t *n) {
  if (!n || n->kind == W8A8_NORM_NONE)
    return n && (n->weight || n->bias) ? W8A8_ERR_ARG : W8A8_OK;
  if (n->kind != W8A8_NORM_RMS && n->kind != W8A8_NORM_LAYER)
    return W8A8_ERR_ARG;
  if (!(n->eps >= FLT_MIN) || !std::isfinite(n->eps)) return W8A8_ERR_ARG;
  if (n->bias && n->kind != W8A8_NORM_LAYER) return W8A8_ERR_ARG;
  if ((n->weight && !aligned(n->weight, 16)) ||
      (n->bias && !aligned(n->bias, 16)))
    return W8A8_ERR_ALIGN;
  return W8A8_OK;
}

// Row strides of a modulation table: the bytes of 2^31 rows stay below 2^63.
constexpr int64_t kMaxModStride = int64_t(1) << 30;

// Bytes a modulation table spans, or -1 for a stride the contract rejects.
int64_t mod_bytes(int64_t stride, int64_t rows, int64_t H) {
  if (stride != 0 && (stride < H || stride % 8 != 0 || stride >= kMaxModStride))
    return -1;
  return ((rows - 1) * stride + H) * 2;
}

// The block norms: everything is checked here, `a` filled in and the kernel
// launched.  Which outputs there are says what is computed.
int block_norm(const uint16_t *x, const uint16_t *branch, int64_t M,
               int64_t H, const w8a8_norm_t *post, const w8a8_norm_t *pre,
               const w8a8_modulation_t *mod, float residual_scale,
               uint16_t *r, uint16_t *y, int8_t *q, float *qs, void *stream) {
  // With up to 24 values a thread and at least 64 threads a row, fewer than
  // 2^36 values keep a launch below 2^32 work-items.
  if (M < 1 || M > kMaxTokenRows || H < 8 || H % 8 != 0 ||
      H > W8A8_NORM_MAX_H || M * H >= (int64_t(1) << 36))
    return W8A8_ERR_SHAPE;
  int st = validate_norm(post);
  if (st == W8A8_OK) st = validate_norm(pre);
  if (st != W8A8_OK) return st;
  if (!std::isfinite(residual_scale)) return W8A8_ERR_ARG;
  w8a8::NormArgs a{};
  if (mod) {
    const bool any = mod->scale || mod->shift || mod->gate || mod->row;
    if (any ? mod->rows < 1 || mod->rows > kMaxRows : mod->rows < 0)
      return W8A8_ERR_SHAPE;
    if (any && !mod->row && mod->rows != 1 && mod->rows != M)
      return W8A8_ERR_SHAPE;
    if (mod->row && !aligned(mod->row, 4)) return W8A8_ERR_ALIGN;
    a.scale = mod->scale;
    a.shift = mod->shift;
    a.gate = mod->gate;
    a.scale_stride = mod->scale_stride;
    a.shift_stride = mod->shift_stride;
    a.gate_stride = mod->gate_stride;
    a.row = mod->row;
    a.rows = any ? (int)mod->rows : 1;
    a.row_step = any && !mod->row && mod->rows > 1 ? 1 : 0;
  } else {
    a.rows = 1;
  }
  // Inputs besides x and branch, with their sizes in bytes.
  const void *in[8];
  int64_t in_bytes[8];
  int n_in = 0;
  const uint16_t *vec[3] = {a.scale, a.shift, a.gate};
  const int64_t stride[3] = {a.scale_stride, a.shift_stride, a.gate_stride};
  for (int i = 0; i < 3; ++i) {
    if (!vec[i]) continue;
    const int64_t bytes = mod_bytes(stride[i], a.rows, H);
    if (bytes < 0) return W8A8_ERR_SHAPE;
    if (!aligned(vec[i], 16)) return W8A8_ERR_ALIGN;
    in[n_in] = vec[i];
    in_bytes[n_in++] = bytes;
  }
  if (a.row) {
    in[n_in] = a.row;
    in_bytes[n_in++] = M * 4;
  }
  if (post) {
    a.post_kind = post->kind;
    a.post_eps = post->eps;
    a.post_weight = post->weight;
    a.post_bias = post->bias;
  }
  if (pre) {
    a.kind = pre->kind;
    a.eps = pre->eps;
    a.weight = pre->weight;
    a.bias = pre->bias;
  }
  for (const uint16_t *w : {a.post_weight, a.post_bias, a.weight, a.bias}) {
    if (!w) continue;
    in[n_in] = w;
    in_bytes[n_in++] = H * 2;
  }
  if (!aligned(x, 16) || !aligned(branch, 16) || !aligned(r, 16) ||
      !aligned(y, 16) || !aligned(q, 8) || !aligned(qs, 4))
    return W8A8_ERR_ALIGN;
  const Range rx = range_of(x, M * H * 2),
              rb = range_of(branch, branch ? M * H * 2 : 0);
  const Range out[4] = {range_of(r, r ? M * H * 2 : 0),
                        range_of(y, y ? M * H * 2 : 0),
                        range_of(q, q ? M * H : 0),
                        range_of(qs, qs ? M * 4 : 0)};
  for (int i = 0; i < 4; ++i) {
    if (!(i == 0 && r == x) && overlap(out[i], rx)) return W8A8_ERR_ALIAS;
    if (overlap(out[i], rb)) return W8A8_ERR_ALIAS;
    for (int j = 0; j < n_in; ++j)
      if (overlap(out[i], range_of(in[j], in_bytes[j])))
        return W8A8_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return W8A8_ERR_ALIAS;
  }
  if ((st = check_device()) != W8A8_OK) return st;
  a.x = x;
  a.branch = branch;
  a.r = r;
  a.y = y;
  a.q = q;
  a.qs = qs;
  a.M = M;
  a.H = (int)H;
  a.residual_scale = residual_scale;
  return hip_status(
      w8a8::launch_norm(a, static_cast<hipStream_t>(stream)));
}

// Shape and group of a packed 4-bit weight.
int validate_w4(int64_t N, int64_t K, int64_t group) {
  if (N < 16 || N % 16 != 0 || N >= (int64_t(1) << 26) || K < 128 ||
      K % 128 != 0 || K > W8A8_MAX_K || N * K >= (int64_t(1) << 37))
    return W8A8_ERR_SHAPE;
  if (group != 32 && group != 64 && group != 128) return W8A8_ERR_ARG;
  return W8A8_OK;
}

// Rows of `width` elements at a stride (both in 2-byte elements).
struct Rows {
  const void *p;
  int64_t rows, width, stride;
};

Range range_of(const Rows &r) {
  return range_of(r.p, r.p ? ((r.rows - 1) * r.stride + r.width) * 2 : 0);
}

// Whether two sets of rows share an element: they do not where their spans are
// apart, or where they lie at one stride and the parts of a row are apart.
bool overlap(const Rows &a, const Rows &b) {
  const Range ra = range_of(a), rb = range_of(b);
  if (!overlap(ra, rb)) return false;
  if (a.stride != b.stride || (a.rows == 1 && b.rows == 1)) return true;
  const int64_t step = a.stride * 2;
  int64_t ahead = ((int64_t)rb.lo - (int64_t)ra.lo) % step;
  if (ahead < 0) ahead += step;
  return ahead < a.width * 2 || step - ahead < b.width * 2;
}

bool stride_ok(int64_t stride, int64_t width, int64_t limit) {
  return stride >= width && stride % 8 == 0 && stride < limit;
}

// One side of the head norms.
int validate_heads(const w8a8_heads_t *h, int64_t M, int64_t D) {
  if (!h->x || !h->y) return W8A8_ERR_NULL;
  if (h->heads < 1 || h->heads > 4096 || M * h->heads * D >= int64_t(1) << 36)
    return W8A8_ERR_SHAPE;
  if (!stride_ok(h->x_stride, h->heads * D, kMaxModStride) ||
      !stride_ok(h->y_stride, h->heads * D, kMaxModStride))
    return W8A8_ERR_SHAPE;
  const int st = validate_norm(&h->norm);
  if (st != W8A8_OK) return st;
  return aligned(h->x, 16) && aligned(h->y, 16) ? W8A8_OK : W8A8_ERR_ALIGN;
}

bool positive(double v) { return v > 0 && std::isfinite(v); }

// Everything of an attention call but its workspace and device; `args` and
// `plan` are filled in.
int validate_attention(const w8a8_attention_t *a, w8a8::AttnArgs *args,
                       w8a8::AttnPlan *plan) {
  const int64_t most = int64_t(1) << 31;
  if (!a) return W8A8_ERR_NULL;
  if (a->B < 1 || a->B > 1 << 20 || a->Tq < 1 || a->Tk < 0 || a->D < 8 ||
      a->D > 128 || a->D % 8 != 0 || a->q_heads < 1 || a->k_heads < 1 ||
      a->q_heads >= most || a->q_heads % a->k_heads != 0 || a->Tq >= most ||
      a->Tk >= most || a->Tq * a->q_heads >= most ||
      a->Tk * a->k_heads >= most)
    return W8A8_ERR_SHAPE;
  if ((!a->q_offsets && a->Tq % a->B != 0) ||
      (!a->k_offsets && a->Tk % a->B != 0))
    return W8A8_ERR_SHAPE;
  const int64_t wq = a->q_heads * a->D, wk = a->k_heads * a->D;
  const int64_t limit = int64_t(1) << 22;
  if (!stride_ok(a->q_stride, wq, limit) ||
      !stride_ok(a->out_stride, wq, limit) ||
      !stride_ok(a->k_stride, wk, limit) || !stride_ok(a->v_stride, wk, limit))
    return W8A8_ERR_SHAPE;
  const float scale_log2 = (float)(a->scale * 1.44269504088896340736);
  if (!(a->scale > 0) || !std::isfinite(scale_log2)) return W8A8_ERR_ARG;
  *plan = w8a8::plan_attention(a->Tq, a->Tk, a->B, a->q_offsets != nullptr,
                               a->q_heads, a->k_heads, a->D);
  if (!w8a8::attention_launchable(*plan, a->k_heads)) return W8A8_ERR_SHAPE;
  *args = w8a8::AttnArgs{
      a->q,        a->k,        a->v,      a->out,
      a->q_stride, a->k_stride, a->v_stride, a->out_stride,
      a->q_offsets, a->k_offsets, a->k_lens,
      (int)a->Tq,  (int)a->Tk,  (int)a->B, (int)a->q_heads,
      (int)a->k_heads, (int)a->D,
      scale_log2, nullptr,
      (int)(a->q_heads / a->k_heads)};
  return W8A8_OK;
}

}  // namespace

extern "C" {

const char *w8a8_status_string(int status) {
  switch (status) {
    case W8A8_OK: return "ok";
    case W8A8_ERR_NULL: return "a required pointer is NULL";
    case W8A8_ERR_SHAPE: return "a size violates the shape contract";
    case W8A8_ERR_ALIGN: return "a pointer is not aligned as required";
    case W8A8_ERR_WORKSPACE: return "workspace missing or too small";
    case W8A8_ERR_OUT_DTYPE: return "unknown output type";
    case W8A8_ERR_ALIAS: return "an output overlaps another buffer";
    case W8A8_ERR_DEVICE: return "no HIP device, or it is not gfx950";
    case W8A8_ERR_HIP: return "a HIP call or kernel launch failed";
    case W8A8_ERR_ARG: return "an option is unknown or out of range";
    default: return "unknown status";
  }
}

int w8a8_last_hip_error(void) { return g_last_hip_error; }

#ifndef W8A8_SOURCE_SHA256
#define W8A8_SOURCE_SHA256 "unknown"
#endif
const char *w8a8_build_id(void) { return W8A8_SOURCE_SHA256; }

size_t w8a8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (!gemm_shape_ok(M, N, K)) return 0;
  return w8a8::plan_gemm(M, N, K).workspace;
}

size_t w8a8_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (!gemm_shape_ok(M, N, K) || M > kMaxTokenRows) return 0;
  return round_up((size_t)(M * K), 256) + round_up((size_t)M * 4, 256) +
         w8a8::plan_gemm(M, N, K).workspace;
}

int w8a8_quantize_act(const uint16_t *x, int64_t M, int64_t K, int8_t *a_q,
                      float *a_scale, void *stream) {
  int st = validate_quant(x, M, K, a_q, a_scale);
  if (st != W8A8_OK) return st;
  if ((st = check_device()) != W8A8_OK) return st;
  return hip_status(w8a8::launch_quantize_act(
      x, a_q, a_scale, M, K, false, static_cast<hipStream_t>(stream)));
}

int w8a8_quantize_act_silu(const uint16_t *x, int64_t M, int64_t K,
                           int8_t *a_q, float *a_scale, void *stream) {
  int st = validate_quant(x, M, K, a_q, a_scale, kGlueMaxK);
  if (st != W8A8_OK) return st;
  if ((st = check_device()) != W8A8_OK) return st;
  return hip_status(w8a8::launch_quantize_act(
      x, a_q, a_scale, M, K, true, static_cast<hipStream_t>(stream)));
}

int w8a8_gemm(const int8_t *a_q, const float *a_scale, const int8_t *w_q,
              const float *w_scale, const uint16_t *bias, void *out,
              int out_dtype, int64_t M, int64_t N, int64_t K,
              void *workspace, size_t workspace_bytes, void *stream) {
  GemmPlan plan;
  int st = validate_gemm(a_q, a_scale, w_q, w_scale, bias, out, out_dtype, M,
                         N, K, workspace, workspace_bytes, &plan);
  if (st != W8A8_OK) return st;
  if ((st = check_device()) != W8A8_OK) return st;
  GemmArgs g{a_q, a_scale, w_q, w_scale, bias, out, out_dtype,
             M,   N,       K,   workspace, workspace_bytes};
  return hip_status(
      w8a8::launch_gemm(g, plan, static_cast<hipStream_t>(stream)));
}

int w8a8_gemm_noalloc(const int8_t *a_q, const float *a_scale,
                      const int8_t *w_q, const float *w_scale,
                      const uint16_t *bias, void *out, int out_dtype,
                      int64_t M, int64_t N, int64_t K, void *stream) {
  // As w8a8_gemm, with the split-K partial sums in the library's own device
  // scratch (one copy per GPU) instead of a caller's workspace: nothing is
  // allocated here.  A plan needing more than the scratch is refused (the
  // planner's bound on partial sums makes that impossible today).
  GemmPlan plan;
  int st = validate_gemm_args(a_q, a_scale, w_q, w_scale, bias, out,
                              out_dtype, M, N, K, &plan);
  if (st != W8A8_OK) return st;
  if (plan.workspace > w8a8::kScratchBytes) return W8A8_ERR_WORKSPACE;
  if ((st = check_device()) != W8A8_OK) return st;
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess) return W8A8_ERR_DEVICE;
  void *scratch = w8a8::scratch_on_device(dev);
  if (scratch == nullptr) {  // set-up failed at the device check: retry
    st = hip_status(w8a8::resolve_scratch(dev));
    if (st != W8A8_OK) return st;
    scratch = w8a8::scratch_on_device(dev);
  }
  st = scratch_alias(scratch, plan, a_q, a_scale, w_q, w_scale, bias, out,
                     out_dtype, M, N, K);
  if (st != W8A8_OK) return st;
  GemmArgs g{a_q, a_scale, w_q, w_scale, bias, out, out_dtype,
             M,   N,       K,   scratch, w8a8::kScratchBytes};
  return hip_status(
      w8a8::launch_gemm(g, plan, static_cast<hipStream_t>(stream)));
}

int w8a8_linear(const uint16_t *x, const int8_t *w_q, const float *w_scale,
                const uint16_t *bias, uint16_t *y, int64_t M, int64_t N,
                int64_t K, void *workspace, size_t workspace_bytes,
                void *stream) {
  if (!x || !w_q || !w_scale || !y) return W8A8_ERR_NULL;
  if (!gemm_shape_ok(M, N, K) || K > kQuantMaxK || M > kMaxTokenRows)
    return W8A8_ERR_SHAPE;
  if (!aligned(x, 16)) return W8A8_ERR_ALIGN;
  const size_t need = w8a8_workspace_bytes(M, N, K);
  if (!workspace || workspace_bytes < need) return W8A8_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return W8A8_ERR_ALIGN;
  int8_t *aq = static_cast<int8_t *>(workspace);
  float *sa = reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                        round_up((size_t)(M * K), 256));
  void *gws = static_cast<char *>(workspace) + round_up((size_t)(M * K), 256) +
              round_up((size_t)M * 4, 256);
  const size_t gws_bytes = workspace_bytes - (need - w8a8::plan_gemm(M, N, K).workspace);
  // The workspace and y must stay clear of the inputs.
  const Range rws = range_of(workspace, (int64_t)need);
  const Range ry = range_of(y, M * N * 2);
  const Range ins[] = {range_of(x, M * K * 2), range_of(w_q, N * K),
                       range_of(w_scale, N * 4),
                       range_of(bias, bias ? N * 2 : 0)};
  for (const Range &r : ins)
    if (overlap(rws, r) || overlap(ry, r)) return W8A8_ERR_ALIAS;
  if (overlap(rws, ry)) return W8A8_ERR_ALIAS;
  GemmPlan plan;
  int st = validate_gemm(aq, sa, w_q, w_scale, bias, y, W8A8_OUT_BF16, M, N, K,
                         gws, gws_bytes, &plan);
  if (st != W8A8_OK) return st;
  if ((st = check_device()) != W8A8_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  st = hip_status(w8a8::launch_quantize_act(x, aq, sa, M, K, false, s));
  if (st != W8A8_OK) return st;
  GemmArgs g{aq, sa, w_q, w_scale, bias, y, W8A8_OUT_BF16,
             M,  N,  K,   gws,     gws_bytes};
  return hip_status(w8a8::launch_gemm(g, plan, s));
}

int w8a8_quantize_weight(const uint16_t *w, int64_t N, int64_t K,
                         int8_t *w_q, float *w_scale, void *stream) {
  int st = validate_quant(w, N, K, w_q, w_scale);
  if (st != W8A8_OK) return st;
  if ((st = check_device()) != W8A8_OK) return st;
  return hip_status(w8a8::launch_quantize_weight(
      w, w_q, w_scale, N, K, static_cast<hipStream_t>(stream)));
}

int w8a8_check_scales(const float *w_scale, int64_t N, int32_t *bad_count,
                      void *stream) {
  if (!w_scale || !bad_count) return W8A8_ERR_NULL;
  if (N < 0 || N > kMaxRows) return W8A8_ERR_SHAPE;
  if (!aligned(w_scale, 4) || !aligned(bad_count, 4)) return W8A8_ERR_ALIGN;
  if (overlap(range_of(w_scale, N * 4), range_of(bad_count, 4)))
    return W8A8_ERR_ALIAS;
  int st = check_device();
  if (st != W8A8_OK) return st;
  return hip_status(w8a8::launch_check_scales(
      w_scale, N, bad_count, static_cast<hipStream_t>(stream)));
}

int w8a8_swiglu_bf16(const uint16_t *h, uint16_t *y, int64_t M, int64_t F,
                     void *stream) {
  if (!h || !y) return W8A8_ERR_NULL;
  if (M < 1 || M > kMaxTokenRows || F < 8 || F % 8 != 0 || F > kMaxRows / 2)
    return W8A8_ERR_SHAPE;
  if (!aligned(h, 16) || !aligned(y, 16)) return W8A8_ERR_ALIGN;
  if (overlap(range_of(h, M * F * 4), range_of(y, M * F * 2)))
    return W8A8_ERR_ALIAS;
  int st = check_device();
  if (st != W8A8_OK) return st;
  return hip_status(
      w8a8::launch_swiglu(h, y, M, F, static_cast<hipStream_t>(stream)));
}

int w8a8_quantize_act_swiglu(const uint16_t *h, int64_t M, int64_t F,
                             int8_t *a_q, float *a_scale, void *stream) {
  if (!h || !a_q || !a_scale) return W8A8_ERR_NULL;
  if (M < 1 || M > kMaxTokenRows || F < 8 || F % 8 != 0 || F > kGlueMaxK)
    return W8A8_ERR_SHAPE;
  if (!aligned(h, 16) || !aligned(a_q, 8) || !aligned(a_scale, 4))
    return W8A8_ERR_ALIGN;
  const Range rh = range_of(h, M * F * 4), rq = range_of(a_q, M * F),
              rs = range_of(a_scale, M * 4);
  if (overlap(rh, rq) || overlap(rh, rs) || overlap(rq, rs))
    return W8A8_ERR_ALIAS;
  int st = check_device();
  if (st != W8A8_OK) return st;
  return hip_status(w8a8::launch_swiglu_quant(
      h, a_q, a_scale, M, F, static_cast<hipStream_t>(stream)));
}

int w8a8_silu_bf16(const uint16_t *x, uint16_t *y, int64_t n, void *stream) {
  if (!x || !y) return W8A8_ERR_NULL;
  if (n < 0 || n % 8 != 0) return W8A8_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(y, 16)) return W8A8_ERR_ALIGN;
  if (x != y && overlap(range_of(x, n * 2), range_of(y, n * 2)))
    return W8A8_ERR_ALIAS;
  int st = check_device();
  if (st != W8A8_OK) return st;
  return hip_status(
      w8a8::launch_silu(x, y, n, static_cast<hipStream_t>(stream)));
}

int w8a8_pow2_renorm(const uint16_t *x, uint16_t *y, int64_t M, int64_t K,
                     void *stream) {
  if (!x || !y) return W8A8_ERR_NULL;
  if (M < 1 || M > kMaxTokenRows || K < 8 || K % 8 != 0 || K > kGlueMaxK)
    return W8A8_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(y, 16)) return W8A8_ERR_ALIGN;
  if (x != y && overlap(range_of(x, M * K * 2), range_of(y, M * K * 2)))
    return W8A8_ERR_ALIAS;
  int st = check_device();
  if (st != W8A8_OK) return st;
  return hip_status(w8a8::launch_pow2_renorm(x, y, M, K,
                                              static_cast<hipStream_t>(stream)));
}

int w8a8_pow2_renorm_quantize(const uint16_t *x, int64_t M, int64_t K,
                              uint16_t *y, int8_t *a_q, float *a_scale,
                              void *stream) {
  if (!x || !y || !a_q || !a_scale) return W8A8_ERR_NULL;
  if (M < 1 || M > kMaxTokenRows || K < 8 || K % 8 != 0 || K > kGlueMaxK)
    return W8A8_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(a_q, 8) ||
      !aligned(a_scale, 4))
    return W8A8_ERR_ALIGN;
  const Range rx = range_of(x, M * K * 2), ry = range_of(y, M * K * 2),
              rq = range_of(a_q, M * K), rs = range_of(a_scale, M * 4);
  if ((x != y && overlap(rx, ry)) || overlap(rx, rq) || overlap(rx, rs) ||
      overlap(ry, rq) || overlap(ry, rs) || overlap(rq, rs))
    return W8A8_ERR_ALIAS;
  int st = check_device();
  if (st != W8A8_OK) return st;
  return hip_status(w8a8::launch_pow2_renorm_quant(
      x, y, a_q, a_scale, M, K, static_cast<hipStream_t>(stream)));
}

int w8a8_norm_modulate(const uint16_t *x, int64_t M, int64_t H,
                       const w8a8_norm_t *pre, const w8a8_modulation_t *mod,
                       uint16_t *y, void *stream) {
  if (!x || !y) return W8A8_ERR_NULL;
  return block_norm(x, nullptr, M, H, nullptr, pre, mod, 1.0f, nullptr, y,
                    nullptr, nullptr, stream);
}

int w8a8_norm_modulate_quantize(const uint16_t *x, int64_t M, int64_t H,
                                const w8a8_norm_t *pre,
                                const w8a8_modulation_t *mod, int8_t *a_q,
                                float *a_scale, void *stream) {
  if (!x || !a_q || !a_scale) return W8A8_ERR_NULL;
  return block_norm(x, nullptr, M, H, nullptr, pre, mod, 1.0f, nullptr,
                    nullptr, a_q, a_scale, stream);
}

int w8a8_gated_residual(const uint16_t *x, const uint16_t *branch, int64_t M,
                        int64_t H, const w8a8_norm_t *post,
                        const w8a8_modulation_t *mod, float residual_scale,
                        uint16_t *r, void *stream) {
  if (!x || !branch || !r) return W8A8_ERR_NULL;
  return block_norm(x, branch, M, H, post, nullptr, mod, residual_scale, r,
                    nullptr, nullptr, nullptr, stream);
}

int w8a8_gated_residual_norm(const uint16_t *x, const uint16_t *branch,
                             int64_t M, int64_t H, const w8a8_norm_t *post,
                             const w8a8_norm_t *pre,
                             const w8a8_modulation_t *mod,
                             float residual_scale, uint16_t *r, uint16_t *y,
                             void *stream) {
  if (!x || !branch || !r || !y) return W8A8_ERR_NULL;
  return block_norm(x, branch, M, H, post, pre, mod, residual_scale, r, y,
                    nullptr, nullptr, stream);
}

int w8a8_gated_residual_norm_quantize(
    const uint16_t *x, const uint16_t *branch, int64_t M, int64_t H,
    const w8a8_norm_t *post, const w8a8_norm_t *pre,
    const w8a8_modulation_t *mod, float residual_scale, uint16_t *r,
    int8_t *a_q, float *a_scale, void *stream) {
  if (!x || !branch || !r || !a_q || !a_scale) return W8A8_ERR_NULL;
  return block_norm(x, branch, M, H, post, pre, mod, residual_scale, r,
                    nullptr, a_q, a_scale, stream);
}

int w8a8_w4_quantize_weight(const uint16_t *w, int64_t N, int64_t K,
                            int64_t group, uint8_t *w4, uint16_t *w4_scale,
                            void *stream) {
  if (!w || !w4 || !w4_scale) return W8A8_ERR_NULL;
  int st = validate_w4(N, K, group);
  if (st != W8A8_OK) return st;
  if (!aligned(w, 16) || !aligned(w4, 16) || !aligned(w4_scale, 16))
    return W8A8_ERR_ALIGN;
  const Range rw = range_of(w, N * K * 2), rq = range_of(w4, N * K / 2),
              rs = range_of(w4_scale, N * K / group * 2);
  if (overlap(rw, rq) || overlap(rw, rs) || overlap(rq, rs))
    return W8A8_ERR_ALIAS;
  if ((st = check_device()) != W8A8_OK) return st;
  return hip_status(w8a8::launch_w4_quantize(
      w, N, K, (int)group, w4, w4_scale, static_cast<hipStream_t>(stream)));
}

int w8a8_w4_pack_weight(const int8_t *codes, const uint16_t *scales,
                        int64_t N, int64_t K, int64_t group, uint8_t *w4,
                        uint16_t *w4_scale, void *stream) {
  if (!codes || !scales || !w4 || !w4_scale) return W8A8_ERR_NULL;
  int st = validate_w4(N, K, group);
  if (st != W8A8_OK) return st;
  if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(w4, 16) ||
      !aligned(w4_scale, 16))
    return W8A8_ERR_ALIGN;
  const int64_t sb = N * K / group * 2;
  const Range rc = range_of(codes, N * K), rs = range_of(scales, sb),
              rq = range_of(w4, N * K / 2), ro = range_of(w4_scale, sb);
  if (overlap(rc, rq) || overlap(rc, ro) || overlap(rs, rq) ||
      overlap(rs, ro) || overlap(rq, ro))
    return W8A8_ERR_ALIAS;
  if ((st = check_device()) != W8A8_OK) return st;
  return hip_status(
      w8a8::launch_w4_pack(codes, scales, N, K, (int)group, w4, w4_scale,
                           static_cast<hipStream_t>(stream)));
}

int w8a8_w4_linear(const uint16_t *x, const uint8_t *w4,
                   const uint16_t *w4_scale, const uint16_t *bias,
                   uint16_t *y, int64_t M, int64_t N, int64_t K,
                   int64_t group, void *stream) {
  if (!x || !w4 || !w4_scale || !y) return W8A8_ERR_NULL;
  if (M < 1 || M > 32 * 65535) return W8A8_ERR_SHAPE;
  int st = validate_w4(N, K, group);
  if (st != W8A8_OK) return st;
  if (!aligned(x, 16) || !aligned(w4, 16) || !aligned(w4_scale, 16) ||
      !aligned(y, 16) || !aligned(bias, 2))
    return W8A8_ERR_ALIGN;
  const Range ry = range_of(y, M * N * 2);
  const Range ins[] = {range_of(x, M * K * 2), range_of(w4, N * K / 2),
                       range_of(w4_scale, N * K / group * 2),
                       range_of(bias, bias ? N * 2 : 0)};
  for (const Range &r : ins)
    if (overlap(ry, r)) return W8A8_ERR_ALIAS;
  if ((st = check_device()) != W8A8_OK) return st;
  return hip_status(w8a8::launch_w4_linear(
      x, w4, w4_scale, bias, y, M, N, K, (int)group,
      static_cast<hipStream_t>(stream)));
}

int w8a8_rope_table(const void *positions, int position_type, int64_t T,
                    const w8a8_rope_t *rope, float *table, void *stream) {
  if (!positions || !rope || !table) return W8A8_ERR_NULL;
  if (T < 1 || T > kMaxTokenRows || rope->axes < 1 ||
      rope->axes > W8A8_ROPE_MAX_AXES)
    return W8A8_ERR_SHAPE;
  int64_t pairs = 0;
  for (int i = 0; i < rope->axes; ++i) {
    if (rope->pairs[i] < 1) return W8A8_ERR_SHAPE;
    pairs += rope->pairs[i];
  }
  if (pairs > W8A8_ROPE_MAX_PAIRS) return W8A8_ERR_SHAPE;
  if (position_type != W8A8_POSITIONS_I32 &&
      position_type != W8A8_POSITIONS_F32)
    return W8A8_ERR_ARG;
  const int how = rope->scaling;
  if (how < W8A8_ROPE_NONE || how > W8A8_ROPE_YARN ||
      !positive(rope->theta) || rope->theta <= 1 ||
      !std::isfinite((float)rope->amplitude))
    return W8A8_ERR_ARG;
  if (how != W8A8_ROPE_NONE && (!positive(rope->factor) || rope->factor < 1))
    return W8A8_ERR_ARG;
  if (how == W8A8_ROPE_NTK)
    for (int i = 0; i < rope->axes; ++i)
      if (!positive((double)w8a8::ntk_theta(*rope, rope->pairs[i])))
        return W8A8_ERR_ARG;
  if (how == W8A8_ROPE_YARN &&
      (!positive(rope->original) || !positive(rope->beta_fast) ||
       !positive(rope->beta_slow)))
    return W8A8_ERR_ARG;
  if (!aligned(positions, 4) || !aligned(table, 16)) return W8A8_ERR_ALIGN;
  if (overlap(range_of(positions, T * rope->axes * 4),
              range_of(table, T * pairs * 8)))
    return W8A8_ERR_ALIAS;
  int st = check_device();
  if (st != W8A8_OK) return st;
  w8a8::RopeArgs a{};
  a.pos = positions;
  a.table = table;
  a.T = T;
  a.pos_type = position_type;
  a.axes = rope->axes;
  a.pairs = (int)pairs;
  a.amplitude = (float)rope->amplitude;
  int at = 0;
  for (int x = 0; x < rope->axes; at += rope->pairs[x++]) {
    w8a8::rope_quarters(*rope, rope->pairs[x], a.quarters + at);
    for (int i = 0; i < rope->pairs[x]; ++i) a.axis[at + i] = (uint8_t)x;
  }
  return hip_status(
      w8a8::launch_rope_table(a, static_cast<hipStream_t>(stream)));
}

int w8a8_head_norm_rope(const w8a8_heads_t *q, const w8a8_heads_t *k,
                        int64_t M, int64_t D, const float *table,
                        int64_t pairs, int64_t rows, const int32_t *row,
                        int interleaved, void *stream) {
  if (!q) return W8A8_ERR_NULL;
  if (M < 1 || M > kMaxTokenRows || D < 8 || D > 256 || D % 8 != 0)
    return W8A8_ERR_SHAPE;
  if (table) {
    if (pairs < 4 || pairs % 4 != 0 || 2 * pairs > D || rows < 1 ||
        rows > kMaxRows || (!row && rows != 1 && rows != M))
      return W8A8_ERR_SHAPE;
    if (!aligned(table, 16) || !aligned(row, 4)) return W8A8_ERR_ALIGN;
  }
  const w8a8_heads_t *sides[2] = {q, k};
  w8a8::HeadArgs a{};
  Rows in[2], out[2];
  int n = 0;
  for (const w8a8_heads_t *h : sides) {
    if (!h) continue;
    const int st = validate_heads(h, M, D);
    if (st != W8A8_OK) return st;
    a.side[n] = w8a8::HeadSide{h->x, h->y, h->norm.weight, h->norm.bias,
                               h->x_stride, h->y_stride, (int)h->heads,
                               h->norm.kind, h->per_head ? (int)D : 0,
                               h->norm.eps};
    in[n] = Rows{h->x, M, h->heads * D, h->x_stride};
    out[n++] = Rows{h->y, M, h->heads * D, h->y_stride};
  }
  for (int i = 0; i < n; ++i) {
    for (int j = 0; j < n; ++j) {
      const bool same = i == j && out[i].p == in[j].p &&
                        out[i].stride == in[j].stride;
      if (!same && overlap(out[i], in[j])) return W8A8_ERR_ALIAS;
      if (j < i && overlap(out[i], out[j])) return W8A8_ERR_ALIAS;
      const int64_t vec = (sides[j]->per_head ? sides[j]->heads : 1) * D * 2;
      const Range ro = range_of(out[i]);
      for (const uint16_t *p : {a.side[j].weight, a.side[j].bias})
        if (p && overlap(ro, range_of(p, vec))) return W8A8_ERR_ALIAS;
    }
    if (table &&
        (overlap(range_of(out[i]), range_of(table, rows * pairs * 8)) ||
         overlap(range_of(out[i]), range_of(row, row ? M * 4 : 0))))
      return W8A8_ERR_ALIAS;
  }
  if (table) {
    a.table = table;
    a.row = row;
    a.rows = (int)rows;
    a.row_step = rows > 1 ? 1 : 0;
    a.pairs = (int)pairs;
    a.interleaved = interleaved != 0;
  } else {
    a.rows = 1;
  }
  a.M = M;
  a.D = (int)D;
  if (w8a8::head_norm_items(a) >= int64_t(1) << 32) return W8A8_ERR_SHAPE;
  const int st = check_device();
  if (st != W8A8_OK) return st;
  return hip_status(
      w8a8::launch_head_norm(a, static_cast<hipStream_t>(stream)));
}

size_t w8a8_attention_workspace_bytes(const w8a8_attention_t *a) {
  w8a8::AttnArgs args;
  w8a8::AttnPlan plan;
  return validate_attention(a, &args, &plan) == W8A8_OK ? plan.workspace : 0;
}

int w8a8_attention(const w8a8_attention_t *a, void *workspace,
                   size_t workspace_bytes, void *stream) {
  if (!a || !a->q || !a->out || (a->Tk > 0 && (!a->k || !a->v)))
    return W8A8_ERR_NULL;
  w8a8::AttnArgs args;
  w8a8::AttnPlan plan;
  int st = validate_attention(a, &args, &plan);
  if (st != W8A8_OK) return st;
  if (!aligned(a->q, 16) || !aligned(a->k, 16) || !aligned(a->v, 16) ||
      !aligned(a->out, 16) || !aligned(a->q_offsets, 4) ||
      !aligned(a->k_offsets, 4) || !aligned(a->k_lens, 4))
    return W8A8_ERR_ALIGN;
  const int64_t wq = a->q_heads * a->D, wk = a->k_heads * a->D;
  const Rows out = {a->out, a->Tq, wq, a->out_stride};
  const Rows ins[] = {{a->q, a->Tq, wq, a->q_stride},
                      {a->Tk ? a->k : nullptr, a->Tk, wk, a->k_stride},
                      {a->Tk ? a->v : nullptr, a->Tk, wk, a->v_stride}};
  const Range lists[] = {
      range_of(a->q_offsets, a->q_offsets ? (a->B + 1) * 4 : 0),
      range_of(a->k_offsets, a->k_offsets ? (a->B + 1) * 4 : 0),
      range_of(a->k_lens, a->k_lens ? a->B * 4 : 0)};
  for (const Rows &r : ins)
    if (overlap(out, r)) return W8A8_ERR_ALIAS;
  for (const Range &r : lists)
    if (overlap(range_of(out), r)) return W8A8_ERR_ALIAS;
  if (plan.workspace > 0) {
    if (!workspace || workspace_bytes < plan.workspace)
      return W8A8_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return W8A8_ERR_ALIGN;
    const Range rw = range_of(workspace, (int64_t)plan.workspace);
    if (overlap(rw, range_of(out))) return W8A8_ERR_ALIAS;
    for (const Rows &r : ins)
      if (overlap(rw, range_of(r))) return W8A8_ERR_ALIAS;
    for (const Range &r : lists)
      if (overlap(rw, r)) return W8A8_ERR_ALIAS;
    args.workspace = workspace;
  }
  if ((st = check_device()) != W8A8_OK) return st;
  return hip_status(w8a8::launch_attention(args, plan,
                                           static_cast<hipStream_t>(stream)));
}

}  // extern "C"
