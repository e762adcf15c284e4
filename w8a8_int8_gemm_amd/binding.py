"""Python binding of libw8a8.so (include/w8a8.h): argument marshalling only.

Torch tensors supply device memory and the current HIP stream; every step
of the computation runs in the library's HIP kernels.  Loading fails loudly
when the shared object is missing: there is no CPU or PyTorch fallback.

BF16 tensors are passed as their bit patterns (the library's uint16 BF16).
"""
from __future__ import annotations

import ctypes
import math
from pathlib import Path

PKG = Path(__file__).resolve().parent
LIB_PATH = PKG / "libw8a8.so"

OUT_BF16, OUT_FP32, OUT_I32 = 0, 1, 2
W8A8_OK = 0
W8A8_ERR_WORKSPACE = 4
STATUS = {
    0: "W8A8_OK", 1: "W8A8_ERR_NULL", 2: "W8A8_ERR_SHAPE",
    3: "W8A8_ERR_ALIGN", 4: "W8A8_ERR_WORKSPACE", 5: "W8A8_ERR_OUT_DTYPE",
    6: "W8A8_ERR_ALIAS", 7: "W8A8_ERR_DEVICE", 8: "W8A8_ERR_HIP",
    9: "W8A8_ERR_ARG",
}
MAX_K = 130944
GLUE_MAX_K = 90112   # SiLU, renormalization and the fused quantizers
NORM_MAX_H = 32768   # block norms
NORM_KINDS = {"none": 0, "rms": 1, "layer": 2}
W4_GROUPS = (32, 64, 128)
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}
ROPE_MAX_AXES = 4
ROPE_MAX_PAIRS = 256


class _Norm(ctypes.Structure):  # w8a8_norm_t
    _fields_ = [("kind", ctypes.c_int), ("eps", ctypes.c_float),
                ("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p)]


class _Modulation(ctypes.Structure):  # w8a8_modulation_t
    _fields_ = [("scale", ctypes.c_void_p), ("shift", ctypes.c_void_p),
                ("gate", ctypes.c_void_p), ("scale_stride", ctypes.c_int64),
                ("shift_stride", ctypes.c_int64),
                ("gate_stride", ctypes.c_int64), ("rows", ctypes.c_int64),
                ("row", ctypes.c_void_p)]


class _Rope(ctypes.Structure):  # w8a8_rope_t
    _fields_ = [("axes", ctypes.c_int), ("pairs", ctypes.c_int * 4),
                ("scaling", ctypes.c_int), ("theta", ctypes.c_double),
                ("factor", ctypes.c_double), ("original", ctypes.c_double),
                ("beta_fast", ctypes.c_double),
                ("beta_slow", ctypes.c_double),
                ("amplitude", ctypes.c_double)]


class _Heads(ctypes.Structure):  # w8a8_heads_t
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("heads", ctypes.c_int64), ("x_stride", ctypes.c_int64),
                ("y_stride", ctypes.c_int64), ("norm", _Norm),
                ("per_head", ctypes.c_int)]


class _Attention(ctypes.Structure):  # w8a8_attention_t
    _fields_ = ([(n, ctypes.c_void_p) for n in ("q", "k", "v", "out")] +
                [(n, ctypes.c_int64) for n in (
                    "q_stride", "k_stride", "v_stride", "out_stride", "Tq",
                    "Tk", "B", "q_heads", "k_heads", "D")] +
                [(n, ctypes.c_void_p) for n in (
                    "q_offsets", "k_offsets", "k_lens")] +
                [("scale", ctypes.c_float)])


# Every symbol include/w8a8.h declares, with its ctypes signature.
_P, _I64, _SZ, _I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
_F = ctypes.c_float
_PN, _PM = ctypes.POINTER(_Norm), ctypes.POINTER(_Modulation)
_PH, _PA = ctypes.POINTER(_Heads), ctypes.POINTER(_Attention)
SIGNATURES = {
    "w8a8_quantize_act": (_I, [_P, _I64, _I64, _P, _P, _P]),
    "w8a8_quantize_act_silu": (_I, [_P, _I64, _I64, _P, _P, _P]),
    "w8a8_gemm": (_I, [_P, _P, _P, _P, _P, _P, _I, _I64, _I64, _I64, _P,
                       _SZ, _P]),
    "w8a8_linear": (_I, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _P, _SZ,
                         _P]),
    "w8a8_gemm_noalloc": (_I, [_P, _P, _P, _P, _P, _P, _I, _I64, _I64,
                               _I64, _P]),
    "w8a8_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "w8a8_gemm_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "w8a8_status_string": (ctypes.c_char_p, [_I]),
    "w8a8_last_hip_error": (_I, []),
    "w8a8_build_id": (ctypes.c_char_p, []),
    "w8a8_silu_bf16": (_I, [_P, _P, _I64, _P]),
    "w8a8_pow2_renorm": (_I, [_P, _P, _I64, _I64, _P]),
    "w8a8_pow2_renorm_quantize": (_I, [_P, _I64, _I64, _P, _P, _P, _P]),
    "w8a8_quantize_weight": (_I, [_P, _I64, _I64, _P, _P, _P]),
    "w8a8_check_scales": (_I, [_P, _I64, _P, _P]),
    "w8a8_swiglu_bf16": (_I, [_P, _P, _I64, _I64, _P]),
    "w8a8_quantize_act_swiglu": (_I, [_P, _I64, _I64, _P, _P, _P]),
    "w8a8_norm_modulate": (_I, [_P, _I64, _I64, _PN, _PM, _P, _P]),
    "w8a8_norm_modulate_quantize": (_I, [_P, _I64, _I64, _PN, _PM, _P, _P,
                                         _P]),
    "w8a8_gated_residual": (_I, [_P, _P, _I64, _I64, _PN, _PM, _F, _P, _P]),
    "w8a8_gated_residual_norm": (_I, [_P, _P, _I64, _I64, _PN, _PN, _PM, _F,
                                      _P, _P, _P]),
    "w8a8_gated_residual_norm_quantize": (_I, [_P, _P, _I64, _I64, _PN, _PN,
                                               _PM, _F, _P, _P, _P, _P]),
    "w8a8_w4_quantize_weight": (_I, [_P, _I64, _I64, _I64, _P, _P, _P]),
    "w8a8_w4_pack_weight": (_I, [_P, _P, _I64, _I64, _I64, _P, _P, _P]),
    "w8a8_w4_linear": (_I, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _P]),
    "w8a8_rope_table": (_I, [_P, _I, _I64, ctypes.POINTER(_Rope), _P, _P]),
    "w8a8_head_norm_rope": (_I, [_PH, _PH, _I64, _I64, _P, _I64, _I64, _P, _I,
                                 _P]),
    "w8a8_attention_workspace_bytes": (_SZ, [_PA]),
    "w8a8_attention": (_I, [_PA, _P, _SZ, _P]),
}


class W8A8Error(RuntimeError):
    def __init__(self, fn: str, status: int, detail: str = ""):
        self.status = status
        super().__init__(f"{fn}: {STATUS.get(status, status)} "
                         f"({lib().w8a8_status_string(status).decode()})"
                         f"{detail}")


_lib = None


def _load(path):
    # torch first: its ROCm build carries its own HIP runtime, and the
    # library must resolve its HIP symbols to that same runtime (found by
    # its soname once loaded).  Loaded before torch, the library would pull
    # in the system HIP runtime and torch would then load a second one; the
    # library's device calls then fail (no device is visible to it).
    import torch  # noqa: F401
    L = ctypes.CDLL(str(path))
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    return L


def _expected_build_id() -> str:
    from . import build as _build
    return _build.source_sha256()


def build_is_stale() -> bool:
    """True when the shared object is missing or was compiled from sources
    other than the ones beside it (read without keeping it loaded)."""
    if not LIB_PATH.exists():
        return True
    if _lib is not None:
        return _lib.w8a8_build_id().decode() != _expected_build_id()
    return _load(LIB_PATH).w8a8_build_id().decode() != _expected_build_id()


def lib():
    """The loaded shared object.  Raises if it has not been built, or if it
    was built from other sources than the ones in the tree (a stale build
    would run old kernels under new code)."""
    global _lib
    if _lib is None:
        if not LIB_PATH.exists():
            raise ImportError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m w8a8_int8_gemm_amd.build` (or "
                "__graft_entry__.build()); there is no fallback path")
        L = _load(LIB_PATH)
        got, want = L.w8a8_build_id().decode(), _expected_build_id()
        if got != want:
            raise ImportError(
                f"{LIB_PATH} was built from other sources (build id "
                f"{got[:12]}, sources {want[:12]}): rebuild it with "
                "`python -m w8a8_int8_gemm_amd.build`")
        _lib = L
    return _lib


def _check(fn: str, status: int):
    if status != W8A8_OK:
        detail = ""
        if status == 8:
            detail = f" hipError={lib().w8a8_last_hip_error()}"
        raise W8A8Error(fn, status, detail)


# ---------------------------------------------------------------------------
# torch-facing wrappers
# ---------------------------------------------------------------------------

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _stream(stream=None):
    """The handle of `stream`, or of the current GPU's current stream (read
    without building a stream object: a call's host time is a few such steps,
    and at a few tokens it is as long as the kernels)."""
    if stream is not None:
        return stream.cuda_stream
    c = _torch()._C
    return c._cuda_getCurrentRawStream(c._cuda_getDevice())


def _on_stream(stream, *tensors):
    """Tensors allocated here on torch's current stream but used by kernels
    enqueued on another `stream`: tell the caching allocator, so that it does
    not hand their memory to a later allocation on the current stream while
    those kernels may still read or write it."""
    if stream is None:
        return
    torch = _torch()
    if stream == torch.cuda.current_stream():
        return
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need(t, dtype, ndim, name, shape=None):
    """t must be a contiguous tensor of `dtype` with `ndim` dims (and, if
    given, exactly `shape`) on the current GPU: the C ABI takes bare
    pointers, so sizes and devices are checked here."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    size = t.shape
    if t.dtype != dtype or len(size) != ndim or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {dtype} with {ndim} "
                         f"dims, got {t.dtype} {tuple(size)}")
    if shape is not None and size != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got "
                         f"{tuple(size)}")
    _on_current_gpu(t, name)


def _on_current_gpu(t, name):
    torch = _torch()
    device = t.get_device()  # -1: not on a GPU
    if device < 0:
        raise ValueError(f"{name} must be on the GPU")
    if device != torch._C._cuda_getDevice():
        raise ValueError(f"{name} must be on the current GPU "
                         f"(cuda:{torch.cuda.current_device()})")


def quantize_act(x, *, silu: bool = False, out=None, stream=None):
    """x: bf16 [M,K] -> (a_q int8 [M,K], a_scale float32 [M]).
    silu=True applies SiLU (rounded to BF16) before quantizing."""
    torch = _torch()
    _need(x, torch.bfloat16, 2, "x")
    M, K = x.shape
    if out is None:
        q = torch.empty((M, K), dtype=torch.int8, device=x.device)
        s = torch.empty((M,), dtype=torch.float32, device=x.device)
    else:
        q, s = out
        _need(q, torch.int8, 2, "out[0]", (M, K))
        _need(s, torch.float32, 1, "out[1]", (M,))
    fn = lib().w8a8_quantize_act_silu if silu else lib().w8a8_quantize_act
    _check("w8a8_quantize_act" + ("_silu" if silu else ""),
           fn(_ptr(x), M, K, _ptr(q), _ptr(s), _stream(stream)))
    if out is None:
        _on_stream(stream, q, s)
    return q, s


def workspace_bytes(M: int, N: int, K: int) -> int:
    """Bytes that serve both linear() and gemm() for this shape."""
    return int(lib().w8a8_workspace_bytes(M, N, K))


def gemm_workspace_bytes(M: int, N: int, K: int) -> int:
    """Bytes gemm() alone needs (its split-K partial sums)."""
    return int(lib().w8a8_gemm_workspace_bytes(M, N, K))


def _workspace(nbytes, device, given=None):
    torch = _torch()
    if given is not None:
        if not given.is_contiguous() or not given.is_cuda:
            raise ValueError("workspace must be a contiguous GPU tensor")
        return given
    if nbytes == 0:
        return None
    return torch.empty((nbytes,), dtype=torch.uint8, device=device)


def gemm(a_q, a_scale, w_q, w_scale, bias=None, out_dtype=None, *, out=None,
         workspace=None, stream=None):
    """INT8 GEMM + fused epilogue.  out_dtype: torch.bfloat16 (default),
    torch.float32 (epilogue before rounding) or torch.int32 (accumulators).
    """
    torch = _torch()
    out_dtype = torch.bfloat16 if out_dtype is None else out_dtype
    codes = {torch.bfloat16: OUT_BF16, torch.float32: OUT_FP32,
             torch.int32: OUT_I32}
    if out_dtype not in codes:
        raise ValueError(f"out_dtype {out_dtype} not supported")
    _need(a_q, torch.int8, 2, "a_q")
    M, K = a_q.shape
    _need(w_q, torch.int8, 2, "w_q")
    N = w_q.shape[0]
    if w_q.shape[1] != K:
        raise ValueError("a_q and w_q disagree on K")
    _need(a_scale, torch.float32, 1, "a_scale", (M,))
    _need(w_scale, torch.float32, 1, "w_scale", (N,))
    if bias is not None:
        _need(bias, torch.bfloat16, 1, "bias", (N,))
    own_out = out is None
    if own_out:
        out = torch.empty((M, N), dtype=out_dtype, device=a_q.device)
    else:
        _need(out, out_dtype, 2, "out", (M, N))
    ws_need = gemm_workspace_bytes(M, N, K)
    ws = _workspace(ws_need, a_q.device, workspace)
    ws_len = 0 if ws is None else ws.numel() * ws.element_size()
    _check("w8a8_gemm", lib().w8a8_gemm(
        _ptr(a_q), _ptr(a_scale), _ptr(w_q), _ptr(w_scale), _ptr(bias),
        _ptr(out), codes[out_dtype], M, N, K, _ptr(ws), ws_len,
        _stream(stream)))
    _on_stream(stream, out if own_out else None,
               ws if workspace is None else None)
    return out


NOALLOC_SCRATCH_BYTES = 64 << 20


def gemm_noalloc(a_q, a_scale, w_q, w_scale, bias=None, out_dtype=None, *,
                 out, stream=None):
    """gemm() without a workspace: the split-K partial sums go to the
    library's own device scratch (w8a8_gemm_noalloc).  ``out`` must be
    given (nothing is allocated).  Calls that overlap in time on one GPU
    share that scratch: keep them on one stream."""
    torch = _torch()
    out_dtype = torch.bfloat16 if out_dtype is None else out_dtype
    codes = {torch.bfloat16: OUT_BF16, torch.float32: OUT_FP32,
             torch.int32: OUT_I32}
    if out_dtype not in codes:
        raise ValueError(f"out_dtype {out_dtype} not supported")
    _need(a_q, torch.int8, 2, "a_q")
    M, K = a_q.shape
    _need(w_q, torch.int8, 2, "w_q")
    N = w_q.shape[0]
    if w_q.shape[1] != K:
        raise ValueError("a_q and w_q disagree on K")
    _need(a_scale, torch.float32, 1, "a_scale", (M,))
    _need(w_scale, torch.float32, 1, "w_scale", (N,))
    if bias is not None:
        _need(bias, torch.bfloat16, 1, "bias", (N,))
    _need(out, out_dtype, 2, "out", (M, N))
    _check("w8a8_gemm_noalloc", lib().w8a8_gemm_noalloc(
        _ptr(a_q), _ptr(a_scale), _ptr(w_q), _ptr(w_scale), _ptr(bias),
        _ptr(out), codes[out_dtype], M, N, K, _stream(stream)))
    return out


def linear(x, w_q, w_scale, bias=None, *, out=None, workspace=None,
           stream=None):
    """y = bf16(((float)(quant(x) . w_q^T) * sa) * sw + bias)."""
    torch = _torch()
    _need(x, torch.bfloat16, 2, "x")
    M, K = x.shape
    _need(w_q, torch.int8, 2, "w_q")
    N = w_q.shape[0]
    if w_q.shape[1] != K:
        raise ValueError("x and w_q disagree on K")
    _need(w_scale, torch.float32, 1, "w_scale", (N,))
    if bias is not None:
        _need(bias, torch.bfloat16, 1, "bias", (N,))
    own_out = out is None
    if own_out:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    else:
        _need(out, torch.bfloat16, 2, "out", (M, N))
    ws = _workspace(workspace_bytes(M, N, K), x.device, workspace)
    ws_len = 0 if ws is None else ws.numel() * ws.element_size()
    _check("w8a8_linear", lib().w8a8_linear(
        _ptr(x), _ptr(w_q), _ptr(w_scale), _ptr(bias), _ptr(out), M, N, K,
        _ptr(ws), ws_len, _stream(stream)))
    _on_stream(stream, out if own_out else None,
               ws if workspace is None else None)
    return out


def silu(x, *, out=None, stream=None):
    torch = _torch()
    _need(x, torch.bfloat16, x.dim(), "x")
    y = torch.empty_like(x) if out is None else out
    _need(y, torch.bfloat16, x.dim(), "out", tuple(x.shape))
    _check("w8a8_silu_bf16", lib().w8a8_silu_bf16(
        _ptr(x), _ptr(y), x.numel(), _stream(stream)))
    if out is None:
        _on_stream(stream, y)
    return y


def pow2_renorm(x, *, out=None, stream=None):
    torch = _torch()
    _need(x, torch.bfloat16, 2, "x")
    M, K = x.shape
    y = torch.empty_like(x) if out is None else out
    _need(y, torch.bfloat16, 2, "out", (M, K))
    _check("w8a8_pow2_renorm", lib().w8a8_pow2_renorm(
        _ptr(x), _ptr(y), M, K, _stream(stream)))
    if out is None:
        _on_stream(stream, y)
    return y


def pow2_renorm_quantize(x, *, out=None, stream=None):
    """x: bf16 [M, K] -> (y bf16 [M, K], a_q int8 [M, K], a_scale float32
    [M]): the power-of-two renormalization and the per-token quantization
    of its result, in one pass."""
    torch = _torch()
    _need(x, torch.bfloat16, 2, "x")
    M, K = x.shape
    if out is None:
        y = torch.empty_like(x)
        q = torch.empty((M, K), dtype=torch.int8, device=x.device)
        s = torch.empty((M,), dtype=torch.float32, device=x.device)
    else:
        y, q, s = out
        _need(y, torch.bfloat16, 2, "out[0]", (M, K))
        _need(q, torch.int8, 2, "out[1]", (M, K))
        _need(s, torch.float32, 1, "out[2]", (M,))
    _check("w8a8_pow2_renorm_quantize", lib().w8a8_pow2_renorm_quantize(
        _ptr(x), M, K, _ptr(y), _ptr(q), _ptr(s), _stream(stream)))
    if out is None:
        _on_stream(stream, y, q, s)
    return y, q, s


def quantize_weight(w, *, out=None, stream=None):
    """w: bf16 [N,K] -> (w_q int8 [N,K], w_scale float32 [N]), one scale
    per output channel; all-zero rows get scale 1."""
    torch = _torch()
    _need(w, torch.bfloat16, 2, "w")
    N, K = w.shape
    if out is None:
        q = torch.empty((N, K), dtype=torch.int8, device=w.device)
        s = torch.empty((N,), dtype=torch.float32, device=w.device)
    else:
        q, s = out
        _need(q, torch.int8, 2, "out[0]", (N, K))
        _need(s, torch.float32, 1, "out[1]", (N,))
    _check("w8a8_quantize_weight", lib().w8a8_quantize_weight(
        _ptr(w), N, K, _ptr(q), _ptr(s), _stream(stream)))
    if out is None:
        _on_stream(stream, q, s)
    return q, s


def check_scales(w_scale, *, out=None, stream=None):
    """Device int32 [1]: how many scales are not finite and > 0."""
    torch = _torch()
    _need(w_scale, torch.float32, 1, "w_scale")
    bad = (torch.empty((1,), dtype=torch.int32, device=w_scale.device)
           if out is None else out)
    _need(bad, torch.int32, 1, "out", (1,))
    _check("w8a8_check_scales", lib().w8a8_check_scales(
        _ptr(w_scale), w_scale.numel(), _ptr(bad), _stream(stream)))
    if out is None:
        _on_stream(stream, bad)
    return bad


def swiglu(h, *, out=None, stream=None):
    """h: bf16 [M, 2F] (gate | up) -> bf16 [M, F]."""
    torch = _torch()
    _need(h, torch.bfloat16, 2, "h")
    M, F2 = h.shape
    if F2 % 2:
        raise ValueError("h must have an even width (gate | up)")
    y = (torch.empty((M, F2 // 2), dtype=torch.bfloat16, device=h.device)
         if out is None else out)
    _need(y, torch.bfloat16, 2, "out", (M, F2 // 2))
    _check("w8a8_swiglu_bf16", lib().w8a8_swiglu_bf16(
        _ptr(h), _ptr(y), M, F2 // 2, _stream(stream)))
    if out is None:
        _on_stream(stream, y)
    return y


def quantize_act_swiglu(h, *, out=None, stream=None):
    """h: bf16 [M, 2F] (gate | up) -> (a_q int8 [M,F], a_scale [M]) of
    SwiGLU(h), in one pass."""
    torch = _torch()
    _need(h, torch.bfloat16, 2, "h")
    M, F2 = h.shape
    if F2 % 2:
        raise ValueError("h must have an even width (gate | up)")
    if out is None:
        q = torch.empty((M, F2 // 2), dtype=torch.int8, device=h.device)
        s = torch.empty((M,), dtype=torch.float32, device=h.device)
    else:
        q, s = out
        _need(q, torch.int8, 2, "out[0]", (M, F2 // 2))
        _need(s, torch.float32, 1, "out[1]", (M,))
    _check("w8a8_quantize_act_swiglu", lib().w8a8_quantize_act_swiglu(
        _ptr(h), M, F2 // 2, _ptr(q), _ptr(s), _stream(stream)))
    if out is None:
        _on_stream(stream, q, s)
    return q, s


# ---------------------------------------------------------------------------
# block norms
# ---------------------------------------------------------------------------

def _norm_arg(kind, weight, bias, eps, H, name):
    """A w8a8_norm_t; the vectors must outlive the call."""
    code = NORM_KINDS.get(kind)
    if code is None:
        raise ValueError(f"{name}: expected one of {sorted(NORM_KINDS)}, got "
                         f"{kind!r}")
    w = b = None
    if weight is not None:
        _need(weight, _torch().bfloat16, 1, f"{name} weight", (H,))
        w = weight.data_ptr()
    if bias is not None:
        _need(bias, _torch().bfloat16, 1, f"{name} bias", (H,))
        b = bias.data_ptr()
    return _Norm(code, eps, w, b)


_MOD_NAMES = ("scale", "shift", "gate")


def _mod_arg(M, H, mod_row, scale=None, shift=None, gate=None):
    """A w8a8_modulation_t from bf16 vectors [H] or tables [rows, H] (rows at
    any stride, their values contiguous) that agree on `rows`; None without
    any."""
    torch = _torch()
    ptr, step, rows = [None] * 3, [0] * 3, None
    for i, t in enumerate((scale, shift, gate)):
        if t is None:
            continue
        name = _MOD_NAMES[i]
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        size, strides = t.shape, t.stride()
        dims = len(size)
        if (t.dtype != torch.bfloat16 or not 1 <= dims <= 2 or
                size[-1] != H or (H > 1 and strides[-1] != 1)):
            raise ValueError(f"{name}: expected {torch.bfloat16} [{H}] or "
                             f"[rows, {H}] with contiguous rows, got "
                             f"{t.dtype} {tuple(size)}")
        _on_current_gpu(t, name)
        n = 1 if dims == 1 else size[0]
        if rows is not None and n != rows:
            raise ValueError(f"{name}: {n} rows, the other vectors have "
                             f"{rows}")
        rows = n
        ptr[i] = t.data_ptr()
        if n != 1:
            step[i] = strides[0]
    row = None
    if mod_row is not None:
        _need(mod_row, torch.int32, 1, "mod_row", (M,))
        row = mod_row.data_ptr()
        if rows is None:  # the index says only which tokens are padding
            rows = 2**31 - 1
    elif rows is None:
        return None
    elif rows != 1 and rows != M:
        raise ValueError(f"{rows} modulation rows for {M} tokens need mod_row")
    return _Modulation(*ptr, *step, rows, row)


def norm_modulate(x, *, norm="rms", weight=None, bias=None, eps=1e-6,
                  scale=None, shift=None, mod_row=None, out=None,
                  stream=None):
    """x: bf16 [M, H] -> bf16 [M, H], norm(x) * (1 + scale) + shift.

    norm: "rms", "layer" or "none"; weight, bias: bf16 [H].  scale, shift:
    bf16 [H], [M, H], or [rows, H] with mod_row (int32 [M]) naming each
    token's row; a row outside [0, rows) marks padding (its output is 0)."""
    torch = _torch()
    _need(x, torch.bfloat16, 2, "x")
    M, H = x.shape
    pre = _norm_arg(norm, weight, bias, eps, H, "norm")
    mod = _mod_arg(M, H, mod_row, scale=scale, shift=shift)
    y = torch.empty_like(x) if out is None else out
    if out is not None:
        _need(y, torch.bfloat16, 2, "out", (M, H))
    _check("w8a8_norm_modulate", lib().w8a8_norm_modulate(
        _ptr(x), M, H, pre, mod, _ptr(y), _stream(stream)))
    if out is None:
        _on_stream(stream, y)
    return y


def norm_modulate_quantize(x, *, norm="rms", weight=None, bias=None,
                           eps=1e-6, scale=None, shift=None, mod_row=None,
                           out=None, stream=None):
    """norm_modulate and the per-token quantization of its values (taken in
    binary32, not rounded to BF16 first) in one pass: x bf16 [M, H] ->
    (a_q int8 [M, H], a_scale float32 [M])."""
    torch = _torch()
    _need(x, torch.bfloat16, 2, "x")
    M, H = x.shape
    pre = _norm_arg(norm, weight, bias, eps, H, "norm")
    mod = _mod_arg(M, H, mod_row, scale=scale, shift=shift)
    if out is None:
        q = x.new_empty((M, H), dtype=torch.int8)
        s = x.new_empty((M,), dtype=torch.float32)
    else:
        q, s = out
        _need(q, torch.int8, 2, "out[0]", (M, H))
        _need(s, torch.float32, 1, "out[1]", (M,))
    _check("w8a8_norm_modulate_quantize", lib().w8a8_norm_modulate_quantize(
        _ptr(x), M, H, pre, mod, _ptr(q), _ptr(s), _stream(stream)))
    if out is None:
        _on_stream(stream, q, s)
    return q, s


def gated_residual(x, branch, *, gate=None, residual_scale=1.0,
                   post_norm="none", post_weight=None, post_bias=None,
                   post_eps=1e-6, mod_row=None, out=None, stream=None):
    """x, branch: bf16 [M, H] -> bf16 [M, H], residual_scale * x + gate *
    post_norm(branch).  gate as norm_modulate's scale; a padding token keeps
    x.  out may be x (in place)."""
    torch = _torch()
    _need(x, torch.bfloat16, 2, "x")
    M, H = x.shape
    _need(branch, torch.bfloat16, 2, "branch", (M, H))
    post = _norm_arg(post_norm, post_weight, post_bias, post_eps, H,
                     "post_norm")
    mod = _mod_arg(M, H, mod_row, gate=gate)
    r = torch.empty_like(x) if out is None else out
    if out is not None:
        _need(r, torch.bfloat16, 2, "out", (M, H))
    _check("w8a8_gated_residual", lib().w8a8_gated_residual(
        _ptr(x), _ptr(branch), M, H, post, mod, residual_scale, _ptr(r),
        _stream(stream)))
    if out is None:
        _on_stream(stream, r)
    return r


def gated_residual_norm(x, branch, *, gate=None, residual_scale=1.0,
                        post_norm="none", post_weight=None, post_bias=None,
                        post_eps=1e-6, norm="rms", weight=None, bias=None,
                        eps=1e-6, scale=None, shift=None, mod_row=None,
                        out=None, stream=None):
    """gated_residual and the norm_modulate of its sum (before that is
    rounded to BF16) in one pass -> (r bf16 [M, H], y bf16 [M, H])."""
    torch = _torch()
    _need(x, torch.bfloat16, 2, "x")
    M, H = x.shape
    _need(branch, torch.bfloat16, 2, "branch", (M, H))
    post = _norm_arg(post_norm, post_weight, post_bias, post_eps, H,
                     "post_norm")
    pre = _norm_arg(norm, weight, bias, eps, H, "norm")
    mod = _mod_arg(M, H, mod_row, scale=scale, shift=shift, gate=gate)
    if out is None:
        r, y = torch.empty_like(x), torch.empty_like(x)
    else:
        r, y = out
        _need(r, torch.bfloat16, 2, "out[0]", (M, H))
        _need(y, torch.bfloat16, 2, "out[1]", (M, H))
    _check("w8a8_gated_residual_norm", lib().w8a8_gated_residual_norm(
        _ptr(x), _ptr(branch), M, H, post, pre, mod, residual_scale, _ptr(r),
        _ptr(y), _stream(stream)))
    if out is None:
        _on_stream(stream, r, y)
    return r, y


def gated_residual_norm_quantize(x, branch, *, gate=None, residual_scale=1.0,
                                 post_norm="none", post_weight=None,
                                 post_bias=None, post_eps=1e-6, norm="rms",
                                 weight=None, bias=None, eps=1e-6, scale=None,
                                 shift=None, mod_row=None, out=None,
                                 stream=None):
    """gated_residual and the norm_modulate_quantize of its sum (before that
    is rounded to BF16) in one pass -> (r bf16 [M, H], a_q int8 [M, H],
    a_scale float32 [M])."""
    torch = _torch()
    _need(x, torch.bfloat16, 2, "x")
    M, H = x.shape
    _need(branch, torch.bfloat16, 2, "branch", (M, H))
    post = _norm_arg(post_norm, post_weight, post_bias, post_eps, H,
                     "post_norm")
    pre = _norm_arg(norm, weight, bias, eps, H, "norm")
    mod = _mod_arg(M, H, mod_row, scale=scale, shift=shift, gate=gate)
    if out is None:
        r = torch.empty_like(x)
        q = x.new_empty((M, H), dtype=torch.int8)
        s = x.new_empty((M,), dtype=torch.float32)
    else:
        r, q, s = out
        _need(r, torch.bfloat16, 2, "out[0]", (M, H))
        _need(q, torch.int8, 2, "out[1]", (M, H))
        _need(s, torch.float32, 1, "out[2]", (M,))
    _check("w8a8_gated_residual_norm_quantize",
           lib().w8a8_gated_residual_norm_quantize(
               _ptr(x), _ptr(branch), M, H, post, pre, mod, residual_scale,
               _ptr(r), _ptr(q), _ptr(s), _stream(stream)))
    if out is None:
        _on_stream(stream, r, q, s)
    return r, q, s


# ---------------------------------------------------------------------------
# linear over few tokens with packed 4-bit weights
# ---------------------------------------------------------------------------

def _w4_out(N, K, group, device, out):
    torch = _torch()
    if group not in W4_GROUPS:
        raise ValueError(f"group: expected one of {W4_GROUPS}, got {group}")
    if N % 16 or K % 128 or not N or not K:
        raise ValueError(f"a packed 4-bit weight needs N % 16 == 0 and "
                         f"K % 128 == 0, got {N} x {K}")
    shapes = ((N // 16, K // 128, 64, 16),
              (N // 16, K // 128, 16, 128 // group))
    if out is None:
        return (torch.empty(shapes[0], dtype=torch.uint8, device=device),
                torch.empty(shapes[1], dtype=torch.bfloat16, device=device))
    w4, s = out
    _need(w4, torch.uint8, 4, "out[0]", shapes[0])
    _need(s, torch.bfloat16, 4, "out[1]", shapes[1])
    return w4, s


def w4_quantize_weight(w, *, group=128, out=None, stream=None):
    """w: bf16 [N, K] -> (w4 uint8 [N/16, K/128, 64, 16], w4_scale bf16
    [N/16, K/128, 16, 128/group]): 4-bit codes with one scale per `group`
    (32, 64 or 128) inputs of a channel, packed for w4_linear."""
    torch = _torch()
    _need(w, torch.bfloat16, 2, "w")
    N, K = w.shape
    w4, s = _w4_out(N, K, group, w.device, out)
    _check("w8a8_w4_quantize_weight", lib().w8a8_w4_quantize_weight(
        _ptr(w), N, K, group, _ptr(w4), _ptr(s), _stream(stream)))
    if out is None:
        _on_stream(stream, w4, s)
    return w4, s


def w4_pack_weight(codes, scales, *, out=None, stream=None):
    """Codes int8 [N, K] (clamped to [-8, 7]) and scales bf16 [N, K/group]
    made elsewhere -> (w4, w4_scale) as w4_quantize_weight."""
    torch = _torch()
    _need(codes, torch.int8, 2, "codes")
    N, K = codes.shape
    _need(scales, torch.bfloat16, 2, "scales")
    if scales.shape[0] != N or not scales.shape[1] or K % scales.shape[1]:
        raise ValueError(f"scales: expected [{N}, K/group], got "
                         f"{tuple(scales.shape)}")
    group = K // scales.shape[1]
    w4, s = _w4_out(N, K, group, codes.device, out)
    _check("w8a8_w4_pack_weight", lib().w8a8_w4_pack_weight(
        _ptr(codes), _ptr(scales), N, K, group, _ptr(w4), _ptr(s),
        _stream(stream)))
    if out is None:
        _on_stream(stream, w4, s)
    return w4, s


def w4_linear(x, w4, w4_scale, bias=None, *, out=None, stream=None):
    """x: bf16 [M, K], a packed 4-bit weight -> bf16 [M, N], x . w^T + bias
    (weight-only: x stays BF16).  Made for a few tokens."""
    torch = _torch()
    _need(x, torch.bfloat16, 2, "x")
    M, K = x.shape
    _need(w4, torch.uint8, 4, "w4")
    tiles, blocks, lanes, nbytes = w4.shape
    if lanes != 64 or nbytes != 16 or blocks * 128 != K:
        raise ValueError(f"w4: expected [N/16, {K}/128, 64, 16], got "
                         f"{tuple(w4.shape)}")
    N = 16 * tiles
    _need(w4_scale, torch.bfloat16, 4, "w4_scale")
    parts = w4_scale.shape[3]
    if w4_scale.shape != (tiles, blocks, 16, parts) or parts not in (1, 2, 4):
        raise ValueError(f"w4_scale: expected [{tiles}, {blocks}, 16, "
                         f"128/group], got {tuple(w4_scale.shape)}")
    if bias is not None:
        _need(bias, torch.bfloat16, 1, "bias", (N,))
    own_out = out is None
    if own_out:
        out = x.new_empty((M, N))
    else:
        _need(out, torch.bfloat16, 2, "out", (M, N))
    _check("w8a8_w4_linear", lib().w8a8_w4_linear(
        _ptr(x), _ptr(w4), _ptr(w4_scale), _ptr(bias), _ptr(out), M, N, K,
        128 // parts, _stream(stream)))
    _on_stream(stream, out if own_out else None)
    return out


# ---------------------------------------------------------------------------
# heads: rotary table, head norms with rotation, attention
# ---------------------------------------------------------------------------

def rope_table(positions, pairs, *, theta=10000.0, scaling="none", factor=1.0,
               original=0.0, beta_fast=32.0, beta_slow=1.0, amplitude=None,
               out=None, stream=None):
    """positions: int32 or float32 [T] or [T, axes] -> float32 [T, 2, P], the
    cosines and sines of P = sum(pairs) pairs a token.

    pairs: how many pairs each axis turns (a number for one axis).  scaling:
    "none", "linear", "ntk" or "yarn" (the last with `original`, the number of
    positions that the unscaled rotation was made for, and an amplitude of
    0.1 ln(factor) + 1 unless given)."""
    torch = _torch()
    if not isinstance(positions, torch.Tensor):
        raise TypeError("positions must be a torch.Tensor")
    kind = {torch.int32: 0, torch.float32: 1}.get(positions.dtype)
    if kind is None:
        raise ValueError(f"positions: expected int32 or float32, got "
                         f"{positions.dtype}")
    pairs = (pairs,) if isinstance(pairs, int) else tuple(pairs)
    if not 1 <= len(pairs) <= ROPE_MAX_AXES or min(pairs) < 1 or \
            sum(pairs) > ROPE_MAX_PAIRS:
        raise ValueError(f"pairs: expected 1 to {ROPE_MAX_AXES} axes of 1 or "
                         f"more pairs, {ROPE_MAX_PAIRS} in all, got {pairs}")
    if positions.dim() == 1 and len(pairs) == 1:
        _need(positions, positions.dtype, 1, "positions")
    else:
        _need(positions, positions.dtype, 2, "positions",
              (positions.shape[0] if positions.dim() else 0, len(pairs)))
    code = ROPE_SCALINGS.get(scaling)
    if code is None:
        raise ValueError(f"scaling: expected one of {sorted(ROPE_SCALINGS)}, "
                         f"got {scaling!r}")
    if amplitude is None:
        amplitude = (0.1 * math.log(factor) + 1
                     if scaling == "yarn" and factor > 1 else 1.0)
    T, P = positions.shape[0], sum(pairs)
    own_out = out is None
    if own_out:
        out = torch.empty((T, 2, P), dtype=torch.float32,
                          device=positions.device)
    else:
        _need(out, torch.float32, 3, "out", (T, 2, P))
    rope = _Rope(len(pairs), (ctypes.c_int * 4)(*pairs), code, theta, factor,
                 original, beta_fast, beta_slow, amplitude)
    _check("w8a8_rope_table", lib().w8a8_rope_table(
        _ptr(positions), kind, T, rope, _ptr(out), _stream(stream)))
    _on_stream(stream, out if own_out else None)
    return out


def _head_rows(t, name, batch=False):
    """t: bf16 [tokens, heads, width], or with `batch` also [sequences, tokens,
    heads, width]; the heads of a token behind each other, tokens at any stride
    (a part of a fused output's columns), sequences behind each other -> (all
    tokens, their stride)."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    size, step = t.shape, t.stride()
    dims = len(size)
    if (t.dtype != torch.bfloat16 or not (dims == 3 or batch and dims == 4) or
            (step[-1] != 1 and size[-1] > 1) or
            (step[-2] != size[-1] and size[-2] > 1)):
        raise ValueError(f"{name}: expected {torch.bfloat16} [tokens, heads, "
                         f"width] with the heads of a token behind each "
                         f"other, got {t.dtype} {tuple(size)} with strides "
                         f"{step}")
    _on_current_gpu(t, name)
    rows = size[-3]
    if rows == 0:  # nothing lies anywhere
        return 0, size[-2] * size[-1]
    if dims == 4 and size[0] > 1:
        if rows == 1:
            return size[0], step[0]
        if step[0] != rows * step[1]:
            raise ValueError(f"{name}: the batch's sequences must follow each "
                             f"other, got strides {step}")
        return size[0] * rows, step[1]
    return rows, step[-3] if rows > 1 else size[-2] * size[-1]


def _heads_arg(x, y, kind, weight, bias, eps, name):
    """A w8a8_heads_t; y: the output given, or None for a new tensor -> (the
    argument, its output); the vectors must outlive the call."""
    stride = _head_rows(x, name)[1]
    _, H, D = size = x.shape
    if y is None:
        y = x.new_empty(size)
        y_stride = H * D
    else:
        y_stride = _head_rows(y, f"{name}'s output")[1]
        if y.shape != size:
            raise ValueError(f"{name}'s output: expected shape {tuple(size)}, "
                             f"got {tuple(y.shape)}")
    per_head, ptr = None, [None, None]
    for i, t in enumerate((weight, bias)):
        if t is None:
            continue
        full = getattr(t, "ndim", 0) == 2
        _need(t, x.dtype, 2 if full else 1, f"{name} {('weight', 'bias')[i]}",
              (H, D) if full else (D,))
        full = full and H > 1  # [1, D] is [D]
        if per_head is not None and per_head != full:
            raise ValueError(f"{name}: weight and bias must both be [{D}] or "
                             f"both [{H}, {D}]")
        per_head, ptr[i] = full, t.data_ptr()
    return _Heads(x.data_ptr(), y.data_ptr(), H, stride, y_stride,
                  (kind, eps, *ptr), bool(per_head)), y


def _table_args(M, table, row):
    """(table, pairs, rows, row) of a rotation."""
    if table is None:
        if row is not None:
            raise ValueError("row needs a table")
        return None, 0, 0, None
    torch = _torch()
    _need(table, torch.float32, 3, "table")
    rows, two, pairs = table.shape
    if two != 2:
        raise ValueError(f"table: expected [rows, 2, pairs], got "
                         f"{tuple(table.shape)}")
    if row is not None:
        _need(row, torch.int32, 1, "row", (M,))
    elif rows != 1 and rows != M:
        raise ValueError(f"a table of {rows} rows for {M} tokens needs row")
    return table.data_ptr(), pairs, rows, _ptr(row)


def head_norm_rope(q, k=None, *, norm="rms", q_weight=None, q_bias=None,
                   k_weight=None, k_bias=None, eps=1e-6, table=None, row=None,
                   interleaved=False, out=None, stream=None):
    """Each head's norm, then its rotation by the token's row of a rope_table:
    q bf16 [M, heads, D] (and k [M, k_heads, D]) -> the same shapes, as a pair
    where k is given.

    Tokens may lie at any stride (parts of a fused Q, K, V output).  norm:
    "rms", "layer" or "none"; weights and biases bf16 [D] or [heads, D].  table:
    float32 [rows, 2, pairs], turning the first 2 pairs values of a head: values
    i and i + pairs, or 2 i and 2 i + 1 (interleaved); row m is token m's, or
    row[m] (int32 [M]; outside the table: padding, zeros).  out: a tensor (a
    pair with k), which may be the inputs."""
    code = NORM_KINDS.get(norm)
    if code is None:
        raise ValueError(f"norm: expected one of {sorted(NORM_KINDS)}, got "
                         f"{norm!r}")
    if k is None:
        if k_weight is not None or k_bias is not None:
            raise ValueError("k_weight and k_bias need k")
        out_q, out_k = out, None
    elif out is None:
        out_q = out_k = None
    elif len(out) != 2:
        raise ValueError("out: expected a pair, for q and for k")
    else:
        out_q, out_k = out
    side_q, out_q = _heads_arg(q, out_q, code, q_weight, q_bias, eps, "q")
    M, _, D = q.shape
    side_k = None
    if k is not None:
        side_k, out_k = _heads_arg(k, out_k, code, k_weight, k_bias, eps, "k")
        if k.shape[0] != M or k.shape[2] != D:
            raise ValueError(f"q and k disagree: {tuple(q.shape)}, "
                             f"{tuple(k.shape)}")
    rot = _table_args(M, table, row)
    _check("w8a8_head_norm_rope", lib().w8a8_head_norm_rope(
        side_q, side_k, M, D, *rot, bool(interleaved), _stream(stream)))
    if out is None:
        _on_stream(stream, out_q, out_k)
    return out_q if k is None else (out_q, out_k)


def rope(x, table, *, row=None, interleaved=False, out=None, stream=None):
    """The rotation alone: x bf16 [M, heads, D] -> the same (head_norm_rope
    without a norm)."""
    if table is None:
        raise ValueError("rope needs a table")
    return head_norm_rope(x, norm="none", table=table, row=row,
                          interleaved=interleaved, out=out, stream=stream)


def _offsets_arg(t, B, name):
    """Pointer of int32 [B + 1] offsets (B None: any number), and B."""
    if t is None:
        return None, B
    _need(t, _torch().int32, 1, name)
    n = t.shape[0]
    if n < 2 or (B is not None and n != B + 1):
        raise ValueError(f"{name}: expected "
                         f"{'two or more' if B is None else B + 1} offsets, "
                         f"got {n}")
    return t.data_ptr(), n - 1


def attention(q, k, v, *, scale=None, q_offsets=None, k_offsets=None,
              k_lens=None, out=None, workspace=None, stream=None):
    """softmax(scale q k^T) v per head, over all keys of a sequence (scale: 1 /
    sqrt(width) unless given).

    q: bf16 [Tq, heads, D]; k, v: [Tk, k_heads, D], k_heads dividing heads (a
    group of query heads shares a key head); tokens at any stride.  One
    sequence, or several: packed behind each other with q_offsets and k_offsets
    (int32 [B + 1]; None: equal lengths), or as a batch q [B, Lq, heads, D], k
    and v [B, Lk, k_heads, D].  k_lens (int32 [B]): how many of a sequence's
    keys count.  Returns bf16 of q's shape; rows outside of all sequences are
    not written, those of a sequence without keys are zero.  workspace:
    attention_workspace_bytes of uint8, of this call alone while it runs."""
    Tq, q_stride = _head_rows(q, "q", True)
    Tk, k_stride = _head_rows(k, "k", True)
    _, v_stride = _head_rows(v, "v", True)
    size, k_size = q.shape, k.shape
    Hq, D = size[-2:]
    Hk = k_size[-2]
    if v.shape != k_size:
        raise ValueError(f"v: expected shape {tuple(k_size)}, got "
                         f"{tuple(v.shape)}")
    if k_size[-1] != D or len(k_size) != len(size):
        raise ValueError(f"q and k disagree: {tuple(size)}, {tuple(k_size)}")
    B = None
    if len(size) == 4:
        if q_offsets is not None or k_offsets is not None:
            raise ValueError("offsets go with [tokens, heads, width]")
        B = size[0]
        if k_size[0] != B:
            raise ValueError(f"q and k disagree: {tuple(size)}, "
                             f"{tuple(k_size)}")
    qo, B = _offsets_arg(q_offsets, B, "q_offsets")
    ko, B = _offsets_arg(k_offsets, B, "k_offsets")
    kl = None
    if k_lens is not None:
        _need(k_lens, _torch().int32, 1, "k_lens", None if B is None else (B,))
        kl, B = k_lens.data_ptr(), k_lens.shape[0]
    own_out = out is None
    if own_out:
        out = q.new_empty(size)
        out_stride = Hq * D
    else:
        _, out_stride = _head_rows(out, "out", True)
        if out.shape != size:
            raise ValueError(f"out: expected shape {tuple(size)}, got "
                             f"{tuple(out.shape)}")
    if scale is None:
        scale = D ** -0.5 if D else 1.0
    a = _Attention(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                   q_stride, k_stride, v_stride, out_stride, Tq, Tk,
                   1 if B is None else B, Hq, Hk, D, qo, ko, kl, scale)
    L, s = lib(), _stream(stream)
    if workspace is None:
        # Most calls need none, and asking costs as much as such a call's checks.
        status = L.w8a8_attention(a, None, 0, s)
        if status == W8A8_ERR_WORKSPACE:
            ws = _workspace(int(L.w8a8_attention_workspace_bytes(a)), q.device)
            status = L.w8a8_attention(a, ws.data_ptr(), ws.numel(), s)
            _on_stream(stream, ws)
    else:
        ws = _workspace(0, q.device, workspace)
        _on_current_gpu(ws, "workspace")
        status = L.w8a8_attention(a, ws.data_ptr(),
                                  ws.numel() * ws.element_size(), s)
    _check("w8a8_attention", status)
    if own_out:
        _on_stream(stream, out)
    return out


def attention_workspace_bytes(Tq, Tk, heads, k_heads, D, *, B=1,
                              packed=False):
    """Bytes attention() needs for B sequences of Tq query and Tk key rows in
    all; packed: with q_offsets."""
    a = _Attention(Tq=Tq, Tk=Tk, B=B, q_heads=heads, k_heads=k_heads, D=D,
                   q_stride=heads * D, k_stride=k_heads * D,
                   v_stride=k_heads * D, out_stride=heads * D, scale=1.0,
                   q_offsets=4 if packed else None, k_offsets=4)
    return int(lib().w8a8_attention_workspace_bytes(a))
