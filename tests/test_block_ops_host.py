"""Refusals of the block norms and the 4-bit linear, on the host: every call
here fails validation before the library touches a device (pointers are fake
addresses that are never dereferenced; without a GPU a valid call ends at the
device check)."""
from __future__ import annotations

import ctypes
import math

import pytest
import torch

from w8a8_int8_gemm_amd import binding as B

OK, NULL, SHAPE, ALIGN, WORKSPACE, OUT_DTYPE, ALIAS, DEVICE, HIP, ARG = range(10)
NONE, RMS, LAYER = 0, 1, 2

A = 0x10_0000_0000
P = {name: A + i * 0x2_0000_0000 for i, name in enumerate(
    ["x", "branch", "r", "y", "q", "qs", "w", "b", "pw", "pb", "scale",
     "shift", "gate", "row", "w4", "s4", "codes", "bias"])}

no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0,
                            reason="fake pointers would reach a kernel")


def norm(kind=RMS, eps=1e-6, weight=P["w"], bias=None):
    return B._Norm(kind, eps, weight, bias)


def mod(scale=P["scale"], shift=P["shift"], gate=P["gate"], stride=4096,
        rows=4, row=P["row"], **kw):
    m = B._Modulation(scale, shift, gate, stride, stride, stride, rows, row)
    for k, v in kw.items():
        setattr(m, k, v)
    return m


def call(which, **kw):
    a = dict(x=P["x"], branch=P["branch"], M=64, H=1024, post=norm(
        weight=P["pw"]), pre=norm(), mod=mod(), rs=1.0, r=P["r"], y=P["y"],
        q=P["q"], qs=P["qs"])
    a.update(kw)
    L = B.lib()
    if which == "norm":
        return L.w8a8_norm_modulate(a["x"], a["M"], a["H"], a["pre"],
                                    a["mod"], a["y"], None)
    if which == "norm_quantize":
        return L.w8a8_norm_modulate_quantize(
            a["x"], a["M"], a["H"], a["pre"], a["mod"], a["q"], a["qs"], None)
    head = (a["x"], a["branch"], a["M"], a["H"], a["post"])
    if which == "residual":
        return L.w8a8_gated_residual(*head, a["mod"], a["rs"], a["r"], None)
    if which == "residual_norm":
        return L.w8a8_gated_residual_norm(*head, a["pre"], a["mod"], a["rs"],
                                          a["r"], a["y"], None)
    return L.w8a8_gated_residual_norm_quantize(
        *head, a["pre"], a["mod"], a["rs"], a["r"], a["q"], a["qs"], None)


ALL = ["norm", "norm_quantize", "residual", "residual_norm",
       "residual_norm_quantize"]
RESIDUAL = ALL[2:]
PRE = [f for f in ALL if f != "residual"]


@no_gpu
@pytest.mark.parametrize("which", ALL)
def test_valid_calls_reach_the_device_check(which):
    assert call(which) == DEVICE
    assert call(which, mod=None, pre=None, post=None) == DEVICE
    assert call(which, M=(1 << 24) - 1, H=8) == DEVICE
    assert call(which, H=32768, mod=mod(stride=32768)) == DEVICE
    assert call(which, mod=mod(row=None, rows=64)) == DEVICE
    assert call(which, mod=mod(row=None, rows=1, stride=0)) == DEVICE
    assert call(which, mod=mod(None, None, None, rows=2**31 - 1)) == DEVICE
    assert call(which, mod=mod(None, None, None, rows=0, row=None)) == DEVICE
    assert call(which, r=P["x"]) == DEVICE  # in place
    assert call(which, pre=norm(LAYER, 2.0**-126, None, P["b"])) == DEVICE


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), NULL), (dict(M=0), SHAPE), (dict(M=-1), SHAPE),
    (dict(M=1 << 24), SHAPE), (dict(H=0), SHAPE), (dict(H=4), SHAPE),
    (dict(H=1020), SHAPE), (dict(H=32776), SHAPE),
    (dict(M=(1 << 24) - 1, H=4104, mod=None), SHAPE),
    (dict(x=P["x"] + 8), ALIGN),
    (dict(mod=mod(rows=0)), SHAPE), (dict(mod=mod(rows=-1)), SHAPE),
    (dict(mod=mod(rows=1 << 31)), SHAPE),
    (dict(mod=mod(rows=4, row=None)), SHAPE),
    (dict(mod=mod(rows=65, row=None)), SHAPE),
    (dict(mod=mod(stride=1016)), SHAPE), (dict(mod=mod(stride=1028)), SHAPE),
    (dict(mod=mod(stride=-1024)), SHAPE),
    (dict(mod=mod(stride=1 << 30)), SHAPE),
    (dict(mod=mod(row=P["row"] + 2)), ALIGN),
    (dict(mod=mod(scale=P["scale"] + 8, shift=P["shift"] + 8,
                  gate=P["gate"] + 8)), ALIGN),
    (dict(mod=mod(rows=0, scale=None, shift=None, gate=None)), SHAPE),
])
@pytest.mark.parametrize("which", ALL)
def test_rejects(which, kw, code):
    assert call(which, **kw) == code


@pytest.mark.parametrize("which", PRE)
@pytest.mark.parametrize("pre,code", [
    (norm(3), ARG), (norm(-1), ARG), (norm(RMS, 0.0), ARG),
    (norm(RMS, 2.0**-127), ARG), (norm(RMS, -1.0), ARG),
    (norm(RMS, math.inf), ARG), (norm(LAYER, math.nan), ARG),
    (norm(RMS, bias=P["b"]), ARG), (norm(NONE), ARG),
    (norm(NONE, weight=None, bias=P["b"]), ARG),
    (norm(RMS, weight=P["w"] + 2), ALIGN),
    (norm(LAYER, bias=P["b"] + 8), ALIGN),
])
def test_norm_arguments(which, pre, code):
    assert call(which, pre=pre) == code
    if which in RESIDUAL:
        assert call(which, post=pre) == code


@pytest.mark.parametrize("which", RESIDUAL)
def test_residual_rejects(which):
    assert call(which, branch=None) == NULL
    assert call(which, r=None) == NULL
    assert call(which, branch=P["branch"] + 2) == ALIGN
    assert call(which, r=P["r"] + 8) == ALIGN
    for rs in (math.nan, math.inf, -math.inf):
        assert call(which, rs=rs) == ARG
    assert call(which, r=P["x"] + 16) == ALIAS       # partly over x
    assert call(which, r=P["branch"]) == ALIAS
    assert call(which, r=P["branch"] - 16) == ALIAS
    for v in ("w", "gate", "row", "pw"):
        if v == "w" and which == "residual":
            continue
        assert call(which, r=P[v] - 64 * 1024 * 2 + 16) == ALIAS, v
    # the last row of a strided table
    assert call(which, r=P["gate"] + 3 * 4096 * 2 + 2032) == ALIAS


def test_output_overlaps():
    y, q, qs = P["y"], P["q"], P["qs"]
    assert call("norm", y=None) == NULL
    assert call("norm_quantize", q=None) == NULL
    assert call("norm_quantize", qs=None) == NULL
    assert call("norm", y=y + 8) == ALIGN
    assert call("norm_quantize", q=q + 4) == ALIGN
    assert call("norm_quantize", qs=qs + 2) == ALIGN
    for v in ("x", "w", "scale", "shift", "row"):
        assert call("norm", y=P[v]) == ALIAS, v
        assert call("norm_quantize", q=P[v]) == ALIAS, v
        assert call("norm_quantize", qs=P[v]) == ALIAS, v
    assert call("norm_quantize", qs=q + 64) == ALIAS
    assert call("residual_norm", y=P["r"] + 4096) == ALIAS
    assert call("residual_norm", r=P["x"], y=P["x"]) == ALIAS
    assert call("residual_norm", y=P["branch"]) == ALIAS
    assert call("residual_norm_quantize", q=P["r"] + 64) == ALIAS
    assert call("residual_norm_quantize", qs=P["branch"] + 64) == ALIAS


def w4(which, **kw):
    a = dict(x=P["x"], w=P["w"], codes=P["codes"], scales=P["scale"],
             w4=P["w4"], s4=P["s4"], bias=P["bias"], y=P["y"], M=4, N=1024,
             K=1024, G=128)
    a.update(kw)
    L = B.lib()
    if which == "quantize":
        return L.w8a8_w4_quantize_weight(a["w"], a["N"], a["K"], a["G"],
                                         a["w4"], a["s4"], None)
    if which == "pack":
        return L.w8a8_w4_pack_weight(a["codes"], a["scales"], a["N"], a["K"],
                                     a["G"], a["w4"], a["s4"], None)
    return L.w8a8_w4_linear(a["x"], a["w4"], a["s4"], a["bias"], a["y"],
                            a["M"], a["N"], a["K"], a["G"], None)


W4 = ["quantize", "pack", "linear"]


@pytest.mark.parametrize("kw,code", [
    (dict(w4=None), NULL), (dict(s4=None), NULL),
    (dict(N=0), SHAPE), (dict(N=8), SHAPE), (dict(N=1032), SHAPE),
    (dict(N=1 << 26), SHAPE), (dict(K=0), SHAPE), (dict(K=64), SHAPE),
    (dict(K=1056), SHAPE), (dict(K=B.MAX_K + 128), SHAPE),
    (dict(N=1 << 25, K=4096), SHAPE),
    (dict(G=0), ARG), (dict(G=16), ARG), (dict(G=256), ARG),
    (dict(G=-128), ARG), (dict(w4=P["w4"] + 8), ALIGN),
    (dict(s4=P["s4"] + 8), ALIGN)])
@pytest.mark.parametrize("which", W4)
def test_w4_rejects(which, kw, code):
    assert w4(which, **kw) == code


def test_w4_own_rejects():
    assert w4("quantize", w=None) == NULL
    assert w4("quantize", w=P["w"] + 8) == ALIGN
    assert w4("quantize", w=P["w4"] + 16) == ALIAS
    assert w4("quantize", s4=P["w4"] + 16) == ALIAS
    assert w4("pack", codes=None) == NULL
    assert w4("pack", scales=None) == NULL
    assert w4("pack", codes=P["codes"] + 8) == ALIGN
    assert w4("pack", scales=P["scale"] + 8) == ALIGN
    assert w4("pack", w4=P["codes"]) == ALIAS
    assert w4("pack", s4=P["scale"]) == ALIAS
    assert w4("linear", x=None) == NULL
    assert w4("linear", y=None) == NULL
    for M in (0, -1, 32 * 65535 + 1):
        assert w4("linear", M=M) == SHAPE
    assert w4("linear", x=P["x"] + 8) == ALIGN
    assert w4("linear", y=P["y"] + 8) == ALIGN
    assert w4("linear", bias=P["bias"] + 1) == ALIGN
    for v in ("x", "w4", "s4", "bias"):
        assert w4("linear", y=P[v]) == ALIAS, v


@no_gpu
def test_w4_valid_calls_reach_the_device_check():
    for which in W4:
        for G in B.W4_GROUPS:
            assert w4(which, G=G) == DEVICE
        assert w4(which, N=16, K=B.MAX_K) == DEVICE
    assert w4("linear", bias=None, M=32 * 65535) == DEVICE
    assert w4("linear", bias=P["bias"] + 2) == DEVICE


def test_binding_checks_tensors():
    """Wrong types, shapes, kinds and devices are refused in Python."""
    bf = torch.bfloat16
    x = torch.zeros((4, 64), dtype=bf)
    with pytest.raises(ValueError):
        B.norm_modulate(x)  # not on the GPU
    with pytest.raises(ValueError):
        B.norm_modulate(x.float())
    with pytest.raises(TypeError):
        B.norm_modulate([1.0])
    with pytest.raises(ValueError):
        B.gated_residual(x, x)
    with pytest.raises(ValueError):
        B.w4_quantize_weight(torch.zeros((128, 128), dtype=bf))
    with pytest.raises(ValueError):
        B.w4_linear(x, torch.zeros(1), torch.zeros(1))
    with pytest.raises(ValueError, match="expected one of"):
        B._norm_arg("batch", None, None, 1e-6, 64, "norm")
    with pytest.raises(ValueError, match="disagree|other vectors|contiguous"):
        B._mod_arg(4, 64, None, scale=torch.zeros((4, 32), dtype=bf))
    with pytest.raises(ValueError, match="group"):
        B._w4_out(128, 128, 48, "cpu", None)
    with pytest.raises(ValueError, match="N % 16"):
        B._w4_out(120, 128, 32, "cpu", None)


def test_struct_layout_matches_the_header():
    """The binding's structs against a C compiler's reading of the header."""
    import pathlib
    import subprocess
    import tempfile
    root = pathlib.Path(__file__).resolve().parents[1]
    src = '#include "w8a8.h"\n#include <stdio.h>\nint main(void){\n'
    want = []
    for name, cls in (("w8a8_norm_t", B._Norm),
                      ("w8a8_modulation_t", B._Modulation)):
        src += f'printf("%zu\\n", sizeof({name}));\n'
        want.append(ctypes.sizeof(cls))
        for field, _ in cls._fields_:
            src += f'printf("%zu\\n", offsetof({name}, {field}));\n'
            want.append(getattr(cls, field).offset)
    src += "return 0;}\n"
    with tempfile.TemporaryDirectory() as d:
        f = pathlib.Path(d) / "t.c"
        f.write_text(src)
        subprocess.run(["gcc", "-std=c11", f"-I{root / 'include'}", str(f),
                        "-o", f"{d}/t"], check=True)
        out = subprocess.run([f"{d}/t"], check=True, capture_output=True,
                             text=True).stdout
    assert [int(v) for v in out.split()] == want
