"""Refusals of the rotary table, the head norms with rotation and the attention,
on the host: every call here fails validation before the library touches a
device (pointers are fake addresses that are never dereferenced; without a GPU
a valid call ends at the device check), and what the binding works out itself."""
from __future__ import annotations

import math

import pytest
import torch

from w8a8_int8_gemm_amd import binding as B

OK, NULL, SHAPE, ALIGN, WORKSPACE, OUT_DTYPE, ALIAS, DEVICE, HIP, ARG = range(10)
NONE, RMS, LAYER = 0, 1, 2

A = 0x10_0000_0000
P = {name: A + i * 0x40_0000_0000 for i, name in enumerate(
    ["q", "k", "v", "out", "yq", "yk", "wq", "bq", "wk", "bk", "table", "row",
     "pos", "qo", "ko", "kl", "ws"])}

no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0,
                            reason="fake pointers would reach a kernel")


# ---------------------------------------------------------------------------
# rotary table
# ---------------------------------------------------------------------------

def rope(pairs=(16, 8), **kw):
    r = B._Rope(len(pairs), (B.ctypes.c_int * 4)(*pairs[:4]), 0, 1e4, 1.0, 0.0,
                0.0, 0.0, 1.0)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def table(**kw):
    a = dict(pos=P["pos"], kind=0, T=10, rope=rope(), table=P["table"])
    a.update(kw)
    return B.lib().w8a8_rope_table(a["pos"], a["kind"], a["T"], a["rope"],
                                   a["table"], None)


YARN = dict(scaling=3, factor=2.0, original=4096.0, beta_fast=32.0,
            beta_slow=1.0)


@no_gpu
@pytest.mark.parametrize("kw", [
    {}, dict(kind=1), dict(T=(1 << 24) - 1), dict(rope=rope((256,))),
    dict(rope=rope((1, 1, 1, 253))), dict(rope=rope(scaling=2, factor=4.0)),
    dict(rope=rope(factor=math.nan)), dict(rope=rope(amplitude=0.0)),
    dict(rope=rope(**YARN))])
def test_table_valid_calls_reach_the_device_check(kw):
    assert table(**kw) == DEVICE


@pytest.mark.parametrize("kw,code", [
    (dict(pos=None), NULL), (dict(rope=None), NULL), (dict(table=None), NULL),
    (dict(T=0), SHAPE), (dict(T=1 << 24), SHAPE), (dict(T=-3), SHAPE),
    (dict(rope=rope(axes=0)), SHAPE), (dict(rope=rope(axes=5)), SHAPE),
    (dict(rope=rope((16, 0))), SHAPE), (dict(rope=rope((16, -4))), SHAPE),
    (dict(rope=rope((200, 57))), SHAPE),
    (dict(rope=rope((2**31 - 1, 2**31 - 1))), SHAPE),
    (dict(kind=2), ARG), (dict(kind=-1), ARG),
    (dict(rope=rope(scaling=4)), ARG), (dict(rope=rope(scaling=-1)), ARG),
    (dict(rope=rope(theta=1.0)), ARG), (dict(rope=rope(theta=math.nan)), ARG),
    (dict(rope=rope(theta=math.inf)), ARG),
    (dict(rope=rope(amplitude=math.nan)), ARG),
    (dict(rope=rope(amplitude=1e39)), ARG),
    (dict(rope=rope((2, 8), scaling=2, factor=1e160)), ARG),
    (dict(rope=rope(scaling=1, factor=0.5)), ARG),
    (dict(rope=rope(scaling=2, factor=math.inf)), ARG),
    (dict(rope=rope(**{**YARN, "original": 0.0})), ARG),
    (dict(rope=rope(**{**YARN, "beta_fast": -1.0})), ARG),
    (dict(rope=rope(**{**YARN, "beta_slow": math.nan})), ARG),
    (dict(pos=P["pos"] + 2), ALIGN), (dict(table=P["table"] + 8), ALIGN),
    (dict(table=P["pos"] + 16), ALIAS), (dict(pos=P["table"] + 4), ALIAS),
])
def test_table_rejects(kw, code):
    assert table(**kw) == code


# ---------------------------------------------------------------------------
# head norms with rotation
# ---------------------------------------------------------------------------

def side(which="q", heads=8, D=64, kind=RMS, eps=1e-6, bias=None, **kw):
    s = B._Heads(P[which], P["y" + which], heads, heads * D, heads * D,
                 B._Norm(kind, eps, P["w" + which] if kind else None, bias), 0)
    for k, v in kw.items():
        if k == "weight":
            s.norm.weight = v
        else:
            setattr(s, k, v)
    return s


def heads(**kw):
    a = dict(q=side(), k=side("k", 2), M=40, D=64, table=P["table"], pairs=32,
             rows=40, row=None, inter=0)
    a.update(kw)
    return B.lib().w8a8_head_norm_rope(a["q"], a["k"], a["M"], a["D"],
                                       a["table"], a["pairs"], a["rows"],
                                       a["row"], a["inter"], None)


@no_gpu
@pytest.mark.parametrize("kw", [
    {}, dict(k=None), dict(table=None, rows=0, pairs=7), dict(inter=1),
    dict(rows=1), dict(rows=7, row=P["row"]), dict(pairs=4),
    dict(rows=2**31 - 1, row=P["row"]), dict(q=side(y=P["q"])),
    dict(q=side(kind=LAYER, bias=P["bq"])), dict(q=side(kind=NONE)),
    dict(q=side(x_stride=1 << 20, y_stride=4096)),
    dict(q=side(per_head=1, kind=LAYER, bias=P["bq"])),
    # q and k side by side in one buffer, in place
    dict(q=side(x_stride=640, y_stride=640, y=P["q"]),
         k=side("k", 2, x=P["q"] + 1024, y=P["q"] + 1024, x_stride=640,
                y_stride=640)),
    dict(M=(1 << 24) - 1, rows=1, q=side(heads=1), k=None),
    dict(D=256, q=side(D=256), k=side("k", 2, D=256), pairs=128),
    dict(D=8, q=side(D=8, heads=4096), k=None, pairs=4),
])
def test_heads_valid_calls_reach_the_device_check(kw):
    assert heads(**kw) == DEVICE


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), NULL), (dict(q=side(x=None)), NULL),
    (dict(k=side("k", 2, y=None)), NULL),
    (dict(M=0), SHAPE), (dict(M=1 << 24, rows=1), SHAPE), (dict(D=0), SHAPE),
    (dict(D=60), SHAPE), (dict(D=264, q=side(D=264), k=None), SHAPE),
    (dict(pairs=0), SHAPE), (dict(pairs=36), SHAPE), (dict(pairs=6), SHAPE),
    (dict(pairs=-4), SHAPE), (dict(rows=0), SHAPE), (dict(rows=39), SHAPE),
    (dict(rows=1 << 31, row=P["row"]), SHAPE),
    (dict(q=side(heads=0)), SHAPE), (dict(q=side(heads=-1)), SHAPE),
    (dict(q=side(heads=4097)), SHAPE), (dict(q=side(x_stride=504)), SHAPE),
    (dict(q=side(y_stride=516)), SHAPE), (dict(q=side(x_stride=1 << 30)), SHAPE),
    (dict(k=side("k", 2, x_stride=-128)), SHAPE),
    (dict(M=(1 << 24) - 1, rows=1, q=side(heads=65, x_stride=4160,
                                          y_stride=4160)), SHAPE),
    (dict(q=side(kind=3)), ARG), (dict(q=side(eps=0.0)), ARG),
    (dict(q=side(eps=math.inf)), ARG), (dict(q=side(bias=P["bq"])), ARG),
    (dict(q=side(kind=NONE, weight=P["wq"])), ARG),
    (dict(q=side(x=P["q"] + 8)), ALIGN), (dict(q=side(y=P["yq"] + 2)), ALIGN),
    (dict(q=side(weight=P["wq"] + 8)), ALIGN),
    (dict(table=P["table"] + 4), ALIGN),
    (dict(row=P["row"] + 2, rows=7), ALIGN),
    (dict(q=side(y=P["q"] + 64)), ALIAS),
    (dict(q=side(y=P["q"], y_stride=1024)), ALIAS),
    (dict(q=side(y=P["k"])), ALIAS), (dict(q=side(y=P["yk"])), ALIAS),
    (dict(q=side(y=P["wk"])), ALIAS), (dict(q=side(y=P["table"])), ALIAS),
    (dict(q=side(y=P["row"]), row=P["row"], rows=7), ALIAS),
    # parts of one row that share values
    (dict(q=side(x_stride=640, y_stride=640, y=P["q"]),
          k=side("k", 2, x=P["q"] + 1008, y=P["yk"], x_stride=640)), ALIAS),
    (dict(q=side(x_stride=640, y_stride=640, y=P["q"]),
          k=side("k", 2, x=P["q"] + 1040, y=P["yk"], x_stride=640)), ALIAS),
])
def test_heads_reject(kw, code):
    assert heads(**kw) == code


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def attend_arg(Hq=8, Hk=2, D=64, **kw):
    a = B._Attention(P["q"], P["k"], P["v"], P["out"], Hq * D, Hk * D, Hk * D,
                     Hq * D, 100, 300, 1, Hq, Hk, D, None, None, None, 0.125)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def attend(ws=P["ws"], bytes=1 << 36, **kw):
    return B.lib().w8a8_attention(attend_arg(**kw), ws, bytes, None)


@no_gpu
@pytest.mark.parametrize("kw", [
    {}, dict(Tk=0, k=None, v=None), dict(B=4), dict(B=100, Tk=0),
    dict(B=7, q_offsets=P["qo"], k_offsets=P["ko"], k_lens=P["kl"]),
    dict(B=1 << 20, q_offsets=P["qo"], k_offsets=P["ko"]),
    dict(Hq=1, Hk=1, D=8, Tq=1, Tk=1), dict(D=128),
    dict(q_stride=(1 << 22) - 8, k_stride=(1 << 22) - 8),
    dict(k=P["q"], v=P["q"]), dict(scale=1e-30),
    dict(Tq=(1 << 28) - 512, Tk=(1 << 30) - 1),
    # out beside q, k, v in the rows of one buffer
    dict(k=P["q"] + 1024, v=P["q"] + 1280, out=P["q"] + 1536, q_stride=1280,
         k_stride=1280, v_stride=1280, out_stride=1280),
])
def test_attention_valid_calls_reach_the_device_check(kw):
    assert attend(**kw) == DEVICE


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL),
    (dict(out=None), NULL),
    (dict(Tq=0), SHAPE), (dict(Tk=-1), SHAPE), (dict(B=0), SHAPE),
    (dict(B=(1 << 20) + 1, q_offsets=P["qo"], k_offsets=P["ko"]), SHAPE),
    (dict(B=3), SHAPE), (dict(B=8, q_offsets=P["qo"]), SHAPE),
    (dict(D=0), SHAPE), (dict(D=136), SHAPE), (dict(D=60), SHAPE),
    (dict(q_heads=0), SHAPE), (dict(k_heads=0), SHAPE), (dict(k_heads=3), SHAPE),
    (dict(q_heads=-8, k_heads=-2), SHAPE), (dict(q_stride=504), SHAPE),
    (dict(k_stride=124), SHAPE), (dict(v_stride=1 << 22), SHAPE),
    (dict(out_stride=516), SHAPE), (dict(Tq=1 << 28), SHAPE),
    (dict(Tk=1 << 30), SHAPE), (dict(Tq=1 << 40), SHAPE),
    (dict(q_heads=1 << 62, k_heads=1 << 62), SHAPE),
    (dict(scale=0.0), ARG), (dict(scale=-1.0), ARG),
    (dict(scale=math.inf), ARG), (dict(scale=math.nan), ARG),
    (dict(q=P["q"] + 8), ALIGN), (dict(k=P["k"] + 2), ALIGN),
    (dict(v=P["v"] + 4), ALIGN), (dict(out=P["out"] + 8), ALIGN),
    (dict(B=4, q_offsets=P["qo"] + 2), ALIGN),
    (dict(B=4, k_offsets=P["ko"] + 1), ALIGN),
    (dict(B=4, k_lens=P["kl"] + 2), ALIGN),
    (dict(out=P["q"]), ALIAS), (dict(out=P["k"] + 64), ALIAS),
    (dict(out=P["v"]), ALIAS),
    (dict(B=4, k_lens=P["out"] + 64), ALIAS),
    (dict(B=4, q_offsets=P["out"]), ALIAS),
    (dict(out=P["q"] + 1008, q_stride=2048, out_stride=2048), ALIAS),
])
def test_attention_rejects(kw, code):
    assert attend(**kw) == code


def test_attention_workspace():
    few = dict(Tq=1, Tk=20000)
    need = B.lib().w8a8_attention_workspace_bytes(attend_arg(**few))
    assert need > 0
    assert need == B.attention_workspace_bytes(1, 20000, 8, 2, 64)
    assert attend(ws=None, bytes=0, **few) == WORKSPACE
    assert attend(bytes=need - 1, **few) == WORKSPACE
    assert attend(ws=P["ws"] + 8, **few) == ALIGN
    for name in ("q", "k", "v", "out"):
        assert attend(ws=P[name], **few) == ALIAS
    assert attend(ws=P["kl"] - 16, k_lens=P["kl"], **few) == ALIAS
    # none where nothing is split, and for what is refused
    assert B.attention_workspace_bytes(20000, 512, 56, 56, 128) == 0
    assert B.lib().w8a8_attention_workspace_bytes(attend_arg(B=3)) == 0
    assert B.lib().w8a8_attention_workspace_bytes(None) == 0
    if torch.cuda.device_count() == 0:
        assert attend(ws=None, bytes=0, Tq=20000, Tk=512) == DEVICE


def test_workspace_does_not_depend_on_what_the_offsets_hold():
    for B_, packed in ((1, False), (4, False), (4, True), (1000, True)):
        a = attend_arg(Tq=4000, Tk=40000, B=B_, k_offsets=P["ko"],
                       q_offsets=P["qo"] if packed else None)
        assert B.lib().w8a8_attention_workspace_bytes(a) == \
            B.attention_workspace_bytes(4000, 40000, 8, 2, 64, B=B_,
                                        packed=packed)


def test_binding_refuses_what_is_not_on_a_gpu():
    t = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="on the GPU"):
        B.attention(t, t, t)
    with pytest.raises(ValueError, match="on the GPU"):
        B.head_norm_rope(t)
    with pytest.raises(ValueError, match="on the GPU"):
        B.rope_table(torch.zeros(4, dtype=torch.int32), 8)
    for call in (lambda: B.attention(None, t, t), lambda: B.rope(None, t),
                 lambda: B.rope_table([1, 2], 8)):
        with pytest.raises(TypeError):
            call()
