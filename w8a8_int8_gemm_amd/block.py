"""One DiT block's six W8A8 projections, composed from library calls.

Data flow of a block (the six quantized Linears of "feat(mps): support
MiniMax-H3 INT8 inference on Apple M5", LightX2V pull request #1672,
description): Q, K and V share one per-token quantization of the block
input; the attention output projection and FC1 each quantize their own
input; FC2 takes SiLU of FC1's BF16 output, quantized ("MLX implementation
and experiment report", "What the default preserves": SiLU applied to the
BF16 value, rounded per the original recipe).  Attention and the norms are
not part of the projection path, so the synthetic block (``BlockRunner``)
feeds its input X to O and FC1 as well; that keeps four quantizations per
block, as in the model.  ``NormedBlock`` has the norms, and the attention
where its heads are described.  Everything here is a sequence of library calls on one stream;
outputs and scratch are preallocated once per token count.  The pages' own
H3 shapes (see datagen) use SwiGLU over a fused gate | up FC1 and feed V's
output (the attention result's shape) to the attention output projection.

Fused QKV (optional): the Q, K and V weights concatenated along the output
channels, [3N, K] with their scales and biases, run as one GEMM on the
shared quantized input.  Every output column depends only on its own weight
row, so the three column blocks of the fused output equal the separate
outputs bit for bit; the larger N fills the chip in fewer, fuller waves.
"""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np

from . import binding as B
from . import datagen as D


def to_device_bf16(bits: np.ndarray, device="cuda"):
    import torch
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(
        torch.bfloat16).to(device)


def from_device_bf16(t) -> np.ndarray:
    import torch
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


@dataclass
class DeviceProj:
    name: str
    N: int
    K: int
    w: object      # int8 [N, K]
    sw: object     # float32 [N]
    bias: object   # bf16 [N]


def upload_proj(p: D.Proj, pp: D.ProjParams, device="cuda") -> DeviceProj:
    import torch
    return DeviceProj(p.name, p.N, p.K,
                      torch.from_numpy(pp.w).to(device),
                      torch.from_numpy(pp.sw).to(device),
                      to_device_bf16(pp.bias, device))


def fuse_qkv(projs: dict) -> dict:
    """Replace projs' q, k, v by one "qkv" projection [3N, K] (device
    tensors concatenated along the output channels)."""
    import torch
    q, k, v = projs["q"], projs["k"], projs["v"]
    assert q.K == k.K == v.K
    fused = DeviceProj("qkv", q.N + k.N + v.N, q.K,
                       torch.cat([q.w, k.w, v.w]), torch.cat([q.sw, k.sw, v.sw]),
                       torch.cat([q.bias, k.bias, v.bias]))
    out = {n: p for n, p in projs.items() if n not in ("q", "k", "v")}
    out["qkv"] = fused
    return out


class BlockRunner:
    """Preallocated buffers for one token count M and one block layout
    (``projs``: the workload's six projections; ``mlp``: "silu", or
    "swiglu" for a fused gate | up FC1; ``o_input``: "x", or "v" to feed
    V's output to the attention output projection).  ``run`` enqueues the
    block's kernels on the current stream (or ``stream``).  ``on_gemm`` is
    called around every GEMM launch and ``on_quant`` around every
    quantization (for per-kernel event timing), as ``f(name, phase)``."""

    def __init__(self, M: int, device="cuda", fused_qkv: bool = False,
                 projs=D.BLOCK_PROJS, mlp: str = "silu", o_input: str = "x"):
        import torch
        if fused_qkv and o_input != "x":
            raise ValueError("fused QKV needs the block input as O's input")
        self.M, self.mlp, self.o_input = M, mlp, o_input
        shape = {p.name: (p.N, p.K) for p in projs}
        H = shape["q"][1]  # block width
        e = lambda *s, dt: torch.empty(s, dtype=dt, device=device)
        # X quantized for Q/K/V, for O (when it reads X) and for FC1
        self.xq = [e(M, H, dt=torch.int8) for _ in range(3)]
        self.xs = [e(M, dt=torch.float32) for _ in range(3)]
        self.oq = (e(M, shape["o"][1], dt=torch.int8) if o_input == "v"
                   else None)
        self.hq = e(M, shape["fc2"][1], dt=torch.int8)
        self.hs = e(M, dt=torch.float32)
        self.out = {n: e(M, shape[n][0], dt=torch.bfloat16)
                    for n in ("o", "fc1", "fc2")}
        if fused_qkv:
            nq = shape["q"][0]
            self.out["qkv"] = e(M, 3 * nq, dt=torch.bfloat16)
            for i, n in enumerate(("q", "k", "v")):
                self.out[n] = self.out["qkv"][:, i * nq:(i + 1) * nq]
        else:
            for n in ("q", "k", "v"):
                self.out[n] = e(M, shape[n][0], dt=torch.bfloat16)
        need = [B.gemm_workspace_bytes(M, N, K) for N, K in shape.values()]
        need.append(B.gemm_workspace_bytes(M, 3 * shape["q"][0], H))
        self.ws = e(max(max(need), 256), dt=torch.uint8)

    def _gemm(self, projs, name, q, s, stream, on_gemm):
        p = projs[name]
        if on_gemm:
            on_gemm(name, "begin")
        B.gemm(q, s, p.w, p.sw, p.bias, out=self.out[name],
               workspace=self.ws, stream=stream)
        if on_gemm:
            on_gemm(name, "end")

    def run_gemms(self, projs: dict, stream=None, on_gemm=None):
        """Only the block's GEMM calls, on the codes and scales the last
        ``run`` left in the buffers (GEMM timing)."""
        for n in (("qkv",) if "qkv" in projs else ("q", "k", "v")):
            self._gemm(projs, n, self.xq[0], self.xs[0], stream, on_gemm)
        self._gemm(projs, "o", self.oq if self.o_input == "v" else self.xq[1],
                   self.xs[1], stream, on_gemm)
        self._gemm(projs, "fc1", self.xq[2], self.xs[2], stream, on_gemm)
        self._gemm(projs, "fc2", self.hq, self.hs, stream, on_gemm)
        return self.out

    def codes_by_projection(self, projs: dict) -> dict:
        """The INT8 input codes each projection of ``projs`` read in the
        last ``run`` (the buffers, not copies)."""
        src = {"q": self.xq[0], "k": self.xq[0], "v": self.xq[0],
               "qkv": self.xq[0],
               "o": self.oq if self.o_input == "v" else self.xq[1],
               "fc1": self.xq[2], "fc2": self.hq}
        return {n: src[n] for n in projs}

    def run(self, x, projs: dict, stream=None, on_gemm=None,
            x_quantized: bool = False, on_quant=None):
        """x: bf16 [M, H].  Returns the dict of BF16 outputs.  With
        ``x_quantized`` the buffers ``xq[0]``, ``xs[0]`` already hold the
        quantization of x (written together with x by
        ``pow2_renorm_quantize`` between blocks) and Q, K and V use them."""
        def gemm(name, q, s):
            self._gemm(projs, name, q, s, stream, on_gemm)

        def quant(name, fn, *a, **kw):
            if on_quant:
                on_quant(name, "begin")
            fn(*a, stream=stream, **kw)
            if on_quant:
                on_quant(name, "end")

        # Q, K, V: one shared quantization of the block input (and, fused,
        # one GEMM over the concatenated weights).
        if not x_quantized:
            quant("quant", B.quantize_act, x, out=(self.xq[0], self.xs[0]))
        for n in (("qkv",) if "qkv" in projs else ("q", "k", "v")):
            gemm(n, self.xq[0], self.xs[0])
        # attention output projection and FC1 quantize their own inputs.
        if self.o_input == "v":
            quant("quant_o", B.quantize_act, self.out["v"],
                  out=(self.oq, self.xs[1]))
            gemm("o", self.oq, self.xs[1])
        else:
            quant("quant", B.quantize_act, x, out=(self.xq[1], self.xs[1]))
            gemm("o", self.xq[1], self.xs[1])
        quant("quant", B.quantize_act, x, out=(self.xq[2], self.xs[2]))
        gemm("fc1", self.xq[2], self.xs[2])
        # FC2 input: SiLU (or SwiGLU of gate | up) of FC1's BF16 output,
        # quantized in the same pass.
        if self.mlp == "swiglu":
            quant("swiglu_quant", B.quantize_act_swiglu, self.out["fc1"],
                  out=(self.hq, self.hs))
        else:
            quant("silu_quant", B.quantize_act, self.out["fc1"], silu=True,
                  out=(self.hq, self.hs))
        gemm("fc2", self.hq, self.hs)
        return self.out


# ---------------------------------------------------------------------------
# a block with its norms, gates and residuals
# ---------------------------------------------------------------------------

@dataclass
class DeviceProj4:
    """A projection with packed 4-bit weights, for a few tokens."""
    name: str
    N: int
    K: int
    w4: object        # uint8 [N/16, K/128, 64, 16]
    w4_scale: object  # bf16 [N/16, K/128, 16, 128/group]
    bias: object      # bf16 [N]


def to_four_bit(p: DeviceProj, group: int = 128) -> DeviceProj4:
    """The 4-bit form of an INT8 projection (its weights w * sw in BF16
    through the converter)."""
    import torch
    w = (p.w.float() * p.sw[:, None]).to(torch.bfloat16)
    return DeviceProj4(p.name, p.N, p.K, *B.w4_quantize_weight(w, group=group),
                       p.bias)


@dataclass
class BlockNorms:
    """What stands between a block's projections (every vector bf16 [H] or
    None).  ``table`` bf16 [rows, 6 H] holds the modulation of a row as
    shift, scale and gate of the attention side, then of the MLP side;
    ``mod_row`` int32 [M] names each token's row (None: one row for all, or
    one for each token; a row outside the table marks a padding token)."""
    table: object
    mod_row: object = None
    norm: str = "rms"             # in front of Q, K, V and of FC1
    weight: tuple = (None, None)
    bias: tuple = (None, None)
    post_norm: str = "none"       # behind the attention output and FC2
    post_weight: tuple = (None, None)
    post_bias: tuple = (None, None)
    residual_scale: float = 1.0
    eps: float = 1e-6

    def before(self, side: int) -> dict:
        """Keywords of the norm in front of side 0 (attention) or 1 (MLP)."""
        H = self.table.shape[1] // 6
        at = 3 * side * H
        return dict(norm=self.norm, weight=self.weight[side],
                    bias=self.bias[side], eps=self.eps,
                    shift=self.table[:, at:at + H],
                    scale=self.table[:, at + H:at + 2 * H])

    def behind(self, side: int) -> dict:
        """Keywords of the gate and residual behind that side."""
        H = self.table.shape[1] // 6
        at = (3 * side + 2) * H
        return dict(post_norm=self.post_norm,
                    post_weight=self.post_weight[side],
                    post_bias=self.post_bias[side], post_eps=self.eps,
                    residual_scale=self.residual_scale,
                    gate=self.table[:, at:at + H])


@dataclass
class BlockHeads:
    """A block's attention: heads of ``width`` values (as many as Q's and K's
    outputs hold; several query heads may share a key head), their norms (each
    vector bf16 [width], [heads, width] or None), the rotation of queries and
    keys (``table`` float32 [rows, 2, pairs] of ``binding.rope_table``, ``row``
    int32 [M]) and the sequences (``binding.attention``'s offsets and key
    lengths; without them all tokens are one sequence, or ``batch`` equal ones).
    A padding token of the norms is a key like any other unless the offsets or
    lengths leave it out.  Tokens of no sequence (offsets that do not cover all
    of them) have an attention of zeros."""
    width: int
    norm: str = "rms"
    q_weight: object = None
    k_weight: object = None
    q_bias: object = None
    k_bias: object = None
    eps: float = 1e-6
    table: object = None
    row: object = None
    interleaved: bool = False
    scale: object = None
    batch: int = 1
    q_offsets: object = None
    k_offsets: object = None
    k_lens: object = None

    def check(self, context: bool):
        """Refuses what the block would not use."""
        if context and (self.table is not None or self.row is not None):
            raise ValueError("a context's keys are not turned")
        if self.row is not None and self.table is None:
            raise ValueError("row needs a table")
        if self.norm == "none" and any(
                t is not None for t in (self.q_weight, self.k_weight,
                                        self.q_bias, self.k_bias)):
            raise ValueError("weights and biases need a norm")


class NormedBlock:
    """A whole block: norm and modulation, Q, K, V, the attention, its output
    projection, gate and residual, the next norm, the MLP, gate and residual.
    Buffers are preallocated for one token count.  With ``four_bit`` the
    projections are DeviceProj4 and activations stay BF16 (a few tokens);
    otherwise DeviceProj, and the norms write INT8 codes.

    ``heads`` describes the attention; without it V's output (the attention
    result's shape) feeds the output projection.  With ``context_tokens`` the
    attention is one to other states (an encoder's): K and V read the
    ``context`` given to ``run``, bf16 [context_tokens, K's inputs], whose keys
    are normed but not turned."""

    def __init__(self, M: int, projs=D.BLOCK_PROJS, mlp: str = "silu",
                 four_bit: bool = False, device="cuda", heads=None,
                 context_tokens=None):
        import torch
        self.M, self.mlp, self.four_bit = M, mlp, four_bit
        self.heads, self.context_tokens = heads, context_tokens
        shape = {p.name: (p.N, p.K) for p in projs}
        H = shape["q"][1]
        bf, i8, f32 = torch.bfloat16, torch.int8, torch.float32
        e = lambda *s, dt=bf: torch.empty(s, dtype=dt, device=device)
        Mk = M if context_tokens is None else context_tokens
        self.out = {n: e(Mk if n in ("k", "v") else M, N)
                    for n, (N, _) in shape.items()}
        self.r = e(M, H)
        if heads is None:
            if context_tokens is not None:
                raise ValueError("context_tokens needs heads")
        else:
            heads.check(context_tokens is not None)
            self.a = e(M, shape["q"][0])
            self.aws = e(max(B.attention_workspace_bytes(
                M, Mk, shape["q"][0] // heads.width,
                shape["k"][0] // heads.width, heads.width, B=self._batch(),
                packed=heads.q_offsets is not None), 16), dt=torch.uint8)
        if four_bit:
            self.y = e(M, H)
            self.h = e(M, shape["fc2"][1])
            return
        self.yq, self.ys = e(M, H, dt=i8), e(M, dt=f32)
        self.oq, self.os = e(M, shape["o"][1], dt=i8), e(M, dt=f32)
        self.hq, self.hs = e(M, shape["fc2"][1], dt=i8), e(M, dt=f32)
        if context_tokens is not None:
            self.cq, self.cs = e(Mk, shape["k"][1], dt=i8), e(Mk, dt=f32)
        need = max(B.gemm_workspace_bytes(m, N, K) for N, K in shape.values()
                   for m in (M, Mk))
        self.ws = e(max(need, 256), dt=torch.uint8)

    def _batch(self) -> int:
        h = self.heads
        if h.k_lens is not None:
            return h.k_lens.shape[0]
        for o in (h.q_offsets, h.k_offsets):
            if o is not None:
                return o.shape[0] - 1
        return h.batch

    def run(self, x, projs: dict, norms: BlockNorms, out=None, stream=None,
            context=None):
        """x: bf16 [M, H] -> bf16 [M, H] (``out``, or a new tensor)."""
        if (context is None) != (self.context_tokens is None):
            raise ValueError("context goes with context_tokens")
        run = self._run4 if self.four_bit else self._run8
        rows = dict(mod_row=norms.mod_row, stream=stream)
        return run(x, projs, norms, rows, out, stream, context)

    @staticmethod
    def _zero(t, stream):
        import torch
        if stream is None:
            t.zero_()
            return
        with torch.cuda.stream(stream):
            t.zero_()

    def _attend(self, stream):
        """The attention of the block's Q, K, V outputs (queries and keys are
        normed and turned where they lie), or V's output without heads."""
        h = self.heads
        if h is None:
            return self.out["v"]
        h.check(self.context_tokens is not None)
        q, k, v = (self.out[n].unflatten(1, (-1, h.width)) for n in "qkv")
        shared = dict(norm=h.norm, eps=h.eps, stream=stream)
        turn = dict(table=h.table, row=h.row, interleaved=h.interleaved)
        qv = dict(q_weight=h.q_weight, q_bias=h.q_bias)
        if self.context_tokens is None:
            if h.norm != "none" or h.table is not None:
                B.head_norm_rope(q, k, k_weight=h.k_weight, k_bias=h.k_bias,
                                 out=(q, k), **qv, **shared, **turn)
        elif h.norm != "none":
            B.head_norm_rope(q, out=q, **qv, **shared)
            B.head_norm_rope(k, q_weight=h.k_weight, q_bias=h.k_bias, out=k,
                             **shared)
        if h.q_offsets is not None:
            # Rows of no sequence, which the attention leaves as they are.
            self._zero(self.a, stream)
        a = self.a.unflatten(1, (-1, h.width))
        if h.batch > 1 and h.q_offsets is None and h.k_offsets is None:
            q, k, v, a = (t.unflatten(0, (h.batch, -1)) for t in (q, k, v, a))
        B.attention(q, k, v, scale=h.scale, q_offsets=h.q_offsets,
                    k_offsets=h.k_offsets, k_lens=h.k_lens, out=a,
                    workspace=self.aws, stream=stream)
        return self.a

    def _run8(self, x, projs, norms, rows, out, stream, context):
        def gemm(name, q, s):
            p = projs[name]
            B.gemm(q, s, p.w, p.sw, p.bias, out=self.out[name],
                   workspace=self.ws, stream=stream)

        y = (self.yq, self.ys)
        B.norm_modulate_quantize(x, **norms.before(0), **rows, out=y)
        keys = y
        if context is not None:
            keys = (self.cq, self.cs)
            B.quantize_act(context, out=keys, stream=stream)
        for n in ("q", "k", "v"):
            gemm(n, *(y if n == "q" else keys))
        B.quantize_act(self._attend(stream), out=(self.oq, self.os),
                       stream=stream)
        gemm("o", self.oq, self.os)
        B.gated_residual_norm_quantize(
            x, self.out["o"], **norms.behind(0), **norms.before(1), **rows,
            out=(self.r, *y))
        gemm("fc1", *y)
        h = (self.hq, self.hs)
        if self.mlp == "swiglu":
            B.quantize_act_swiglu(self.out["fc1"], out=h, stream=stream)
        else:
            B.quantize_act(self.out["fc1"], silu=True, out=h, stream=stream)
        gemm("fc2", *h)
        return B.gated_residual(self.r, self.out["fc2"], **norms.behind(1),
                                **rows, out=out)

    def _run4(self, x, projs, norms, rows, out, stream, context):
        def linear(name, a):
            p = projs[name]
            B.w4_linear(a, p.w4, p.w4_scale, p.bias, out=self.out[name],
                        stream=stream)

        B.norm_modulate(x, **norms.before(0), **rows, out=self.y)
        for n in ("q", "k", "v"):
            linear(n, self.y if n == "q" or context is None else context)
        linear("o", self._attend(stream))
        B.gated_residual_norm(x, self.out["o"], **norms.behind(0),
                              **norms.before(1), **rows,
                              out=(self.r, self.y))
        linear("fc1", self.y)
        act = B.swiglu if self.mlp == "swiglu" else B.silu
        act(self.out["fc1"], out=self.h, stream=stream)
        linear("fc2", self.h)
        return B.gated_residual(self.r, self.out["fc2"], **norms.behind(1),
                                **rows, out=out)
