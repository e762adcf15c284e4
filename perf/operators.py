"""Cases of the block norms and of the 4-bit linear: what is measured of them.

Three kinds of case, each a call that a transformer block makes around its
projections:

* ``norm``: the norm before a projection, modulated per token, to BF16 or to
  INT8 codes with per-token scales;
* ``residual``: the norm after a projection, its gate and the scaled residual
  sum, alone or followed by the next norm (to BF16 or to INT8 codes);
* ``w4``: a Linear over few tokens with packed 4-bit weights and group scales.

``own`` selects the library's calls; otherwise the same outputs come from
elementary torch operations in 32 bits.  INT8 codes are returned as the values
they stand for, in BF16.
"""
import math

import torch

own = False

# Rows of a norm case and the width of its rows; tokens of a w4 case.
MAX_ROW_VALUES = 37503 * 5376
MAX_WEIGHTS = 28672 * 5376


def listed():
    return [
        # One token through a block's first norm: the latency of a launch.
        _norm("norm_one_token", 1, 5376, "rms", affine=True, mods=1),
        # 544x960, 124 frames: every latent frame and the audio tokens have
        # their own shift and scale; layer norm without weights.
        _norm("norm_per_frame", 19077, 5376, "layer", affine=False, mods=38),
        # A serving batch of 64 tokens, straight to a projection's codes.
        _norm("norm_quantize_64", 64, 5376, "rms", affine=True, mods=64,
              quantize=True),
        # 768x1344, 124 frames, to a projection's codes: the longest input.
        _norm("norm_quantize_longest", 37503, 5376, "rms", affine=True,
              mods=75, quantize=True),
        # One token at the width of 56 heads of 128, both norms.
        _residual("residual_norm_one_token", 1, 7168, "rms", "rms", mods=1),
        # A ragged, padded batch of a narrow model: residual alone.
        _residual("residual_odd", 301, 1000, "layer", "none", mods=301,
                  padded=True),
        # 4096 tokens, norms on both sides of the projection.
        _residual("residual_norm_4096", 4096, 5376, "rms", "rms", mods=4),
        # 544x960, 124 frames, no norm behind the projection, codes for the
        # next one; the last tokens are padding.
        _residual("residual_quantize_per_frame", 19077, 5376, "none", "layer",
                  mods=38, quantize=True, padded=True),
        # One token, square projection: the smallest weight stream.
        _w4("w4_one_token", 1, 5376, 5376, 128),
        # One token, fused gate | up projection: the longest weight stream.
        _w4("w4_one_token_gate_up", 1, 28672, 5376, 128),
        # A handful of tokens, middle groups.
        _w4("w4_8_tokens", 8, 21504, 5376, 64),
        # 64 tokens, long rows, the smallest groups.
        _w4("w4_64_tokens", 64, 5376, 21504, 32),
    ]


def _norm(name, M, H, norm, affine, mods, quantize=False, padded=False):
    return {"name": name, "kind": "norm", "M": M, "H": H, "norm": norm,
            "affine": affine, "mods": mods, "quantize": quantize,
            "padded": padded}


def _residual(name, M, H, post, norm, mods, quantize=False, padded=False):
    return {"name": name, "kind": "residual", "M": M, "H": H, "post": post,
            "norm": norm, "affine": True, "mods": mods, "quantize": quantize,
            "padded": padded}


def _w4(name, M, N, K, group):
    return {"name": name, "kind": "w4", "M": M, "N": N, "K": K,
            "group": group}


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(["norm", "residual", "w4"])
    if kind == "w4":
        K = 128 * _spread(rng, 1, 168)
        N = 16 * _spread(rng, 1, min(1792, MAX_WEIGHTS // (16 * K)))
        c = _w4("", _spread(rng, 1, 64), N, K, rng.choice([32, 64, 128]))
    else:
        H = 8 * _spread(rng, 8, 2048)
        # A residual moves up to twice what a norm does, and a modulation
        # row for every token as much again.
        M = _spread(rng, 1, min(37503, MAX_ROW_VALUES // H) // 4)
        mods = rng.choice([1, min(M, 1 + rng.randrange(64)), M])
        quantize, padded = rng.random() < 0.5, rng.random() < 0.5
        if kind == "norm":
            c = _norm("", M, H, rng.choice(["rms", "layer"]),
                      rng.random() < 0.5, mods, quantize, padded)
        else:
            norm = rng.choice(["none", "rms", "layer"])
            c = _residual("", M, H, rng.choice(["none", "rms", "layer"]),
                          norm, mods, quantize and norm != "none", padded)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _activations(g, M, H):
    """Standard normal, one entry in a thousand 20 times larger, in BF16."""
    x = torch.randn(M, H, generator=g, device="cuda")
    big = torch.rand(M, H, generator=g, device="cuda") < 0.001
    return torch.where(big, 20 * x, x).to(torch.bfloat16)


def _normal(g, *shape, mean=0.0, std=1.0):
    return (mean + std * torch.randn(*shape, generator=g, device="cuda")).to(
        torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    s = dict(case)
    M = case["M"]
    if case["kind"] == "w4":
        N, K, G = case["N"], case["K"], case["group"]
        s["x"] = _activations(g, M, K)
        # packed codes: 16 channels x 128 inputs a block, 64 lanes x 16 bytes
        s["w4"] = torch.randint(0, 256, (N // 16, K // 128, 64, 16),
                                generator=g, device="cuda", dtype=torch.uint8)
        s["w4_scale"] = torch.exp(-4.0 + 0.3 * torch.randn(
            N // 16, K // 128, 16, 128 // G, generator=g, device="cuda")).to(
                torch.bfloat16)
        s["bias"] = _normal(g, N, std=0.02)
        return s
    H, R = case["H"], case["mods"]
    s["x"] = _activations(g, M, H)
    # One modulation row per frame or token, its parts side by side.
    table = _normal(g, R, 3 * H, std=0.25)
    s["shift"], s["scale"], s["gate"] = table.split(H, dim=1)
    s["weight"] = s["bias"] = s["post_weight"] = s["post_bias"] = None
    if case["affine"]:
        s["weight"] = _normal(g, H, mean=1.0, std=0.1)
        if case["norm"] == "layer":
            s["bias"] = _normal(g, H, std=0.1)
    if case["kind"] == "residual":
        s["branch"] = _activations(g, M, H)
        if case["post"] != "none":
            s["post_weight"] = _normal(g, H, mean=1.0, std=0.1)
        if case["post"] == "layer":
            s["post_bias"] = _normal(g, H, std=0.1)
    # Token -> modulation row: runs of equal rows, and none (-1) for padding.
    s["mod_row"] = None
    if case["padded"] or R not in (1, M):
        row = torch.arange(M, device="cuda") * R // M
        if case["padded"]:
            row[M - M // 16:] = -1
        s["mod_row"] = row.to(torch.int32)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    if s["kind"] == "w4":
        return _plain_w4(s)
    return _plain_rows(s)


def _run_own(s):
    from w8a8_int8_gemm_amd import binding as B
    if s["kind"] == "w4":
        return B.w4_linear(s["x"], s["w4"], s["w4_scale"], s["bias"])
    mods = {"mod_row": s["mod_row"]}
    if s["norm"] != "none":
        mods.update(norm=s["norm"], weight=s["weight"], bias=s["bias"],
                    scale=s["scale"], shift=s["shift"])
    if s["kind"] == "norm":
        if not s["quantize"]:
            return B.norm_modulate(s["x"], **mods)
        return _values(*B.norm_modulate_quantize(s["x"], **mods))
    mods.update(gate=s["gate"], residual_scale=0.5, post_norm=s["post"],
                post_weight=s["post_weight"], post_bias=s["post_bias"])
    if s["norm"] == "none":
        return B.gated_residual(s["x"], s["branch"], **mods)
    if not s["quantize"]:
        return B.gated_residual_norm(s["x"], s["branch"], **mods)
    r, q, a = B.gated_residual_norm_quantize(s["x"], s["branch"], **mods)
    return r, _values(q, a)


def _values(q, a):
    """INT8 codes and their per-token scales -> the values, in BF16."""
    v = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    return torch.mul(q, a[:, None], out=v)


EPS = 1e-6


def _plain_norm(v, kind, weight, bias):
    if kind == "none":
        return v
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    v = v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)
    if weight is not None:
        v = v * weight.float()
    if bias is not None:
        v = v + bias.float()
    return v


def _plain_mod(t, row):
    """The tokens' rows of a modulation table, in 32 bits."""
    if row is not None:
        t = t[row.long().clamp_min(0)]
    return t.float()


def _plain_rows(s):
    x, row = s["x"], s["mod_row"]
    live = None if row is None else (row >= 0)[:, None]
    out = []
    v = x.float()
    if s["kind"] == "residual":
        b = _plain_norm(s["branch"].float(), s["post"], s["post_weight"],
                        s["post_bias"])
        r = 0.5 * v + _plain_mod(s["gate"], row) * b
        v = r if live is None else torch.where(live, r, v)
        out.append(v.to(torch.bfloat16))
    if s["norm"] != "none":
        y = _plain_norm(v, s["norm"], s["weight"], s["bias"])
        y = (y * (1 + _plain_mod(s["scale"], row)) +
             _plain_mod(s["shift"], row))
        if live is not None:
            y = torch.where(live, y, torch.zeros_like(y))
        if s["quantize"]:
            a = y.abs().amax(1, keepdim=True) / 127
            q = torch.round(y / torch.where(a > 0, a, torch.ones_like(a)))
            y = q.clamp(-127, 127) * a
        out.append(y.to(torch.bfloat16))
    return out[0] if len(out) == 1 else tuple(out)


def _plain_w4(s):
    N, K, G = s["N"], s["K"], s["group"]
    p = s["w4"]
    u = torch.stack([p & 15, p >> 4], -1)   # a byte's low and high code
    # block bytes [4 x 16 lanes][4 dwords][4 bytes][2] hold channel = lane
    # % 16 and input = 32 * dword + 8 * (lane / 16) + 4 * half + byte
    u = u.view(N // 16, K // 128, 4, 16, 4, 4, 2).permute(0, 3, 1, 4, 2, 6, 5)
    w = u.reshape(N, K // G, G).float() - 8
    w = w * s["w4_scale"].float().permute(0, 2, 1, 3).reshape(N, K // G, 1)
    y = s["x"].float() @ w.view(N, K).t() + s["bias"].float()
    return y.to(torch.bfloat16)


# ---------------------------------------------------------------------------
# the work of a pass, and its result in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    M = case["M"]
    if case["kind"] == "w4":
        N, K, G = case["N"], case["K"], case["group"]
        return {"bytes": N * K // 2 + 2 * N * K // G + 2 * M * K +
                2 * M * N + 2 * N, "flops": 2 * M * N * K}
    H, R = case["H"], case["mods"]
    res, has_norm = case["kind"] == "residual", case["norm"] != "none"
    # per value: inputs, the residual written, the norm's output
    per = 2 + (4 if res else 0) + (
        (1 if case["quantize"] else 2) if has_norm else 0)
    vectors = (1 if res else 0) + (2 if has_norm else 0)
    size = M * H * per + 2 * R * H * vectors
    size += 2 * H * ((1 if case["affine"] and has_norm else 0) +
                     (1 if res and case["post"] != "none" else 0))
    size += 4 * M * (1 if case["quantize"] else 0)
    return {"bytes": size, "flops": M * H * (12 if res and has_norm else 8)}


def _norm64(v, kind, weight, bias):
    """sqrt(H) * v / sqrt(|v|^2 + H eps), v less its mean for a layer norm."""
    if kind == "none":
        return v
    n = v.shape[1]
    if kind == "layer":
        v = v - (v.sum(1) / n).unsqueeze(1)
    length = (torch.linalg.vecdot(v, v) + n * 1e-6).sqrt()
    v = v * (math.sqrt(n) / length).unsqueeze(1)
    if weight is not None:
        v = v * weight.double()
    return v if bias is None else v + bias.double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "w4":
        return _exact_w4(s)
    M, H = case["M"], case["H"]
    x = s["x"].double()
    table = s["mod_row"]
    if table is None:
        at = torch.zeros(M, dtype=torch.int64, device=x.device)
        if case["mods"] == M:
            at = torch.arange(M, device=x.device)
    else:
        at = table.long()
    dead = at < 0
    at = torch.where(dead, torch.zeros_like(at), at)
    got = []
    v = x
    if case["kind"] == "residual":
        v = torch.addcmul(0.5 * x, s["gate"].double()[at], _norm64(
            s["branch"].double(), case["post"], s["post_weight"],
            s["post_bias"]))
        v[dead] = x[dead]
        got.append(v)
    if case["norm"] != "none":
        y = torch.addcmul(
            s["shift"].double()[at], 1 + s["scale"].double()[at],
            _norm64(v, case["norm"], s["weight"], s["bias"]))
        y[dead] = 0
        if case["quantize"]:
            step = y.abs().max(1).values / 127
            y = y / step.clamp_min(1e-300).unsqueeze(1)
            y = y.round().clamp(-127, 127) * step.unsqueeze(1)
        got.append(y)
    return got[0] if len(got) == 1 else tuple(got)


def _exact_w4(s):
    N, K, G = s["N"], s["K"], s["group"]
    dev = s["x"].device
    n = torch.arange(N, device=dev)[:, None]
    k = torch.arange(K, device=dev)[None, :]
    # where the code of channel n and input k lies
    lane = ((k % 32) // 8) * 16 + n % 16
    byte = ((k % 128) // 32) * 4 + k % 4
    code = s["w4"][n // 16, k // 128, lane, byte].to(torch.int32)
    code = torch.where((k % 8 >= 4).expand_as(code), code // 16, code % 16)
    del lane, byte
    scale = s["w4_scale"].double()[n // 16, k // 128, n % 16, (k % 128) // G]
    y = s["x"].double() @ (scale * (code - 8)).T.contiguous()
    return y + s["bias"].double()
