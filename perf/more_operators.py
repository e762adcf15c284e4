"""Cases of the operators between a block's Q, K, V and its output projection.

Three kinds of case:

* ``table``: cosines and sines of the rotary positions of a token's axes
  (latent frame, row, column; or one axis), plain or scaled for long contexts;
* ``heads``: the norms of queries and keys for each head with the rotation in
  the same pass, read from the fused Q, K, V output, or the rotation alone;
* ``attend``: attention of queries to keys and values of another length (an
  encoder's states, padded or packed, or the block's own), heads sharing keys.

``own`` selects the library's calls; otherwise the same outputs come from
elementary torch operations in 32 bits (angles in 64).
"""
import math
import random

import torch

own = False

MAX_HEAD_VALUES = 37503 * 2 * 5376    # q and k values of a heads case
MAX_SCORES = 19077 * 19077 * 56 * 128  # query-key pairs times head widths
MAX_ATTEND_VALUES = 19077 * 56 * 128   # values of q, and of k, of an attend case
EPS = 1e-6


def listed():
    return [
        # One new token of a long context, scaled eight times: the latency.
        _table("table_one_token", 1, (64,), "yarn", 8.0, 100000),
        # 768x1344, 124 frames: frame, row and column of every token.
        _table("table_three_axes", 37503, (22, 21, 21), "none", 1.0, 64),
        # One token's queries and keys in front of its attention.
        _heads("heads_one_token", 1, 56, 56, 128, "rms", 64, False),
        # A ragged batch of a narrow model: shared keys, part of the head
        # rotated, interleaved pairs, padding rows.
        _heads("heads_shared_part", 301, 20, 4, 80, "layer", 20, True,
               per_head=True, padded=True),
        # 544x960, 124 frames, heads of the wide block, out of the fused
        # Q, K, V output.
        _heads("heads_19077", 19077, 56, 56, 128, "rms", 64, False),
        # 768x1344, 124 frames: the rotation alone, interleaved.
        _heads("rotate_37503", 37503, 42, 42, 128, "none", 64, True),
        # One query to a short prompt's states.
        _attend("attend_one_query", 1, 1, 512, 56, 56, 128, "dense"),
        # A video's tokens to a padded prompt's states.
        _attend("attend_prompt", 1, 19077, 512, 56, 56, 128, "padded"),
        # A packed batch of odd lengths, four heads sharing keys, one
        # sequence without any key.
        _attend("attend_packed", 6, 700, 333, 16, 4, 64, "packed"),
        # A few queries (the audio's of one frame) to a whole video.
        _attend("attend_few_to_many", 1, 64, 37503, 56, 56, 128, "dense"),
        # 4096 tokens to themselves.
        _attend("attend_self_4096", 1, 4096, 4096, 42, 42, 128, "dense"),
        # 544x960, 124 frames: a video to itself, all heads.
        _attend("attend_self_19077", 1, 19077, 19077, 56, 56, 128, "dense"),
    ]


def _table(name, T, pairs, scaling, factor, reach):
    return {"name": name, "kind": "table", "T": T,
            "pairs": ",".join(map(str, pairs)), "scaling": scaling,
            "factor": factor, "reach": reach}


def _heads(name, M, Hq, Hk, D, norm, pairs, interleaved, per_head=False,
           padded=False):
    return {"name": name, "kind": "heads", "M": M, "Hq": Hq, "Hk": Hk, "D": D,
            "norm": norm, "pairs": pairs, "interleaved": interleaved,
            "per_head": per_head, "padded": padded}


def _attend(name, B, Lq, Lk, Hq, Hk, D, layout):
    """layout: "dense" [B, L]; "padded": dense, but each sequence has a number
    of keys that count; "packed": sequences of odd lengths up to Lq and Lk
    behind each other."""
    return {"name": name, "kind": "attend", "B": B, "Lq": Lq, "Lk": Lk,
            "Hq": Hq, "Hk": Hk, "D": D, "layout": layout}


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(["table", "heads", "heads", "attend", "attend"])
    if kind == "table":
        pairs = [_spread(rng, 1, 64) for _ in range(rng.randint(1, 3))]
        pairs[0] += -sum(pairs) % 4
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        c = _table("", _spread(rng, 1, min(65536, 37503 * 64 // sum(pairs))),
                   pairs, scaling,
                   1.0 if scaling == "none" else rng.choice([2.0, 8.0, 40.0]),
                   _spread(rng, 16, 1000000))
    elif kind == "heads":
        D = 8 * rng.choice([4, 8, 8, 10, 12, 16, 16, 16, 24, 32])
        Hk = _spread(rng, 1, 56)
        Hq = Hk * rng.choice([1, 1, 2, 4])
        pairs = D // 2 if rng.random() < 0.6 else 4 * rng.randint(1, D // 8)
        M = _spread(rng, 1, min(37503, MAX_HEAD_VALUES // (Hq + Hk) // D // 2))
        c = _heads("", M, Hq, Hk, D, rng.choice(["rms", "rms", "layer",
                                                 "none"]), pairs,
                   rng.random() < 0.5, rng.random() < 0.3, rng.random() < 0.3)
    else:
        D = rng.choice([32, 64, 64, 80, 96, 128, 128, 128])
        Hk = _spread(rng, 1, 56)
        Hq = Hk * rng.choice([1, 1, 2, 4, 8])
        B = _spread(rng, 1, 16)
        size = MAX_ATTEND_VALUES // (B * Hq * D) // 2
        Lq = _spread(rng, 1, min(size, 32768))
        Lk = _spread(rng, 1, max(1, min(size, 65536, MAX_SCORES // 8 // (
            B * Hq * D * Lq))))
        c = _attend("", B, Lq, Lk, Hq, Hk, D,
                    rng.choice(["dense", "padded", "packed"]))
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _lengths(case):
    """Queries and keys of each sequence (by the case's sizes alone)."""
    B, Lq, Lk = case["B"], case["Lq"], case["Lk"]
    r = random.Random(B * 1000003 + Lq * 1009 + Lk)
    q, k = [Lq] * B, [Lk] * B
    if case["layout"] == "padded":
        k = [r.randint((Lk + 1) // 2, Lk) for _ in range(B)]
    elif case["layout"] == "packed":
        q = [r.randint(1, Lq) for _ in range(B)]
        k = [r.randint(1, Lk) for _ in range(B)]
        q[0], k[0] = Lq, Lk
        if B > 2:
            k[B // 2] = 0
    return q, k


def _starts(lengths):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return at


def _normal(g, *shape, mean=0.0, std=1.0):
    return (mean + std * torch.randn(*shape, generator=g, device="cuda")).to(
        torch.bfloat16)


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _pairs(case):
    return [int(p) for p in str(case["pairs"]).split(",")]


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    s = dict(case)
    if case["kind"] == "table":
        s["pairs"] = _pairs(case)
        s["positions"] = torch.randint(
            0, case["reach"], (case["T"], len(s["pairs"])), generator=g,
            device="cuda", dtype=torch.int32)
        return s
    if case["kind"] == "heads":
        M, Hq, Hk, D = case["M"], case["Hq"], case["Hk"], case["D"]
        P = case["pairs"]
        # The fused projection's output: q | k | v of a token side by side.
        s["qkv"] = _normal(g, M, (Hq + 2 * Hk) * D, std=1.5)
        for n, H in (("q", Hq), ("k", Hk)):
            w = (H, D) if case["per_head"] else (D,)
            s[n + "_weight"] = s[n + "_bias"] = None
            if case["norm"] != "none":
                s[n + "_weight"] = _normal(g, *w, mean=1.0, std=0.1)
            if case["norm"] == "layer":
                s[n + "_bias"] = _normal(g, *w, std=0.1)
        angle = 2 * math.pi * torch.rand(M, P, generator=g, device="cuda",
                                         dtype=torch.float64)
        s["table"] = torch.stack([angle.cos(), angle.sin()], 1).float()
        s["row"] = None
        if case["padded"]:
            # The batch's tokens point at their positions; the last ones at
            # none (padding).
            row = torch.randperm(M, generator=g, device="cuda")
            row[M - M // 16:] = -1
            s["row"] = row.to(torch.int32)
        return s
    B, Lq, Lk = case["B"], case["Lq"], case["Lk"]
    Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
    q, k = _lengths(case)
    s["lengths"] = (q, k)
    # Normed queries and keys: scores of a few units, some keys favoured.
    if case["layout"] == "packed":
        tq, tk = (sum(q),), (sum(k),)
        s["q_offsets"], s["k_offsets"] = _int32(_starts(q)), _int32(_starts(k))
    else:
        tq, tk = (B, Lq), (B, Lk)
        s["q_offsets"] = s["k_offsets"] = None
    s["k_lens"] = _int32(k) if case["layout"] == "padded" else None
    s["q"] = _normal(g, *tq, Hq, D, std=1.5)
    s["k"] = _normal(g, *tk, Hk, D, std=1.5)
    s["v"] = _normal(g, *tk, Hk, D)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    return {"table": _plain_table, "heads": _plain_heads,
            "attend": _plain_attend}[s["kind"]](s)


THETA = 10000.0
ORIGINAL = 4096  # positions that the unscaled rotation was made for


def _split(s):
    """q [M, Hq, D] and k [M, Hk, D] within the fused output."""
    Hq, Hk, D = s["Hq"], s["Hk"], s["D"]
    q = s["qkv"][:, :Hq * D].unflatten(1, (Hq, D))
    return q, s["qkv"][:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))


def _run_own(s):
    from w8a8_int8_gemm_amd import binding as B
    if s["kind"] == "table":
        more = {}
        if s["scaling"] == "yarn":
            more["original"] = ORIGINAL
        return B.rope_table(s["positions"], s["pairs"], theta=THETA,
                            scaling=s["scaling"], factor=s["factor"], **more)
    if s["kind"] == "heads":
        q, k = _split(s)
        rot = {"row": s["row"], "interleaved": s["interleaved"]}
        if s["norm"] == "none":
            return B.rope(q, s["table"], **rot), B.rope(k, s["table"], **rot)
        return B.head_norm_rope(
            q, k, norm=s["norm"], eps=EPS, q_weight=s["q_weight"],
            q_bias=s["q_bias"], k_weight=s["k_weight"], k_bias=s["k_bias"],
            table=s["table"], **rot)
    return B.attention(s["q"], s["k"], s["v"], q_offsets=s["q_offsets"],
                       k_offsets=s["k_offsets"], k_lens=s["k_lens"])


def _frequencies(P, scaling, factor):
    """Radians a position of an axis' P pairs, and the table's amplitude."""
    i = torch.arange(P, device="cuda", dtype=torch.float64)
    theta = THETA
    if scaling == "ntk" and P > 1:
        theta = THETA * factor ** (P / (P - 1))
    f = theta ** (-i / P)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling != "yarn":
        return f, 1.0
    # YaRN (Peng et al., 2023): pairs that turn more than 32 times over the
    # original length keep their frequency, those below one are interpolated.
    at = [P * math.log(ORIGINAL / (turns * 2 * math.pi)) / math.log(THETA)
          for turns in (32.0, 1.0)]
    low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), 2 * P - 1)
    ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
    return (f / factor * ramp + f * (1 - ramp),
            0.1 * math.log(factor) + 1 if factor > 1 else 1.0)


def _plain_table(s):
    angle = []
    for a, P in enumerate(s["pairs"]):
        f, amplitude = _frequencies(P, s["scaling"], s["factor"])
        angle.append(s["positions"][:, a, None].double() * f)
    angle = torch.cat(angle, 1)
    return (torch.stack([angle.cos(), angle.sin()], 1) * amplitude).float()


def _plain_heads(s):
    row, P = s["row"], s["pairs"]
    table = s["table"]
    if row is not None:
        table = table[row.long().clamp_min(0)]
    c, d = table[:, None, 0], table[:, None, 1]
    out = []
    for n, x in zip(("q", "k"), _split(s)):
        x = x.float()
        if s["norm"] == "layer":
            x = x - x.mean(-1, keepdim=True)
        if s["norm"] != "none":
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
            x = x * s[n + "_weight"].float()
        if s["norm"] == "layer":
            x = x + s[n + "_bias"].float()
        if s["interleaved"]:
            a, b = x[..., 0:2 * P:2], x[..., 1:2 * P:2]
            r = torch.stack([a * c - b * d, b * c + a * d], -1).flatten(-2)
        else:
            a, b = x[..., :P], x[..., P:2 * P]
            r = torch.cat([a * c - b * d, b * c + a * d], -1)
        x = torch.cat([r, x[..., 2 * P:]], -1)
        if row is not None:
            x = torch.where((row >= 0)[:, None, None], x, torch.zeros_like(x))
        out.append(x.to(torch.bfloat16))
    return tuple(out)


def _sequences(s):
    """(query rows, key rows) of each sequence, as slices of flat tensors."""
    q, k = s["lengths"]
    if s["layout"] == "packed":
        qa, ka = _starts(q), _starts(k)
    else:
        qa = [b * s["Lq"] for b in range(s["B"])]
        ka = [b * s["Lk"] for b in range(s["B"])]
    return [(slice(qa[b], qa[b] + q[b]), slice(ka[b], ka[b] + k[b]))
            for b in range(s["B"])]


def _plain_attend(s):
    Hq, Hk, D = s["Hq"], s["Hk"], s["D"]
    G = Hq // Hk
    q, k, v = (s[n].reshape(-1, *s[n].shape[-2:]) for n in "qkv")
    out = torch.empty_like(q)
    for qs, ks in _sequences(s):
        n, m = qs.stop - qs.start, ks.stop - ks.start
        if m == 0:
            out[qs] = 0
            continue
        step = max(1, (1 << 29) // (G * n * m))
        for h in range(0, Hk, step):
            e = min(Hk, h + step)
            # [heads, G n, D] x [heads, D, m]
            a = q[qs, h * G:e * G].float().view(n, e - h, G * D).transpose(
                0, 1).reshape(e - h, n * G, D) * (1 / math.sqrt(D))
            p = a @ k[ks, h:e].float().permute(1, 2, 0).contiguous()
            p = torch.exp(p - p.amax(-1, keepdim=True))
            o = p @ v[ks, h:e].float().transpose(0, 1).contiguous()
            o = o / p.sum(-1, keepdim=True)
            out[qs, h * G:e * G] = o.view(e - h, n, G * D).transpose(
                0, 1).reshape(n, (e - h) * G, D).to(torch.bfloat16)
    return out.view(s["q"].shape)


# ---------------------------------------------------------------------------
# the work of a pass, and its result in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    if case["kind"] == "table":
        P, T = sum(_pairs(case)), case["T"]
        return {"bytes": 4 * T * len(_pairs(case)) + 8 * T * P,
                "flops": 20 * T * P}
    if case["kind"] == "heads":
        M, D, P = case["M"], case["D"], case["pairs"]
        values = M * (case["Hq"] + case["Hk"]) * D
        return {"bytes": 4 * values + 8 * M * P, "flops": 8 * values}
    q, k = _lengths(case)
    D, Hq, Hk = case["D"], case["Hq"], case["Hk"]
    return {"bytes": 4 * sum(q) * Hq * D + 4 * sum(k) * Hk * D,
            "flops": 4 * sum(a * b for a, b in zip(q, k)) * Hq * D}


def exact(case, seed):
    s = prepare(case, seed)
    return {"table": _exact_table, "heads": _exact_heads,
            "attend": _exact_attend}[case["kind"]](s)


def _exact_table(s):
    out = []
    s_ = s["factor"]
    for a, P in enumerate(s["pairs"]):
        f = []
        for i in range(P):
            base = 10000.0
            if s["scaling"] == "ntk" and P > 1:
                base *= math.exp(math.log(s_) * 2 * P / (2 * P - 2))
            w = math.exp(-2 * i / (2 * P) * math.log(base))
            if s["scaling"] == "linear":
                w /= s_
            if s["scaling"] == "yarn":
                def dim(turns):
                    return 2 * P * math.log(4096 / (turns * 2 * math.pi)) / (
                        2 * math.log(base))
                low = max(math.floor(dim(32)), 0)
                high = min(math.ceil(dim(1)), 2 * P - 1)
                if high <= low:
                    high = low + 0.001
                t = min(max((i - low) / (high - low), 0.0), 1.0)
                w = w * (1 - t) + w / s_ * t
            f.append(w)
        f = torch.tensor(f, dtype=torch.float64, device="cuda")
        out.append(torch.outer(s["positions"][:, a].double(), f))
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       torch.cat(out, 1))
    if s["scaling"] == "yarn":
        turn = turn * (1 + 0.1 * math.log(s_))
    return torch.view_as_real(turn).permute(0, 2, 1).contiguous()


def _exact_heads(s):
    P, D, M = s["pairs"], s["D"], s["M"]
    at = torch.arange(M, device="cuda") if s["row"] is None else s["row"].long()
    dead = at < 0
    t = s["table"].double()[at.clamp_min(0)]
    turn = torch.complex(t[:, 0].contiguous(), t[:, 1].contiguous())
    # where a pair's two values lie in the head
    i = torch.arange(P, device="cuda")
    first, second = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + P)
    got, begin = [], 0
    for n in ("q", "k"):
        H = s["H" + n]
        x = s["qkv"][:, begin:begin + H * D].double().reshape(M, H, D)
        begin += H * D
        if s["norm"] == "layer":
            x = x - (x.sum(2) / D).unsqueeze(2)
        if s["norm"] != "none":
            x = x * (math.sqrt(D) / (torch.linalg.vecdot(x, x) +
                                     D * 1e-6).sqrt()).unsqueeze(2)
            x = x * s[n + "_weight"].double()
        if s["norm"] == "layer":
            x = x + s[n + "_bias"].double()
        z = torch.complex(x[..., first], x[..., second]) * turn.unsqueeze(1)
        x[..., first], x[..., second] = z.real, z.imag
        x[dead] = 0
        got.append(x)
    return tuple(got)


def _exact_attend(s):
    G, D = s["Hq"] // s["Hk"], s["D"]
    q, k, v = (s[n].flatten(0, -3) for n in "qkv")
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    for qs, ks in _sequences(s):
        if ks.stop == ks.start:
            continue
        step = max(1, (1 << 28) // (ks.stop - ks.start))
        for h in range(s["Hk"]):
            kt = k[ks, h].double().T.contiguous()
            vh = v[ks, h].double()
            for g in range(h * G, (h + 1) * G):
                for a in range(qs.start, qs.stop, step):
                    b = min(a + step, qs.stop)
                    z = q[a:b, g].double() @ kt / math.sqrt(D)
                    z = (z - torch.logsumexp(z, 1).unsqueeze(1)).exp_()
                    out[a:b, g] = z @ vh
    return out.view(s["q"].shape)
