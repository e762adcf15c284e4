"""The rotary table, the head norms with rotation and the attention in 64 bits,
with bounds on what the 32-bit arithmetic and the roundings to BF16 may cost
(first order in the unit roundoff u = 2^-24)."""
from __future__ import annotations

import math

import torch

from tests import normref as R

U = 2.0 ** -24
BF16 = R.BF16


# ---------------------------------------------------------------------------
# rotary table
# ---------------------------------------------------------------------------

def frequencies(p, theta=10000.0, scaling="none", factor=1.0, original=0.0,
                beta_fast=32.0, beta_slow=1.0):
    if scaling == "ntk" and p > 1:
        theta = theta * factor ** (p / (p - 1))
    f = [theta ** (-i / p) for i in range(p)]
    if scaling == "linear":
        f = [v / factor for v in f]
    if scaling == "yarn":
        at = lambda b: (p * math.log(original / (2 * math.pi * b)) /
                        math.log(theta))
        low = max(math.floor(at(beta_fast)), 0)
        high = min(math.ceil(at(beta_slow)), 2 * p - 1)
        ramp = [min(max((i - low) / max(high - low, 0.001), 0), 1)
                for i in range(p)]
        f = [v * r / factor + v * (1 - r) for v, r in zip(f, ramp)]
    return torch.tensor(f, dtype=torch.float64)


def table(positions, pairs, amplitude=1.0, **kw):
    """(cosines and sines [T, 2, P], bound)."""
    pos = positions.double().cpu().view(positions.shape[0], -1)
    angle = torch.cat([pos[:, a, None] * frequencies(p, **kw)
                       for a, p in enumerate(pairs)], 1)
    want = amplitude * torch.stack([angle.cos(), angle.sin()], 1)
    # Either side's angle is off by a few units of 2^-53 of itself (power,
    # quotients, product).  What is left of it within a quadrant (below pi/4)
    # rounds twice as an argument, as does its constant: 3 u pi/4; the series'
    # last steps 1.5 u, the amplitude and its product 2 u: under 6 u in all.
    bound = abs(amplitude) * (angle.abs()[:, None] * 2.0 ** -50 + 6 * U)
    return want, bound


# ---------------------------------------------------------------------------
# head norms with rotation
# ---------------------------------------------------------------------------

def heads(x, norm="none", weight=None, bias=None, eps=1e-6, table=None,
          row=None, interleaved=False):
    """(values [M, H, D], bound before the rounding to BF16)."""
    M, H, D = x.shape
    v = x.double()
    flat = lambda t: None if t is None else t.double().expand(M, H, D).reshape(
        M * H, D)
    v, e = R.norm(v.reshape(M * H, D), torch.zeros(
        M * H, D, dtype=torch.float64, device=x.device), norm, flat(weight),
        flat(bias), eps)
    v, e = v.view(M, H, D), e.view(M, H, D)
    if table is None:
        return v, e
    rows, _, P = table.shape
    at = torch.arange(M, device=x.device) * (rows > 1)
    if row is not None:
        at = row.long()
    dead = (at < 0) | (at >= rows)
    t = table.double()[at.clamp(0, rows - 1)][:, None]
    c, s = t[:, :, 0], t[:, :, 1]
    a = slice(0, 2 * P, 2) if interleaved else slice(0, P)
    b = slice(1, 2 * P, 2) if interleaved else slice(P, 2 * P)
    out, be = v.clone(), e.clone()

    def turned(x, y, ex, ey, s):
        # a product and a fused multiply-add round
        return (x * c + y * s, ex * c.abs() + ey * s.abs() +
                2 * U * ((x * c).abs() + (y * s).abs()))
    out[..., a], be[..., a] = turned(v[..., a], v[..., b], e[..., a],
                                     e[..., b], -s)
    out[..., b], be[..., b] = turned(v[..., b], v[..., a], e[..., b],
                                     e[..., a], s)
    out[dead], be[dead] = 0, 0
    return out, be


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def sequences(Tq, Tk, B, q_offsets=None, k_offsets=None, k_lens=None):
    """(first query, queries, first key, keys) of each sequence."""
    def spans(T, offsets):
        if offsets is None:
            return [(b * (T // B), T // B) for b in range(B)]
        o = offsets.tolist()
        return [(o[b], o[b + 1] - o[b]) for b in range(B)]
    out = []
    for b, (q, k) in enumerate(zip(spans(Tq, q_offsets),
                                   spans(Tk, k_offsets))):
        keys = k[1]
        if k_lens is not None:
            keys = min(max(int(k_lens[b]), 0), keys)
        out.append((*q, k[0], keys))
    return out


def attention(q, k, v, spans, scale=None):
    """(values [Tq, Hq, D], bound before the rounding to BF16, rows covered).

    With w_j the weights of a row and o its result, a relative error d_j of
    weight j moves the result by sum_j w_j d_j (v_j - o) (the weights are
    divided by the sum of the very weights that are used), at most max|d| times
    the weighted deviation of v, itself at most its root mean square sigma.
      d: rounding a weight to BF16, 2^-8 (to second order 2^-8 (1 + 2^-7));
         the score, at most D roundings of its partial sums, times the scale;
         the exponent, two roundings of its size, and 2^(..), 2^-22.
    Sums over n keys: n roundings of the magnitudes w_j |v_j|, and as many in
    the weights' own sum (times |o|); joins and the division a few more."""
    D, G = q.shape[2], q.shape[1] // k.shape[1]
    scale = 1 / math.sqrt(D) if scale is None else scale
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    covered = torch.zeros(q.shape[0], dtype=torch.bool, device=q.device)
    for q0, nq, k0, nk in spans:
        covered[q0:q0 + nq] = True
        if not nq or not nk:
            continue
        for h in range(q.shape[1]):
            a = q[q0:q0 + nq, h].double()
            b = k[k0:k0 + nk, h // G].double()
            x = v[k0:k0 + nk, h // G].double()
            s = a @ b.t().contiguous() * scale
            w = torch.softmax(s, 1)
            o = w @ x
            sigma = ((w @ (x * x)) - o * o).clamp_min(0).sqrt()
            size = (a.abs() @ b.abs().t().contiguous() * scale).amax(
                1, keepdim=True)
            d = (BF16 * (1 + 2.0 ** -7) + D * U * size +
                 2 * U * s.abs().amax(1, keepdim=True) + 2.0 ** -22)
            n = nk + 80
            out[q0:q0 + nq, h] = o
            # sigma from its difference is itself uncertain in 64 bits
            bound[q0:q0 + nq, h] = (
                d * (sigma + 1e-7 * o.abs()) + n * U * (w @ x.abs() + o.abs()))
    return out, bound, covered


check_bf16 = R.check_bf16
