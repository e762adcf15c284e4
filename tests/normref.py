"""The block norms in 64 bits, with bounds on what binary32 arithmetic and the
one rounding to BF16 may cost (first order in the unit roundoff u = 2^-24).

A sum over a row of H values, added in any order with chains of at most
H / 64 + 32 roundings, is off by at most (H / 64 + 32) u times the sum of the
magnitudes.  Bounds of a step's inputs are carried through its derivative."""
from __future__ import annotations

import torch

U = 2.0 ** -24
BF16 = 2.0 ** -8          # half a BF16 step, relative
TINY = 2.0 ** -133        # a BF16 subnormal step


def rounds(H):
    return (H / 64 + 32) * U


def norm(v, e, kind, weight, bias, eps):
    """(values, bound) of a norm of v, itself known up to e."""
    H = v.shape[1]
    n, mean = v, None
    if kind == "none":
        return v, e
    c = rounds(H)
    if kind == "layer":
        mean = v.mean(1, keepdim=True)
        n = v - mean
        e = (e + e.mean(1, keepdim=True) + c * v.abs().mean(1, keepdim=True)
             + U * n.abs())
    rs = 1 / torch.sqrt((n * n).mean(1, keepdim=True) + eps)
    n = n * rs
    # the mean square is off by its own sum (c, and 2 for the division and the
    # eps) and by e; its root halves both; rsqrt and the product round, by up
    # to 2 u and u
    rel = c / 2 + 4 * U + rs * (e * e).mean(1, keepdim=True).sqrt()
    e = rs * e + n.abs() * rel
    if weight is not None:
        n, e = n * weight, e * weight.abs()
    if bias is not None:
        n = n + bias
    return n, e + U * n.abs() + 2.0 ** -149


def block(x, branch=None, *, gate=None, residual_scale=1.0, post_norm="none",
          post_weight=None, post_bias=None, post_eps=1e-6, norm_kind=None,
          weight=None, bias=None, eps=1e-6, scale=None, shift=None,
          mod_row=None):
    """((r, bound), (y, bound)) of a call, each in 64 bits and unrounded; the
    bounds hold before the rounding to BF16.  Tensors are on one device."""
    M, H = x.shape
    d = lambda t: None if t is None else t.double()
    rows = next((1 if t.dim() == 1 else t.shape[0]
                 for t in (gate, scale, shift) if t is not None), None)
    if mod_row is not None:
        at = mod_row.long()
        limit = rows if rows is not None else 2**31 - 1
        dead = (at < 0) | (at >= limit)
        at = torch.where(dead, torch.zeros_like(at), at)
    else:
        at = torch.arange(M, device=x.device) * (rows == M and M > 1)
        dead = torch.zeros(M, dtype=torch.bool, device=x.device)

    def take(t):
        if t is None:
            return None
        return t.double().view(1, H) if t.dim() == 1 else t.double()[at]

    v = d(x)
    e = torch.zeros_like(v)
    r = None
    if branch is not None:
        p, e = norm(d(branch), e, post_norm, d(post_weight), d(post_bias),
                    post_eps)
        g = take(gate)
        if g is not None:
            p, e = p * g, e * g.abs()
        rs = torch.tensor(residual_scale, dtype=torch.float32).double().item()
        a = rs * v
        v = a + p
        e = e + U * (a.abs() + p.abs() + v.abs())
        v = torch.where(dead[:, None], d(x), v)
        e = torch.where(dead[:, None], torch.zeros_like(e), e)
        r = (v, e)
    y = None
    if norm_kind is not None:
        n, e = norm(v, e, norm_kind, d(weight), d(bias), eps)
        sc, sh = take(scale), take(shift)
        if sc is not None:
            n, e = n * (1 + sc), e * (1 + sc).abs() + 2 * U * (n * (1 + sc)).abs()
        if sh is not None:
            n = n + sh
        e = e + U * n.abs() + 2.0 ** -149
        n = torch.where(dead[:, None], torch.zeros_like(n), n)
        e = torch.where(dead[:, None], torch.zeros_like(e), e)
        y = (n, e)
    return r, y


def check_bf16(got, want, bound):
    """got (BF16) is want rounded once, want known up to bound."""
    off = (got.double() - want).abs()
    most = bound + BF16 * (want.abs() + bound) + TINY
    bad = ~(off <= most)
    assert not bad.any(), (
        f"{int(bad.sum())} of {bad.numel()} off, worst at "
        f"{(off / most).argmax().item()}: {(off / most).max().item():.3g} of "
        "the bound")


def check_codes(q, s, want, bound):
    """q, s are the per-token quantization of want, known up to bound."""
    s, q = s.double(), q.double()
    amax = want.abs().amax(1)
    eb = bound.amax(1)
    assert ((s - amax / 127).abs() <= eb / 127 + 2 * U * s + 2.0 ** -149).all()
    zero = s == 0
    assert (q[zero] == 0).all()
    assert (amax[zero] <= eb[zero] + 127 * 2.0 ** -149).all()
    live = ~zero
    q, s, want, bound = q[live], s[live, None], want[live], bound[live]
    # the code is the value over the scale that was written, to the nearest
    off = (q - (want / s).clamp(-127, 127)).abs()
    assert (off <= 0.5 + bound / s + 4 * 127 * U).all(), off.max()
    assert (q.abs().amax(1) == 127).all()
