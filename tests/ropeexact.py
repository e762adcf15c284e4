"""The rotary table's frequencies and angles to 60 digits."""
from __future__ import annotations

import math
from decimal import ROUND_CEILING, ROUND_FLOOR, Context, Decimal, localcontext

DIGITS = Context(prec=60)
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


def frequencies(p, theta=10000.0, scaling="none", factor=1.0, original=0.0,
                beta_fast=32.0, beta_slow=1.0):
    """Radians a position of each of an axis's p pairs."""
    with localcontext(DIGITS):
        theta, factor, original = (Decimal(v) for v in (theta, factor, original))
        if scaling == "ntk" and p > 1:
            theta *= (factor.ln() * p / (p - 1)).exp()
        f = [(-theta.ln() * i / p).exp() for i in range(p)]
        if scaling == "linear":
            f = [v / factor for v in f]
        if scaling == "yarn":
            at = lambda b: p * (original / (2 * PI * Decimal(b))).ln() / theta.ln()
            whole = lambda v, how: v.to_integral_value(rounding=how)
            low = max(whole(at(beta_fast), ROUND_FLOOR), Decimal(0))
            high = min(whole(at(beta_slow), ROUND_CEILING), Decimal(2 * p - 1))
            span = max(high - low, Decimal("0.001"))
            ramp = [min(max((i - low) / span, Decimal(0)), Decimal(1))
                    for i in range(p)]
            f = [v * r / factor + v * (1 - r) for v, r in zip(f, ramp)]
        return f


def turned(position, frequency):
    """(cosine, sine, size of the angle) of a position, the angle's whole turns
    taken off before it is rounded to binary64 (an error below 2^-51)."""
    with localcontext(DIGITS):
        angle = Decimal(position) * frequency
        left = float(angle.remainder_near(2 * PI))
        return math.cos(left), math.sin(left), abs(float(angle))
