"""Rotary frequencies from their definition in 60 decimal digits."""

import math
from decimal import Decimal, localcontext

DIGITS = 60
# pi to 63 digits
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


def turns(rotary, base, scaling="plain", factor=1.0, length=0.0, low=0.0, high=0.0):
    """Each pair's frequency as turns a position. The arguments are the doubles that the call is given."""
    with localcontext() as c:
        c.prec = DIGITS
        base, factor, length, low, high = (Decimal(x) for x in (base, factor, length, low, high))
        out = []
        if scaling == "ramp":
            def at(n):
                return rotary * (length / (2 * PI * n)).ln() / (2 * base.ln())

            first, last = max(math.floor(at(high)), 0), min(math.ceil(at(low)), rotary - 1)
        for i in range(rotary // 2):
            b = (-Decimal(2 * i) / rotary * base.ln()).exp()
            keep = Decimal(1)
            if scaling == "linear":
                keep = Decimal(0)
            elif scaling == "bands":
                keep = (length * b / (2 * PI) - low) / (high - low)
            elif scaling == "ramp":
                keep = 1 - Decimal(i - first) / max(Decimal(last - first), Decimal("0.001"))
            keep = min(max(keep, Decimal(0)), Decimal(1))
            out.append(b * (keep + (1 - keep) / factor) / (2 * PI))
        return out


def angle(position, turn):
    """position times a frequency in turns, as radians from -pi to pi."""
    with localcontext() as c:
        c.prec = DIGITS
        x = position * turn
        return float((x - x.to_integral_value()) * 2 * PI)
