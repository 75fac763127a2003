"""The 4-bit quantiser in rational arithmetic: every rounding is taken from the
exact value, with no floating-point step in between."""
from __future__ import annotations

from fractions import Fraction

import numpy as np

GROUP = 64


def round_half(x: Fraction) -> float:
    """x rounded once to fp16 (to nearest, ties to even; beyond the range: an infinity)."""
    if x == 0:
        return 0.0
    a = abs(x)
    e = -14                                    # exponent of the step below: 2^(e - 10), at least 2^-24
    while e < 16 and a >= Fraction(2) ** (e + 1):
        e += 1
    ulp = Fraction(2) ** (e - 10)
    y = round(a / ulp) * ulp                   # Fraction rounds ties to even
    y = float("inf") if y >= 65536 else float(y)
    return y if x > 0 else -y


def quantise_group(x):
    """(codes [64], step, low) of 64 finite values; codes 0 and step NaN where low or step is not finite."""
    f = [Fraction(float(v)) for v in x]
    low, step = round_half(min(f)), round_half((max(f) - min(f)) / 15)
    if np.isinf(low) or np.isinf(step):
        return [0] * len(f), float("nan"), low
    if step == 0:
        return [0] * len(f), step, low
    return [min(15, max(0, round((v - Fraction(low)) / Fraction(step)))) for v in f], step, low
