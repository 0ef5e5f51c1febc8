"""Rotary plans hold their frequencies to the 2^-53 turns that mk.h states, for
parameters of any value (not only those that fp32 holds exactly): against 50-digit
arithmetic."""
import decimal
from decimal import Decimal as D

import pytest

from decode_megakernel_03_gb300 import build as mkbuild
from decode_megakernel_03_gb300 import mk

PI = D("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.fixture(scope="module", autouse=True)
def L():
    mkbuild.build()
    return mk.lib()


def frequencies(n, theta, scaling="none", factor=1.0, low=1.0, high=4.0, original_length=0):
    theta, factor, low, high, length = map(D, (theta, factor, low, high, original_length))
    f = [(-(2 * D(i) / n) * theta.ln()).exp() for i in range(n // 2)]
    out = []
    for i, x in enumerate(f):
        if scaling == "linear":
            x /= factor
        elif scaling == "bands":
            mix = min(D(1), max(D(0), (length * x / (2 * PI) - low) / (high - low)))
            x = (1 - mix) * x / factor + mix * x
        elif scaling == "yarn":
            def pair(turns):
                return n * (length / (turns * 2 * PI)).ln() / (2 * theta.ln())
            lo = max(D(0), pair(high).to_integral_value(decimal.ROUND_FLOOR))
            hi = min(D(n - 1), pair(low).to_integral_value(decimal.ROUND_CEILING))
            ramp = min(D(1), max(D(0), (i - lo) / (hi - lo))) if hi > lo else D(int(i > lo))
            x = x * (1 - ramp) + x / factor * ramp
        out.append(x)
    return out


@pytest.mark.parametrize("d,part", [(64, 64), (128, 128), (128, 60)])
@pytest.mark.parametrize("kw", [dict(theta=500000.0), dict(theta=84234.3), dict(theta=1234567.89),
                                dict(theta=10000.0, scaling="linear", factor=2.6),
                                dict(theta=84234.3, scaling="bands", factor=8.7, low=1.1, high=4.3,
                                     original_length=8192),
                                dict(theta=84234.3, scaling="yarn", factor=16.1, low=1.1, high=31.7,
                                     original_length=4096)])
def test_frequencies_to_2_to_the_minus_53_turns(kw, d, part):
    with decimal.localcontext() as c:
        c.prec = 50
        turns = mk.Rope(d, rotary_dim=part, **kw).struct.turns
        for i, f in enumerate(frequencies(part, **kw)):
            assert abs(D(turns[i]) / D(2)**64 - f / (2 * PI)) <= D(2)**-53, i
