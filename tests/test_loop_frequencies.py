"""The frequencies of rotary positions against their formulas in 60 decimal digits: the bound that the header states."""
from decimal import Decimal as D
from decimal import getcontext

import numpy as np
import pytest

getcontext().prec = 60
PI = D("3.14159265358979323846264338327950288419716939937510582097494459")


def power(x, e):
    return (e * x.ln()).exp()


def formulas(dim, theta=10000.0, scaling="none", factor=1.0, original_len=0, beta_fast=32.0, beta_slow=1.0, low_turns=1.0,
             high_turns=4.0):
    """Of every pair: its frequency, the one before scaling, and how much larger than theirs the error of a scaled one may be."""
    theta, factor, rows = D(theta), D(factor), D(original_len)
    if scaling == "base":
        theta *= power(factor, D(dim) / (dim - 2))
    worse = D(1)
    if scaling == "bands":
        worse += D(high_turns) / (D(high_turns) - D(low_turns))
    out = []
    for i in range(dim // 2):
        plain = f = power(theta, D(-2 * i) / dim)
        if scaling == "linear":
            f = f / factor
        elif scaling == "yarn":
            at = lambda turns: dim * (rows / (D(turns) * 2 * PI)).ln() / (2 * theta.ln())  # noqa: E731
            low = max(D(int(at(beta_fast).to_integral_value("ROUND_FLOOR"))), D(0))
            high = min(D(int(at(beta_slow).to_integral_value("ROUND_CEILING"))), D(dim - 1))
            r = min(max((i - low) / max(high - low, D(0.001)), D(0)), D(1))
            f = f * (r / factor + 1 - r)
        elif scaling == "bands":
            m = min(max((rows * f / (2 * PI) - D(low_turns)) / (D(high_turns) - D(low_turns)), D(0)), D(1))
            f = f * ((1 - m) / factor + m)
        out.append((f, plain, (2 * theta.ln() + 8) * worse))
    return out


def off(dim, **kw):
    """The largest error of an angle's step, in radians a position, as a share of what the header allows."""
    import deepseek_v4_hybrid_gb300 as M
    got = M.rope_freqs(dim, device="cpu", **kw).numpy().view(np.uint64)
    worst = D(0)
    for g, (f, plain, k) in zip(got, formulas(dim, **kw)):
        allowed = plain * k * D(2) ** -53 + 2 * PI * D(2) ** -64
        worst = max(worst, abs(D(int(g)) * D(2) ** -64 * 2 * PI - f) / allowed)
    return worst


@pytest.mark.parametrize("dim", [4, 24, 64, 96, 128, 1022, 1024])
@pytest.mark.parametrize("theta", [1.5, 10000.0, 500000.0, 1e6, 1e9])
@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=3.0), dict(scaling="linear", factor=40.0),
                                dict(scaling="base", factor=8.0), dict(scaling="base", factor=1000.7),
                                dict(scaling="yarn", factor=40.0, original_len=4096), dict(scaling="yarn", factor=3.3, original_len=32768),
                                dict(scaling="bands", factor=8.0, original_len=8192),
                                dict(scaling="bands", factor=7.0, original_len=3000, low_turns=3.5, high_turns=4.0)],
                         ids=lambda k: "_".join(f"{v}" for v in k.values()) or "plain")
def test_frequencies_within_the_bound(dim, theta, kw):
    assert off(dim, theta=theta, **kw) <= 1


def test_small_frequencies_are_cut_at_a_step_of_the_fraction():
    """Far down the steps of the 64-bit fraction are what an angle is off by, not the rounding of f: f 2^-51 alone would be
    exceeded thousands of times."""
    import deepseek_v4_hybrid_gb300 as M
    kw = dict(theta=1e6, scaling="linear", factor=40.0)
    got = M.rope_freqs(64, device="cpu", **kw).numpy().view(np.uint64)
    share = [abs(D(int(g)) * D(2) ** -64 * 2 * PI - f) / (f * D(2) ** -51) for g, (f, _, _) in zip(got, formulas(64, **kw))]
    assert max(share) > 1000 and share[0] <= 1
