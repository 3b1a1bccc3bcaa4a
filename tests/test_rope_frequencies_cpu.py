"""Rotary frequencies are the multiples of 2^-64 turns nearest to their definition, which is
evaluated here with 120 decimal digits from the same fp64 numbers (CPU)."""
import decimal
import math
import random
from decimal import Decimal as D

import pytest

from row_wise_rmsnorm_fwd_gb300 import binding, build

PI = D("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899"
       "8628034825342117067982148086513282306647093844609550582231725359408128")
TURN = 2 ** 64


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()


@pytest.fixture(autouse=True)
def digits():
    with decimal.localcontext() as c:
        c.prec = 120
        yield


def power(base, exponent):
    return (exponent * D(base).ln()).exp()


def turns(rot, base=10000.0, scaling="none", factor=1.0, original_len=0, low=None, high=None,
          divisors=None):
    """Turns a position of each pair."""
    low, high = (D(b if a is None else a) for a, b in
                 zip((low, high), {"ramp": (1, 32)}.get(scaling, (1, 4))))
    k, out = D(factor), []
    if scaling == "ramp":
        first, last = (rot * (original_len / (t * 2 * PI)).ln() / (2 * D(base).ln())
                       for t in (high, low))
        first, last = max(math.floor(first), 0), min(math.ceil(last), rot - 1)
    for i in range(rot // 2):
        f = power(base, D(-2 * i) / rot) / (2 * PI)
        kept = D(1)
        if scaling == "linear":
            kept = D(0)
        elif scaling == "base":
            f *= power(factor, D(-2 * i) / (rot - 2))
        elif scaling == "ramp":
            kept = 1 - (i - first) / max(D(last - first), D("0.001"))
        elif scaling == "bands":
            kept = (original_len * f - low) / (high - low)
        kept = min(max(kept, D(0)), D(1))
        f = f / k * (1 - kept) + f * kept
        out.append(f if divisors is None else f / D(divisors[i]))
    return out


def check(rot, **rule):
    freqs, _ = binding.rmsnorm_rope_freqs(rot, device="cpu", **rule)
    for i, (got, want) in enumerate(zip(freqs.tolist(), turns(rot, **rule))):
        off = got - want * TURN
        off = abs(off - TURN * (off / TURN).to_integral_value(decimal.ROUND_HALF_EVEN))
        # half a step; what is formed before the rounding is off by far less than 2^-10 of one
        assert off <= D(1) / 2 + D(2) ** -10, (rot, rule, i, float(off))


@pytest.mark.parametrize("rot", [2, 4, 6, 20, 64, 80, 96, 128, 256, 1024])
@pytest.mark.parametrize("base", [1.0001, 2.0, 10.0, 10000.0, 500000.0, 1e6, 1e300])
def test_plain(rot, base):
    check(rot, base=base)


SCALINGS = [dict(scaling="linear", factor=3.0), dict(scaling="linear", factor=0.1 * 70),
            dict(scaling="base", factor=2.5), dict(scaling="base", factor=1e30),
            dict(scaling="ramp", factor=4.0, original_len=8192),
            dict(scaling="ramp", factor=40.0, original_len=4096, low=1.5, high=24.0),
            dict(scaling="bands", factor=8.0, original_len=8192),
            dict(scaling="bands", factor=7.0, original_len=2 ** 40, low=0.3, high=2.7)]


@pytest.mark.parametrize("rot", [4, 64, 96, 128])
@pytest.mark.parametrize("rule", SCALINGS, ids=lambda r: "-".join(map(str, r.values())))
def test_scaled(rot, rule):
    check(rot, base=10000.0, **rule)
    check(rot, base=500000.0, **rule)


@pytest.mark.parametrize("least", [1.0, 1e-3, 1e-9])
@pytest.mark.parametrize("scaling", ["none", "linear", "bands"])
def test_divisors(least, scaling):
    """Divisors below one: many turns a position, of which the whole ones do not count."""
    rng = random.Random(5)
    rule = {} if scaling == "none" else dict(scaling=scaling, factor=2.0, original_len=8192)
    div = [least * math.exp(rng.uniform(0, 4)) for _ in range(32)]
    check(64, divisors=div, **rule)


def test_any_divisor_is_taken():
    """Frequencies of more turns than there are bits for: some number, and no error."""
    freqs, _ = binding.rmsnorm_rope_freqs(8, device="cpu", divisors=[5e-324, 1e-300, 1e300, 1.7e308])
    assert freqs.tolist()[2:] == [0, 0]
