"""The frequencies of rotations against the published formula in decimal arithmetic:
base^(-2 i / dims), and for stretched positions the interpolation by parts."""

from decimal import ROUND_CEILING, ROUND_FLOOR, Decimal, getcontext

import pytest

import strided_gemm_gb300 as sg

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


def by_parts(dims, base, factor, original, fast, slow):
    getcontext().prec = 50
    ln = Decimal(base).ln()

    def index(turns):
        """The pair that turns so often in `original` positions: original base^(-2 i / dims) / (2 pi) = turns."""
        return dims * (Decimal(original) / (Decimal(turns) * 2 * PI)).ln() / (2 * ln)

    low = max(index(fast).to_integral_value(ROUND_FLOOR), Decimal(0))
    high = min(index(slow).to_integral_value(ROUND_CEILING), Decimal(dims - 1))
    out = []
    for i in range(dims // 2):
        f = (-ln * 2 * i / dims).exp()
        slowed = min(max((i - low) / max(high - low, Decimal("0.001")), Decimal(0)), Decimal(1)) if factor != 1 else Decimal(0)
        out.append((f * (1 - slowed) + f / Decimal(factor) * slowed, original * f / (2 * PI)))
    return out


@pytest.mark.parametrize("dims,base,factor,original,fast,slow", [
    (64, 10000.0, 1.0, 4096, 32.0, 1.0), (64, 10000.0, 4.0, 4096, 32.0, 1.0), (128, 10000.0, 32.0, 4096, 32.0, 1.0),
    (128, 500000.0, 8.0, 8192, 32.0, 1.0), (64, 10000.0, 40.0, 4096, 32.0, 1.0), (16, 100.0, 2.0, 64, 8.0, 0.5),
    (2, 10000.0, 4.0, 4096, 32.0, 1.0), (64, 10000.0, 4.0, 16, 32.0, 1.0),
])
def test_frequencies_follow_the_formula(dims, base, factor, original, fast, slow):
    got = sg.rope_frequencies(dims, base=base, factor=factor, original=original, fast=fast, slow=slow)
    want = by_parts(dims, base, factor, original, fast, slow)
    assert len(got) == len(want) == dims // 2
    for g, (w, turns) in zip(got, want):
        # A handful of roundings of 2^-53, the power's exponent among them (up to 13 in size).
        assert abs(Decimal(g) - w) <= w * Decimal(2) ** -47
    if factor != 1.0:
        for g, (w, turns), plain in zip(got, want, sg.rope_frequencies(dims, base=base)):
            if turns >= fast:
                assert g == pytest.approx(plain, rel=1e-12)
            assert plain / factor * (1 - 1e-12) <= g <= plain * (1 + 1e-12)
