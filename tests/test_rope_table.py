"""CPU tests of the rotary table's fractions against values of 100 digits."""
import decimal
import math
from decimal import Decimal

import pytest

PI = Decimal("3.141592653589793238462643383279502884197169399375105820974944592307816406286208998628034825342117067982")


@pytest.fixture(scope="module")
def rn():
    from residual_add_rmsnorm_vec_gb300 import build

    build.build()
    import residual_add_rmsnorm_vec_gb300 as p

    return p


def off(bits, radians):
    """Distance of a table's entry from the fraction of a turn, in 2^-64 turns."""
    d = (Decimal(bits % 2**64) - radians / (2 * PI) * 2**64) % 2**64
    return float(min(abs(d), abs(2**64 - abs(d))))


@pytest.mark.parametrize("base", [10000.0, 500000.0, 1e6, 7.5, 1.0, 0.25, 1e-12, 1e300])
@pytest.mark.parametrize("rot_dim", [2, 64, 128, 96])
def test_default_frequencies_to_the_nearest_fraction(rn, base, rot_dim):
    table = rn.rope_table(rot_dim, base=base, device="cpu")
    with decimal.localcontext(decimal.Context(prec=100)):
        for p, bits in enumerate(table.turns.tolist()):
            radians = (-(Decimal(base).ln()) * 2 * p / rot_dim).exp()
            assert off(bits, radians) <= 0.5 + 1e-6, p


def test_given_frequencies_to_the_nearest_fraction(rn):
    given = [1.0, -0.5, 1e-5, 3e-20, 5e-324, -0.0, math.pi, 2 * math.pi, 6.25, -123456.789, 1e15, 4.2e25, -7.7e29]
    table = rn.rope_table(2 * len(given), inv_freq=given, device="cpu")
    with decimal.localcontext(decimal.Context(prec=100)):
        for f, bits in zip(given, table.turns.tolist()):
            assert off(bits, Decimal(f)) <= 0.5 + 1e-6, f


@pytest.mark.parametrize("position", [1, 12345, 2**31 - 1, -(2**31), 2**40 + 7, 2**53 + 1])
def test_far_phases(rn, position):
    # the phase that the kernel takes (the product modulo 2^64) against the angle itself
    table = rn.rope_table(128, device="cpu")
    with decimal.localcontext(decimal.Context(prec=100)):
        for p, bits in enumerate(table.turns.tolist()):
            radians = Decimal(position) * (-(Decimal(10000).ln()) * 2 * p / 128).exp()
            assert off(bits % 2**64 * position, radians) <= abs(position) * (0.5 + 1e-6), p


def test_frequencies_of_any_size(rn):
    # beyond the digits above: whole turns leave nothing (a multiple of pi is no double)
    table = rn.rope_table(4, inv_freq=[1e308, -1e308], device="cpu")
    a, b = table.turns.tolist()
    assert (a + b) % 2**64 == 0 and a != 0
    assert rn.rope_table(4, base=math.inf, device="cpu").turns.tolist()[1] == 0
    with pytest.raises(ValueError):
        rn.rope_table(4, base=math.nan, device="cpu")
