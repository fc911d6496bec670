"""The fractions of a turn that rotary positions are made of, against whole-number
arithmetic: 64 bits of each are right, which a double cannot hold."""
from fractions import Fraction

import pytest

pytest.importorskip("torch")


def pi():
    """pi to 2^-190: 16 atan(1/5) - 4 atan(1/239)."""
    one = 1 << 200

    def atan_inverse(x):
        total, term, n = 0, one // x, 1
        while term:
            total += (term // n) * (1 if n % 4 == 1 else -1)
            term, n = term // (x * x), n + 2
        return total

    return Fraction(16 * atan_inverse(5) - 4 * atan_inverse(239), one)


def root(x, n):
    """The largest whole number whose n-th power is at most x."""
    lo, hi = 0, 1 << (x.bit_length() // n + 1)
    while hi - lo > 1:
        mid = (lo + hi) // 2
        lo, hi = (mid, hi) if mid ** n <= x else (lo, mid)
    return lo


def power(base, num, den):
    """base^(num / den), to 2^-150 of itself, of a base of at least 1 and num <= 0."""
    base = Fraction(base) ** -num
    bits = 170 + base.numerator.bit_length() // den
    return Fraction(root((base.denominator << (bits * den)) // base.numerator, den), 1 << bits)


def expected(rot, base, scaling):
    kind = scaling["type"] if scaling else "none"
    f = [power(base, -2 * i, rot) for i in range(rot // 2)]
    if kind == "linear":
        return [x / Fraction(scaling["factor"]) for x in f]
    if kind == "ntk":
        return [x * power(scaling["factor"], -2 * i, rot - 2) for i, x in enumerate(f)]
    if kind == "wavelength":
        out = []
        for x in f:
            t = x * scaling["original"] / (2 * pi())
            keep = min(Fraction(1), max(Fraction(0), (t - scaling["low"]) / (scaling["high"] - scaling["low"])))
            out.append(x * keep + x / scaling["factor"] * (1 - keep))
        return out
    if kind == "yarn":
        lo, hi = scaling["between"]
        ramp = [min(Fraction(1), max(Fraction(0), Fraction(i - lo, hi - lo))) for i in range(rot // 2)]
        return [x * (1 - r) + x / scaling["factor"] * r for x, r in zip(f, ramp)]
    return f


@pytest.mark.parametrize("rot,base,scaling", [
    (128, 500000.0, None), (64, 10000.0, None), (16, 1000000.0, None), (112, 1234.5, None),
    (128, 500000.0, {"type": "linear", "factor": 4}), (64, 10000.0, {"type": "linear", "factor": 2.5}),
    (64, 10000.0, {"type": "ntk", "factor": 8}),
    (128, 500000.0, {"type": "wavelength", "factor": 8, "low": 1, "high": 4, "original": 8192}),
    # turns over 4096 positions: 32 at pair 10.47, one at 22.51
    (64, 10000.0, {"type": "yarn", "factor": 4, "original": 4096, "between": (10, 23)}),
])
def test_turns_are_right_to_their_last_bit(rot, base, scaling):
    import __graft_entry__
    __graft_entry__.build()
    from head_heterogeneous_block_gb300 import rotary
    given = {k: v for k, v in scaling.items() if k != "between"} if scaling else None
    freq, _ = rotary._frequencies(rot, base, given)
    turns = rotary._turns(freq)
    ref = expected(rot, base, scaling)
    for t, x in zip(turns, ref):
        assert abs(t - x / (2 * pi()) * 2 ** 64) <= Fraction(1, 2) + Fraction(1, 2 ** 60)
    # and the frequencies beside them are the nearest doubles
    assert rotary.rotary_frequencies(rot, base, given)[0] == [float(x) for x in ref]


@pytest.mark.parametrize("factor", [1e-6, 0.5, 1.0])
def test_yarn_leaves_values_alone_where_it_stretches_nothing(factor):
    import __graft_entry__
    __graft_entry__.build()
    from head_heterogeneous_block_gb300.rotary import rotary_frequencies
    scaling = {"type": "yarn", "factor": factor, "original": 4096}
    assert rotary_frequencies(64, 10000.0, scaling)[1] == 1.0
    assert rotary_frequencies(64, 10000.0, {**scaling, "attention_factor": 0.7})[1] == 0.7
