"""The frequencies' distance from the formula, in 60-digit arithmetic, within the bound that the header
states: (5 + ln base) * 2^-53 relative, (9 + ln base + min(factor, 256)) * 2^-53 with YaRN, and 2^-65
turn. The exponent -2 i / rot_dim is rounded once (ln base times 2^-53 in the power), pow is good to two
roundings, division by 2 pi and by a factor are one each, 2 pi itself is off by less than one. YaRN's
ramp r is off by 2^-53; against f (1 - r) + f r / factor, with 1 - r >= 1/254, that weighs at most
min(factor, 254), and its products and sums add four roundings."""
import math
from decimal import Decimal, getcontext

import pytest

from sparse_attention_lightning_indexer_gb300 import build, ds4idx

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


def _turns(rot, base, scaling, factor, original, fast, slow):
    """Turns a position of each pair, as Decimals."""
    base, factor = Decimal(base), Decimal(factor)
    f = [(-Decimal(2 * i) / rot * base.ln()).exp() for i in range(rot // 2)]
    if scaling == "linear":
        f = [x / factor for x in f]
    if scaling == "yarn":
        def pair(turns):
            p = rot * (Decimal(original) / (2 * PI * Decimal(turns))).ln() / (2 * base.ln())
            assert abs(p - p.to_integral_value()) > Decimal("1e-9")    # no border of the floor or ceil
            return p
        low, high = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), rot - 1)
        ramp = [min(Decimal(1), max(Decimal(0), Decimal(i - low) / max(Decimal(high - low), Decimal("0.001"))))
                for i in range(rot // 2)]
        f = [x * (1 - r) + x / factor * r for x, r in zip(f, ramp)]
    return [x / (2 * PI) for x in f]


@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 3.0), ("linear", 40.0),
                                            ("yarn", 1.0), ("yarn", 4.0), ("yarn", 40.0), ("yarn", 1000.0)])
@pytest.mark.parametrize("rot", [2, 30, 48, 64, 96, 192, 256])
@pytest.mark.parametrize("base", [1.5, 1e4, 5e5, 1e6, 1.5e8])
def test_frequencies_within_the_stated_bound(rot, base, scaling, factor):
    build.build()
    getcontext().prec = 60
    fr = ds4idx.rotary_freqs(rot, base, scaling=scaling, factor=factor, original_max_position=4096)
    if scaling == "yarn":
        rel = 9 + math.log(base) + min(factor, 256)
    else:
        rel = 5 + math.log(base)
    step = Decimal(2) ** -65
    for i, want in enumerate(_turns(rot, base, scaling, factor, 4096, 32.0, 1.0)):
        got = Decimal(int(fr.freqs[i])) / Decimal(2) ** 64
        assert abs(got - want) <= Decimal(rel) * Decimal(2) ** -53 * want + step, i
