"""The steps of gdn_rope_frequencies against the frequencies in 60 digits."""

from decimal import Decimal, localcontext

import pytest

import gated_delta_net_causal_gb300 as gdn
from gated_delta_net_causal_gb300 import _build
from tests import rope_exact

KIND = {"plain": gdn.GDN_ROPE_PLAIN, "linear": gdn.GDN_ROPE_LINEAR, "bands": gdn.GDN_ROPE_BANDS,
        "ramp": gdn.GDN_ROPE_RAMP}
SCALING = [dict(scaling="plain"), dict(scaling="linear", factor=4.0), dict(scaling="linear", factor=0.3),
           dict(scaling="bands", factor=8.0, length=8192.0, low=1.0, high=4.0),
           dict(scaling="bands", factor=3.7, length=5000.5, low=0.31, high=900.0),
           dict(scaling="ramp", factor=16.0, length=4096.0, low=1.0, high=32.0),
           dict(scaling="ramp", factor=1.1, length=77777.0, low=0.5, high=3.0)]


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


@pytest.mark.parametrize("rotary", [2, 4, 32, 42, 64, 96, 126, 128])
@pytest.mark.parametrize("base", [10000.0, 500000.0, 1e6, 1.5, 1.0 + 2.0 ** -40, 1e8 / 3, 1e300])
@pytest.mark.parametrize("i", range(len(SCALING)))
def test_steps_are_the_nearest(rotary, base, i):
    """A step is the frequency in units of 2^-64 of a turn, rounded to the nearest: half a unit, and what its own
    arithmetic (two doubles a number, about 2^-95 of a frequency of up to 2^62 units) adds, far below 2^-20."""
    a = SCALING[i]
    t = gdn.rope_spec(rotary, base=base, scaling=KIND[a["scaling"]], factor=a.get("factor", 1.0),
                      original_length=a.get("length", 0.0), low=a.get("low", 0.0), high=a.get("high", 0.0))
    with localcontext() as c:
        c.prec = rope_exact.DIGITS
        for j, f in enumerate(rope_exact.turns(rotary, base, **a)):
            off = abs(Decimal(t.step[j]) - f * 2 ** 64)
            assert off <= Decimal("0.5") + Decimal(2) ** -20, (j, float(off))
