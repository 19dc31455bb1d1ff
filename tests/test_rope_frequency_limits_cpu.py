"""gdn_rope_frequencies where a frequency is out of the doubles' range, or nearly."""

import ctypes

import pytest

import gated_delta_net_causal_gb300 as gdn
from gated_delta_net_causal_gb300 import _build

INVALID, OK = 1, 0


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return gdn.library()


def call(lib, scaling, factor, length=4096.0, low=1.0, high=4.0, base=1e4, rotary=64):
    t = gdn.GdnRopeTable()
    t.rotary_dim = 77
    st = lib.gdn_rope_frequencies(rotary, 0, base, scaling, factor, length, low, high, 1.0, ctypes.byref(t))
    return st, t


@pytest.mark.parametrize("scaling", [gdn.GDN_ROPE_LINEAR, gdn.GDN_ROPE_BANDS, gdn.GDN_ROPE_RAMP])
@pytest.mark.parametrize("factor", [1e-310, 5e-324])
def test_a_frequency_that_is_not_finite_is_refused(lib, scaling, factor):
    st, t = call(lib, scaling, factor)
    assert st == INVALID and t.rotary_dim == 77  # nothing is written


def test_factors_that_nothing_is_stretched_by(lib):
    """Every pair turns more often than high: none is divided by the factor."""
    st, t = call(lib, gdn.GDN_ROPE_BANDS, 1e-310, length=1e300, low=1.0, high=2.0, base=1.5)
    plain = call(lib, gdn.GDN_ROPE_PLAIN, 1.0, base=1.5)[1]
    assert st == OK and list(t.step) == list(plain.step)


@pytest.mark.parametrize("scaling", [gdn.GDN_ROPE_BANDS, gdn.GDN_ROPE_RAMP])
@pytest.mark.parametrize("length,low,high", [(1e308, 1e-300, 1e308), (5e-324, 1.0, 2.0), (1e308, 5e-324, 1e-323),
                                             (4096.0, 1.0, 1.0 + 2.0 ** -52), (1e-300, 1e307, 1e308)])
@pytest.mark.parametrize("base", [1.0 + 2.0 ** -52, 1e4, 1.7e308])
@pytest.mark.parametrize("factor", [1.0, 1e308])
def test_the_ends_of_the_doubles_range(lib, scaling, length, low, high, base, factor):
    """Accepted, with steps between those of the stretched and of the plain frequencies (half a unit each, and one for a
    quotient next to a border)."""
    for rotary in (2, 64, 128):
        st, t = call(lib, scaling, factor, length, low, high, base, rotary)
        plain = call(lib, gdn.GDN_ROPE_PLAIN, 1.0, base=base, rotary=rotary)[1]
        least = call(lib, gdn.GDN_ROPE_LINEAR, factor, base=base, rotary=rotary)[1]
        assert st == OK
        for i in range(rotary // 2):
            assert least.step[i] - 2 <= t.step[i] <= plain.step[i] + 2, (rotary, i)
