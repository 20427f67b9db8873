"""Entry points for long contexts at the edges of their arguments, without a GPU."""
import ctypes
import math
from decimal import Decimal, getcontext

import pytest

import __graft_entry__

__graft_entry__.build()
import gated_rank_subspace_gb300 as gsi  # noqa: E402

L = gsi.lib()


@pytest.mark.parametrize("rate", [2.0**40, -2.0**40, 2.0**40 - 2.0**-12, 1e12, 2.0**33 + 2.0**-19, 12345.678, 2.0**40 / math.pi, 1e-300])
def test_phases_of_large_and_small_rates(rate):
    getcontext().prec = 120
    turn = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798214808651")
    w, out = (ctypes.c_double * 1)(rate), (ctypes.c_uint64 * 1)()
    assert L.gsi_rotary_phases(w, 1, out) == 0
    off = (int(out[0]) - int((Decimal(rate) / turn % 1 * 2**64).to_integral_value())) % 2**64
    # two roundings to whole units, and 2^-106 of up to 2^38 turns
    assert min(off, 2**64 - off) <= 2


@pytest.mark.parametrize("rate", [2.0**40 * (1 + 2**-52), -3e17, 3e17, 1e300, -1.7e308])
def test_phases_that_two_doubles_do_not_hold_are_refused(rate):
    # (from 2^53 turns on the lower one has lost half turns, and from 2^1000 on it is not finite in these units)
    w, out = (ctypes.c_double * 2)(1.0, rate), (ctypes.c_uint64 * 2)(7, 7)
    assert L.gsi_rotary_phases(w, 2, out) == 1
    assert "rate 1" in L.gsi_last_error().decode() and list(out) == [7, 7]
    with pytest.raises(gsi.GsiError, match="2\\^40"):
        gsi.Rotary.from_rates([1.0, rate], device="cpu")
