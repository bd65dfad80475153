"""CPU: rotary configurations at the ends of their ranges, and the stated precision of the frequencies."""
import ctypes
from decimal import Decimal, getcontext

import numpy as np
import pytest

from continuous_batching_paged_ragged_gb300 import pkv

TINY = 5e-324  # the smallest positive double


def _create(built, **change):
    args = dict(head_dim=128, rot_dim=128, layout=0, scaling=0, base=1e4, factor=2.0, original_context=4096.0, low_turns=0.0,
                high_turns=0.0, output_scale=0.0)
    args.update(change)
    h = ctypes.c_void_p()
    status = built.pkv_rope_create(ctypes.byref(pkv.pkv_rope_config(**args)), ctypes.byref(h))
    if status == pkv.PKV_OK:
        f = pkv.pkv_rope_frequencies(h.value)
        built.pkv_rope_destroy(h)
        return status, f
    assert not h.value and built.pkv_last_error()
    return status, None


@pytest.mark.parametrize("change", [dict(scaling=1, factor=TINY), dict(scaling=2, factor=TINY), dict(scaling=3, factor=TINY),
                                    dict(output_scale=1e39), dict(output_scale=-1e300)])
def test_what_does_not_fit_is_refused(built, change):
    """A frequency past the largest double, or a scale past the largest fp32 value: every rotated value would be NaN."""
    assert _create(built, **change)[0] == pkv.PKV_ERR_INVALID_ARG


@pytest.mark.parametrize("change", [dict(scaling=1, factor=1e300), dict(scaling=1, factor=1e-308, base=1.0000001), dict(scaling=2, low_turns=TINY, high_turns=1e308),
                                    dict(scaling=3, low_turns=1e307, high_turns=1e308), dict(scaling=3, original_context=1e308),
                                    dict(scaling=2, original_context=TINY), dict(base=1e308), dict(output_scale=3e38)])
def test_far_but_finite_is_accepted(built, change):
    status, f = _create(built, **change)
    assert status == pkv.PKV_OK and np.all(np.isfinite(f)) and np.all(f >= 0)


@pytest.mark.parametrize("base,r,factor", [(10000.0, 128, 0), (500000.0, 64, 0), (1.5, 256, 0), (1000000.0, 128, 8)])
def test_frequencies_have_the_stated_precision(built, base, r, factor):
    """pkv.h: 2^-22 turns at any int32 position.  Against 50 decimal digits: f / 2 pi off by at most 2^-53, f itself by 2^-51."""
    getcontext().prec = 50
    _, f = _create(built, head_dim=256, rot_dim=r, base=base, scaling=1 if factor else 0, factor=float(factor or 1))
    for i, x in enumerate(f):
        want = (-Decimal(2 * i) / r * Decimal(base).ln()).exp() / (factor or 1)
        assert abs(Decimal(float(x)) - want) <= want * Decimal(2) ** -51
