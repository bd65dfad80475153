"""CPU: the rotary handle's frequencies against their formulas, and the refusals made before any launch."""
import ctypes
import math

import numpy as np
import pytest

from continuous_batching_paged_ragged_gb300 import pkv


def _formula(d, r, base, scaling, factor, original, lo_turns, hi_turns):
    out = []
    for i in range(r // 2):
        f = base ** (-2.0 * i / r)
        w = 1.0
        if scaling == "linear":
            w = 0.0
        elif scaling == "bands":
            w = min(1.0, max(0.0, (original * f / (2 * math.pi) - lo_turns) / (hi_turns - lo_turns)))
        elif scaling == "ramp":
            def pair(t):
                return r * math.log(original / (2 * math.pi * t)) / (2 * math.log(base))
            lo, hi = max(math.floor(pair(hi_turns)), 0), min(math.ceil(pair(lo_turns)), r - 1)
            w = 1.0 - min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
        out.append(w * f + (1 - w) * f / factor if w < 1 else f)
    return np.array(out)


@pytest.mark.parametrize("scaling,turns", [("none", (0, 0)), ("linear", (0, 0)), ("bands", (1, 4)), ("bands", (0.5, 9)),
                                           ("ramp", (1, 32)), ("ramp", (2, 16))])
@pytest.mark.parametrize("d,r,base", [(64, 64, 10000.0), (128, 64, 500000.0), (256, 16, 10000.0), (128, 128, 1.5)])
def test_frequencies(built, scaling, turns, d, r, base):
    rope = pkv.Rope(d, r, base=base, scaling=scaling, factor=8.0, original_context=8192, low_turns=turns[0],
                    high_turns=turns[1])
    want = _formula(d, r, base, scaling, 8.0, 8192, *turns)
    # the host's pow and log against Python's: each within an ulp or two of 2^-52, amplified by the weights' slope
    np.testing.assert_allclose(rope.frequencies(), want, rtol=1e-12)
    rope.close()


def test_default_turns_are_the_documented_ones(built):
    for scaling, turns in (("bands", (1, 4)), ("ramp", (1, 32))):
        a = pkv.Rope(128, scaling=scaling, factor=4.0, original_context=4096).frequencies()
        b = pkv.Rope(128, scaling=scaling, factor=4.0, original_context=4096, low_turns=turns[0], high_turns=turns[1])
        assert np.array_equal(a, b.frequencies())


@pytest.mark.parametrize("change,status", [
    (dict(head_dim=96), pkv.PKV_ERR_UNSUPPORTED), (dict(rot_dim=24), pkv.PKV_ERR_UNSUPPORTED),
    (dict(rot_dim=144), pkv.PKV_ERR_INVALID_ARG), (dict(rot_dim=-16), pkv.PKV_ERR_INVALID_ARG),
    (dict(layout=2), pkv.PKV_ERR_INVALID_ARG), (dict(scaling=4), pkv.PKV_ERR_INVALID_ARG),
    (dict(base=1.0), pkv.PKV_ERR_INVALID_ARG), (dict(base=float("nan")), pkv.PKV_ERR_INVALID_ARG),
    (dict(scaling=1, factor=0.0), pkv.PKV_ERR_INVALID_ARG), (dict(scaling=2, original_context=0.0), pkv.PKV_ERR_INVALID_ARG),
    (dict(scaling=3, low_turns=4.0, high_turns=4.0), pkv.PKV_ERR_INVALID_ARG),
    (dict(output_scale=float("inf")), pkv.PKV_ERR_INVALID_ARG)])
def test_bad_configurations_are_refused(built, change, status):
    args = dict(head_dim=128, rot_dim=128, layout=0, scaling=0, base=1e4, factor=2.0, original_context=4096.0,
                low_turns=0.0, high_turns=0.0, output_scale=0.0)
    args.update(change)
    h = ctypes.c_void_p()
    assert built.pkv_rope_create(ctypes.byref(pkv.pkv_rope_config(**args)), ctypes.byref(h)) == status
    assert not h.value and built.pkv_last_error()


def test_calls_without_a_pool_are_refused(built):
    n = None
    assert built.pkv_rope_append(n, 0, n, n, 0, n, 0, n, 0, n, n, 1, n, n) == pkv.PKV_ERR_INVALID_ARG
    assert built.pkv_positions(n, n, n, 1, 1, n, n) == pkv.PKV_ERR_INVALID_ARG
    assert built.pkv_copy_blocks(n, n, 1, n) == pkv.PKV_ERR_INVALID_ARG
    assert built.pkv_fork_rows(n, n, 1, n, 1, n, 1, n) == pkv.PKV_ERR_INVALID_ARG
    assert built.pkv_compact(n, n, 1, 1, n, n, n, n, 0, n) == pkv.PKV_ERR_INVALID_ARG
    assert built.pkv_compact_workspace_bytes(n) == 0
    assert built.pkv_rope_frequencies(n, None, 0) == 0
