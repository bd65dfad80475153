"""Pins for the 4-bit cache oracle: scales and codes by search and exact fractions, the record's layout by hand."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import int4


def test_scale_is_the_smallest_of_eight_bits_that_covers_the_group():
    rng = np.random.default_rng(0)
    tops = np.unique(np.concatenate([rng.integers(1, 0x7C00, 400).astype(np.uint16), [1, 2, 7, 8, 0x3FF, 0x400, 0x7BFF]]))
    for a in tops.astype(np.uint16).view(np.float16).astype(np.float64):
        s = int4.scale_of(a)
        m, e = Fraction(s), 0
        assert (m * 2**24).denominator == 1 and a <= 7 * s
        n = int(m * 2**24)
        assert n >> max(0, n.bit_length() - 8) << max(0, n.bit_length() - 8) == n  # eight significant bits
        below = [x for x in int4.SCALES if x < s]
        assert 7 * below[-1] < a  # the next smaller does not cover it
        assert float(np.float16(s)) == s
    assert int4.scale_of(0.0) == 0.0


def test_codes_are_the_nearest_integers_and_nothing_is_clipped():
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((40, 64)) * np.exp2(rng.uniform(-20, 12, (40, 1)))).astype(np.float16)
    x[0] = 0
    x[1, :32] = np.float16(65504)
    x[2, :32] = np.arange(32) * np.float16(0.5) - 8          # many ties
    x[3, :32] = (rng.integers(-5, 6, 32) * 2.0**-24).astype(np.float16)
    codes, scales = int4.quantize_rows(x)
    assert codes.min() >= -7 and codes.max() <= 7
    for r in range(40):
        for i in range(64):
            assert codes[r, i] == int4.code_of(x[r, i], scales[r, i // 32]), (r, i)
            assert abs(float(x[r, i]) - codes[r, i] * scales[r, i // 32]) <= scales[r, i // 32] / 2
    assert scales[0].max() == 0 and not codes[0].any()
    half = np.float16(3.5)
    assert int4.code_of(half, 1.0) == 4 and int4.code_of(np.float16(2.5), 1.0) == 2  # ties to even


def test_a_code_times_its_scale_is_an_fp16_number():
    for s in int4.SCALES[:-256]:
        if 7 * s > 65504:
            continue
        for c in range(8):
            assert float(np.float16(c * s)) == c * s


def test_record_layout_by_hand():
    d = 64
    k = np.zeros((1, 1, d), np.float16)
    v = np.zeros((1, 1, d), np.float16)
    k[0, 0, 35] = 7.0      # group 1, value 3: byte 1's upper half; scale 1, code 7
    v[0, 0, 0] = -14.0     # group 0, value 0; scale 2, code -7
    rec = np.zeros((1, 1, 18 * d), np.uint8)
    int4.append_reference_4bit(rec, k, v, [5])
    r = rec[0, 0]
    assert r[256 + 5 * 16 + 1] == 8 | 15 << 4 and r[256 + 5 * 16] == 0x88
    assert r[8 * d + 5 * 16] == 1 | 8 << 4
    scales = r[16 * d:].view(np.float16).reshape(16, 2, d // 32)
    assert scales[5].tolist() == [[0, 1], [2, 0]] and not scales[[i for i in range(16) if i != 5]].any()
    assert not r[4 * 16:5 * 16].any() and not r[6 * 16:7 * 16].any()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_records_hold_what_rows_stand_for(d):
    rng = np.random.default_rng(d)
    k, v = (rng.standard_normal((3, 2, d)).astype(np.float16) for _ in range(2))
    rec = np.full((2, 2, 18 * d), 0xAA, np.uint8)
    int4.append_reference_4bit(rec, k, v, [17, -1, 3])
    for t, slot in ((0, 17), (2, 3)):
        for kv, x in enumerate((k, v)):
            want = int4.values(x)[t]
            for h in range(2):
                r = rec[slot // 16, h]
                codes = r[8 * d * kv:8 * d * (kv + 1)].reshape(d // 32, 16, 16)[:, slot % 16]
                c = np.stack([codes & 15, codes >> 4], -1).reshape(d).astype(float) - 8
                s = r[16 * d:].view(np.float16).reshape(16, 2, d // 32)[slot % 16, kv].astype(float)
                assert np.array_equal(c * np.repeat(s, 32), want[h])
