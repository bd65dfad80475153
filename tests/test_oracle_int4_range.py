"""The ends of fp16's range in the 4-bit cache oracle."""
import numpy as np

from oracle import int4


def test_a_code_times_its_scale_is_an_fp16_number_at_every_magnitude():
    """Every finite fp16 magnitude as a group's largest: all 15 codes of its scale are fp16 numbers, the value is held within
    half a step, and the scale is the least that covers it, or 9344 (65408 / 7), the largest of eight bits whose codes all are."""
    tops = np.arange(0, 0x7C00, dtype=np.uint16).view(np.float16)
    x = np.zeros((len(tops), int4.GROUP), np.float16)
    x[:, 3] = tops
    x[:, 17] = -tops
    codes, scales = int4.quantize_rows(x)
    s = scales[:, 0]
    products = s[:, None] * np.arange(-7, 8)
    with np.errstate(over="ignore"):
        assert np.array_equal(products.astype(np.float16).astype(np.float64), products)
    held = int4.dequantize_rows(codes, scales)
    assert (np.abs(held - x.astype(np.float64)) <= s[:, None] / 2).all() and np.abs(codes).max() == 7
    covered = tops <= 65408
    assert (tops[covered].astype(np.float64) <= 7 * s[covered]).all() and (s[~covered] == 9344).all()
    assert (~covered).sum() == 3 and s[covered].max() == 9344
    assert all(s[i] == int4.scale_of(float(tops[i])) for i in range(0, len(tops) - 3, 97))
