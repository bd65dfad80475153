"""4-bit cache oracle: integer codes with a scale for every 32 values of a cached row.

Test infrastructure only (see the package docstring).

What the pages fix: an 8-bit and a 4-bit cache as sizes to reckon with ("An advertised batch limit proves nothing until
sampled", section "Context math sets the ceiling the fields ignore"), and quantizing as the remedy when the cache is the
limit ("Continuous Batching Is Not a Bigger Batch", section "Checking it on a real system").  Readings taken:

  * 32 consecutive values of a cached row -- a token's d values of one KV head, K and V separately -- share a scale s: the
    smallest number of at most 8 significant bits, and a multiple of 2^-24, with max|x| <= 7 s (0 for 32 zeros), but at
    most 9344: magnitudes past 7 * 9344 = 65408 count as that, so that no code stands for more than fp16 holds;
  * each value is the integer nearest to x / s, ties to even, so -7 .. 7, stored plus 8; it stands for code * s;
  * a (block, KV head) is a record of 18 d bytes: K's codes [d / 32][16 tokens][16 bytes] (the lower half of a byte
    first), V's, then the scales [16 tokens][K, V][d / 32] in fp16.
"""
from __future__ import annotations

import bisect
from fractions import Fraction

import numpy as np

GROUP = 32
BS = 16
TOP = 65408.0  # the largest 7 s that is an fp16 number

# every number of at most 8 significant bits that is a multiple of 2^-24, ascending, past 65504 / 7
SCALES = sorted({m * 2.0 ** e for m in range(256) for e in range(-24, 8)})


def scale_of(amax: float) -> float:
    """The smallest scale s with amax <= 7 s, by search."""
    return SCALES[bisect.bisect_left([7 * s for s in SCALES], float(amax))]


def code_of(x: float, s: float) -> int:
    """The integer nearest to x / s, ties to even, in exact arithmetic."""
    return 0 if s == 0 else round(Fraction(float(x)) / Fraction(s))


def quantize_rows(x: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """fp16 [..., d] -> (codes int8 [..., d] in -7 .. 7, scales float64 [..., d / 32])."""
    x = np.asarray(x).astype(np.float64)
    assert np.all(np.isfinite(x)), "the 4-bit cache takes finite keys and values"
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    table = np.array(SCALES)
    s = table[np.searchsorted(7 * table, np.minimum(np.abs(g).max(-1), TOP), side="left")]
    q = np.divide(g, s[..., None], out=np.zeros_like(g), where=s[..., None] > 0)  # 11 bits over 8: a tie is exact
    return np.rint(q).astype(np.int8).reshape(x.shape), s


def dequantize_rows(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """float64 [..., d]: code * s, exactly."""
    return codes.astype(np.float64) * np.repeat(scales, GROUP, axis=-1)


def values(x: np.ndarray) -> np.ndarray:
    """What rows stand for once they are in the cache."""
    return dequantize_rows(*quantize_rows(x))


def append_reference_4bit(records: np.ndarray, k: np.ndarray, v: np.ndarray, slot_mapping) -> None:
    """In place, one layer's records uint8 [num_blocks, Hkv, 18 d]: the new tokens' rows into their slots (-1: skipped)."""
    d = k.shape[-1]
    for kv, x in enumerate((k, v)):
        codes, scales = quantize_rows(x)
        stored = (codes.astype(np.int16) + 8).astype(np.uint8)
        for t, slot in enumerate(slot_mapping):
            if slot < 0:
                continue
            blk, r = int(slot) // BS, int(slot) % BS
            for h in range(x.shape[1]):
                rec = records[blk, h]
                for i in range(0, d, 2):
                    rec[8 * d * kv + i // GROUP * 256 + r * 16 + i % GROUP // 2] = stored[t, h, i] | stored[t, h, i + 1] << 4
                at = 16 * d + (r * 2 + kv) * (d // GROUP) * 2
                rec[at:at + d // GROUP * 2] = scales[t, h].astype(np.float16).view(np.uint8)
