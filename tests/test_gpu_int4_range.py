"""GPU: the ends of fp16's range on the 4-bit cache.  A code stands for code * s, an fp16 number, and every reader gives that:
the decode after an append or with it fused, prompt chunks, and pkv_gather.

Exactness: with keys of zero every score is 0, the softmax's weights are one power of two, and a row of equal values v has the
output n v / n, off by the division's 2^-23 of v: the fp16 number v itself."""
import numpy as np
import pytest
import torch

import oracle
import test_gpu_int4 as int4_tests
from oracle import int4
from continuous_batching_paged_ragged_gb300 import pkv

pytestmark = pytest.mark.gpu

INT4 = pkv.PKV_KV_INT4
LARGE = [65504.0, -65504.0, 65472.0, 65440.0, 65408.0, 65376.0, 60000.0, 30000.0]
LAYOUTS = [(64, 2), (64, 8), (128, 6), (128, 1), (256, 4), (256, 8)]


def _equal_rows(sizes, d, hq):
    """(q, k, v, rows): for every size a row of one key, one of 37 with a new token, and one of 30 with 20."""
    rows, q, k, v = [], [], [], []
    for size in sizes:
        for ctx, n in ((1, 1), (37, 1), (30, 20)):
            rows.append((ctx, n))
            q.append(np.random.default_rng(ctx).standard_normal((n, hq, d)).astype(np.float16))
            k.append(np.zeros((ctx, 1, d), np.float16))
            v.append(np.full((ctx, 1, d), size, np.float16))
            v[-1][..., 1::2] *= np.float16(-1)
    return q, k, v, rows


def _check_equal_rows(sizes, d, hq, fused, **window):
    """All rows in one pass (the chunks of 20 among them), and the single tokens by themselves (fused: one launch)."""
    q, k, v, rows = _equal_rows(sizes, d, hq)
    for pick in (range(len(rows)), [i for i, r in enumerate(rows) if r[1] == 1]):
        outs = int4_tests._run_values([q[i] for i in pick], [k[i] for i in pick], [v[i] for i in pick], hq, 1, d,
                                      [rows[i][0] for i in pick], [rows[i][1] for i in pick], fused, **window)
        for out, i in zip(outs, pick):
            want = int4.values(v[i][:1])[0, 0]
            assert (out.astype(np.float64) == want).all(), (rows[i], float(v[i][0, 0, 0]), np.unique(out), np.unique(want))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_large_values_stored_and_read_back(cuda, built, d):
    x = np.random.default_rng(d).standard_normal((len(LARGE), 2, d)).astype(np.float16)
    for i, size in enumerate(LARGE):
        x[i, i % 2, i::7] = size
        x[i, 1 - i % 2, 5 * i] = -size
    pool = pkv.Pool(1, 2, 2, d, 2, kv_dtype=INT4)
    pool.buffer[:-256].zero_()
    want = pool.cache_view().cpu().numpy().copy()
    slots = np.arange(len(x), dtype=np.int64) * 3
    dx, ds = torch.from_numpy(x).cuda(), torch.from_numpy(slots).cuda()
    pkv.pkv_append(pool.handle, 0, dx, dx.flip(0).contiguous(), ds, len(x))
    int4.append_reference_4bit(want[0], x, x[::-1].copy(), slots)
    assert pool.check() == 0 and np.array_equal(pool.cache_view().cpu().numpy(), want)
    ko, vo = torch.empty_like(dx), torch.empty_like(dx)
    pkv.pkv_gather(pool.handle, 0, ds, len(x), ko, vo)
    assert np.array_equal(ko.cpu().numpy().astype(np.float64), int4.values(x))
    assert np.array_equal(vo.flip(0).cpu().numpy().astype(np.float64), int4.values(x))


@pytest.mark.parametrize("d,hq", LAYOUTS)
@pytest.mark.parametrize("fused", [False, True])
def test_large_values_attended(cuda, built, d, hq, fused):
    _check_equal_rows(LARGE, d, hq, fused)
    _check_equal_rows(LARGE[:3], d, hq, fused, window=9, sinks=3)


@pytest.mark.parametrize("d,hq", LAYOUTS)
@pytest.mark.parametrize("fused", [False, True])
def test_large_keys_attended(cuda, built, d, hq, fused):
    """Keys at the top of the range against small queries, in decode rows and a chunk: scores of the values that are held."""
    rng = np.random.default_rng(3)
    rows, q, k, v = [(1, 1), (40, 1), (37, 2), (50, 20)], [], [], []
    for ctx, n in rows:
        q.append((rng.standard_normal((n, hq, d)) * 2.0**-14).astype(np.float16))
        x = rng.standard_normal((ctx, 1, d)).astype(np.float16)
        x[::3, :, 7] = np.float16(65504)
        x[1::5, :, 40] = np.float16(-65472)
        x[2::4, :, 41] = np.float16(65440)
        k.append(x)
        v.append(rng.standard_normal((ctx, 1, d)).astype(np.float16))
    outs = int4_tests._run_values(q, k, v, hq, 1, d, [r[0] for r in rows], [r[1] for r in rows], fused)
    for b in range(len(rows)):
        int4_tests._close(outs[b], q[b], int4.values(k[b]), int4.values(v[b]), f"row {b}")


SMALL = [m * 2.0**-24 for m in (1, -3, 5, 7, 9, -15, 33, 127, 1021)] + [2.0**-14 + 2.0**-24, 7 * 1.5 * 2.0**-15]


@pytest.mark.parametrize("d,hq", LAYOUTS)
@pytest.mark.parametrize("fused", [False, True])
def test_small_values_attended(cuda, built, d, hq, fused):
    """Down to fp16's smallest number."""
    _check_equal_rows(SMALL, d, hq, fused)
    _check_equal_rows(SMALL[:4], d, hq, fused, window=9, sinks=3)


@pytest.mark.parametrize("d,hq", LAYOUTS)
@pytest.mark.parametrize("bits", [2, 4, 7, 10, 12])
def test_one_key_of_small_values_is_its_values(cuda, built, d, hq, bits):
    """A row of one key has the output that the key's value stands for, whatever the group holds beside it; a row of 40 is
    off by its weights' rounding and half of fp16's smallest number."""
    rng = np.random.default_rng(bits)
    rows = [(1, 1), (40, 1), (1, 1), (25, 20)]
    q = [rng.standard_normal((n, hq, d)).astype(np.float16) for _, n in rows]
    k = [rng.standard_normal((c, 1, d)).astype(np.float16) for c, _ in rows]
    v = [(rng.integers(-2**bits, 2**bits + 1, (c, 1, d)) * 2.0**-24).astype(np.float16) for c, _ in rows]
    outs = int4_tests._run_values(q, k, v, hq, 1, d, [r[0] for r in rows], [r[1] for r in rows])
    for b in range(4):
        held = int4.values(v[b])
        if rows[b][0] == 1:
            assert (outs[b].astype(np.float64) == held[0, 0]).all(), b
            continue
        want, a = (oracle.window_attention_row(q[b], int4.values(k[b]), x, 1 << 30, 0) for x in (held, np.abs(held)))
        assert (np.abs(outs[b].astype(np.float64) - want) <= a * (2.0**-11 * 1.001 + 2.0**-13) + 2.0**-25 * 1.001).all(), b


@pytest.mark.parametrize("d,hq", LAYOUTS)
@pytest.mark.parametrize("size", [1000.0, 8000.0, 20000.0, 60000.0])
@pytest.mark.parametrize("fused", [False, True])
def test_large_scores(cuda, built, d, hq, size, fused):
    """Queries and keys of one direction, scores up to 2^37: the largest key takes all the weight, wherever it lies, and keys of
    equal scores share it.  The next score is a thousandth of the largest away or more, more than 2^10 log2 units."""
    rng = np.random.default_rng(int(size) + d)
    rows, q, k, v = [(1, 1), (40, 1), (700, 1), (700, 1), (700, 1), (90, 2)], [], [], []
    for i, (ctx, n) in enumerate(rows):
        sign = np.where(rng.random(d) < 0.5, 1.0, -1.0)
        x = sign * size * rng.uniform(-0.9, 0.9, (ctx, 1, 1))
        x[[0, 3, ctx - n, ctx // 2, ctx - n, 5][i]] = sign * size
        if i == 4:
            x[:] = sign * size       # a uniform softmax of scores far from zero
        q.append((np.ones((n, hq, 1)) * sign * (-size if i == 4 else size)).astype(np.float16))
        k.append(x.astype(np.float16))
        v.append(rng.standard_normal((ctx, 1, d)).astype(np.float16))
    outs = int4_tests._run_values(q, k, v, hq, 1, d, [r[0] for r in rows], [r[1] for r in rows], fused)
    for b in range(len(rows)):
        held = int4.values(v[b])
        want, a = (oracle.window_attention_row(q[b], int4.values(k[b]), x, 1 << 30, 0) for x in (held, np.abs(held)))
        # weights: 1 each (exact) or 0; the output's rounding and the sums' 2^-24 a term
        assert (np.abs(outs[b].astype(np.float64) - want) <= 2.0**-11 * 1.001 * np.abs(want) + 2.0**-14 * a + 2.0**-25).all(), b
