"""GPU: the 4-bit cache.

What is stored is compared bit for bit with the oracle's records, and reading back with what they stand for.  Attention
against the float64 oracle over those values, with A = sum of weight * |value| per output (at least |out|):
  * the softmax weight is rounded to fp16: half a step, 2^-11 A;
  * the output is rounded to fp16: 2^-11 |out|, or 2^-25 below the smallest normal;
  * scores: codes and q are multiplied exactly and added in fp32 over at most 256 terms, scaled once a group: off by less
    than 2^-24 * 256 of sum |q k| / sqrt(d) in log2 units.  The seeded values are under 2 sqrt(3), so sum |q k| / sqrt(d) <=
    12 sqrt(d) <= 192, in practice (random signs) a tenth of it: 2^-16 * 20 < 2^-11.6 at most, and 2^-14 on its weights' A
    is granted, twice (numerator and denominator) with the exponential's 2^-22 and the sums' 2^-24 a term inside it."""
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import int4
from continuous_batching_paged_ragged_gb300 import pkv, synth, workload
from helpers_gpu import host_rows, poison, run_batch, row_slice

pytestmark = pytest.mark.gpu

INT4 = pkv.PKV_KV_INT4


def _bytes(x):
    return x.contiguous().view(torch.uint8)


def _same(a, b):
    return torch.equal(_bytes(a), _bytes(b))


def _close(got, q, k, v, what="", window=1 << 30, sinks=0):
    """got fp16 [q_len, Hq, d] against the oracle over values k, v (float64), within the bound above."""
    want = oracle.window_attention_row(q, k, v, window, sinks)
    a = oracle.window_attention_row(q, k, np.abs(v), window, sinks)
    g = got.astype(np.float64)
    assert np.isfinite(g).all(), what
    bound = 2.0**-11 * 1.001 * (a + np.abs(want)) + 2.0**-13 * a + 2.0**-24
    err = np.abs(g - want)
    assert (err <= bound).all(), f"{what}: off by {err.max()}, {(err / bound).max()} of the bound"


def _many_magnitudes(rng, n, hkv, d):
    """fp16 rows scaled over 2^-20 .. 2^12, groups of a row too, with zeros, ties, the fp16 maximum and subnormals."""
    x = rng.standard_normal((n, hkv, d // 32, 32)) * np.exp2(rng.uniform(-20, 12, (n, hkv, d // 32, 1)))
    x = x.reshape(n, hkv, d).astype(np.float16)
    x[0, 0] = 0
    x[1, 0, :32] = np.arange(32) * 0.5 - 8          # ties: scale 8 / 7 rounded up; and exactly representable ones below
    x[1, 0, 32:64] = (np.arange(32) % 15 - 7) * 0.5  # scale 0.5
    x[1, 0, 32] = 3.5
    x[2, -1, 5] = 65504.0
    x[2, -1, 40] = -65504.0
    x[3, 0] = (rng.integers(-1000, 1000, d) * 2.0**-24).astype(np.float16)
    x[4, 0] = (rng.integers(-3, 4, d) * 2.0**-24).astype(np.float16)
    return x


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T", [1, 5, 73])
def test_append_and_gather_bit_exact(cuda, built, d, T):
    rng = np.random.default_rng(d + T)
    hkv, nb = 3, 9
    pool = pkv.Pool(2, hkv, hkv, d, nb, kv_dtype=INT4)
    pool.buffer[:-256].random_(0, 256, generator=torch.Generator(device="cuda").manual_seed(T))
    want = pool.cache_view().cpu().numpy().copy()
    k, v = _many_magnitudes(rng, max(T, 5), hkv, d)[:T], _many_magnitudes(rng, max(T, 5), hkv, d)[:T][::-1].copy()
    slots = rng.permutation(nb * 16)[:T].astype(np.int64)
    if T > 8:
        slots[7] = -1
    dk, dv, ds = (torch.from_numpy(x).cuda() for x in (k, v, slots))
    pkv.pkv_append(pool.handle, 1, dk, dv, ds, T)
    assert pool.check() == 0 and pkv.pkv_last_launch_count(pool.handle) == 1
    int4.append_reference_4bit(want[1], k, v, slots)
    assert np.array_equal(pool.cache_view().cpu().numpy(), want)
    # read back, every slot twice and some rows left alone
    back = np.concatenate([slots, slots[::-1], [-1, -1]])
    ko, vo = (torch.full((len(back), hkv, d), float("nan"), dtype=torch.float16, device="cuda") for _ in range(2))
    pkv.pkv_gather(pool.handle, 1, torch.from_numpy(back).cuda(), len(back), ko, vo)
    assert pool.check() == 0
    for got, x in ((ko, k), (vo, v)):
        stands = np.clip(int4.values(x), -65504, 65504)  # 7 s may pass the fp16 maximum
        g = got.cpu().numpy()
        for i, s in enumerate(back):
            if s < 0:
                assert np.isnan(g[i]).all()
            else:
                assert np.array_equal(g[i].astype(np.float64), stands[list(slots).index(s)])
    assert np.array_equal(pool.cache_view().cpu().numpy(), want)


@pytest.mark.parametrize("kv", [pkv.PKV_KV_F16, pkv.PKV_KV_E4M3, INT4])
def test_gather_reports_bad_slots_and_leaves_their_rows(cuda, built, kv):
    pool = pkv.Pool(1, 4, 2, 64, 4, kv_dtype=kv)
    k = torch.randn(3, 2, 64, device="cuda").half()
    slots = torch.tensor([0, 17, 63], device="cuda")
    pkv.pkv_append(pool.handle, 0, k, k, slots, 3)
    ko, vo = torch.full((4, 2, 64), 7.0, dtype=torch.float16, device="cuda"), torch.full((4, 2, 64), 7.0, dtype=torch.float16, device="cuda")
    pkv.pkv_gather(pool.handle, 0, torch.tensor([64, 17, -2, 2**40], device="cuda"), 4, ko, vo)
    assert pool.check() == pkv.PKV_DEVERR_SLOT_RANGE
    assert (ko[[0, 2, 3]] == 7).all() and (vo[[0, 2, 3]] == 7).all()
    assert (ko[1] - k[1]).abs().max() <= k[1].abs().max() / 14 * 1.01 and torch.equal(ko[1], vo[1])
    if kv == pkv.PKV_KV_F16:
        assert torch.equal(ko[1], k[1])


def test_gather_of_the_8bit_cache_is_its_codes_times_scales(cuda, built):
    from oracle import fp8
    rng = np.random.default_rng(0)
    k = (rng.standard_normal((20, 2, 128)) * np.exp2(rng.uniform(-8, 8, (20, 2, 1)))).astype(np.float16)
    pool = pkv.Pool(1, 4, 2, 128, 3, kv_dtype=pkv.PKV_KV_E4M3)
    dk, slots = torch.from_numpy(k).cuda(), torch.randperm(48, device="cuda")[:20]
    pkv.pkv_append(pool.handle, 0, dk, dk.flip(0).contiguous(), slots, 20)
    ko, vo = torch.empty_like(dk), torch.empty_like(dk)
    pkv.pkv_gather(pool.handle, 0, slots, 20, ko, vo)
    want = fp8.dequantize_rows(*fp8.quantize_rows(k))
    assert np.array_equal(ko.cpu().numpy().astype(np.float64), want.astype(np.float16).astype(np.float64))
    assert np.array_equal(vo.flip(0).cpu().numpy().astype(np.float64), want.astype(np.float16).astype(np.float64))


def test_refusals(cuda, built):
    pool = pkv.Pool(2, 4, 2, 64, 4, kv_dtype=INT4)
    x = torch.zeros(8, 2, 64, dtype=torch.float16, device="cuda")
    y = torch.zeros_like(x)
    s = torch.zeros(8, dtype=torch.int64, device="cuda")
    pkv.pkv_gather(pool.handle, 0, s, 0, x, y)
    assert pkv.pkv_last_launch_count(pool.handle) == 0
    for layer, args, status in [(2, (s, 1, x, y), pkv.PKV_ERR_OUT_OF_RANGE), (-1, (s, 1, x, y), pkv.PKV_ERR_OUT_OF_RANGE),
                                (0, (s, -1, x, y), pkv.PKV_ERR_INVALID_ARG), (0, (None, 1, x, y), pkv.PKV_ERR_INVALID_ARG),
                                (0, (s, 1, None, y), pkv.PKV_ERR_INVALID_ARG), (0, (s, 1, x, None), pkv.PKV_ERR_INVALID_ARG),
                                (0, (s, 1, x.data_ptr() + 2, y), pkv.PKV_ERR_INVALID_ARG), (0, (s, 1, x, x), pkv.PKV_ERR_INVALID_ARG)]:
        with pytest.raises(pkv.PkvError) as e:
            pkv.pkv_gather(pool.handle, layer, *args)
        assert e.value.status == status and pkv.pkv_last_launch_count(pool.handle) == 0
    assert pkv.pkv_pool_layer_ptr(pool.handle, 1, 0) == pool.cache_view()[1].data_ptr()
    assert pkv.pkv_pool_layer_ptr(pool.handle, 1, 1) == pool.layer(1, 1).data_ptr()
    assert pkv.pkv_pool_scales_ptr(pool.handle, 1) == pool.scales_view()[1].data_ptr()
    assert pkv.pkv_pool_layer_ptr(pool.handle, 2, 0) == 0 and pkv.pkv_pool_scales_ptr(pool.handle, 2) == 0


def test_validation_covers_the_new_calls(cuda, built, monkeypatch):
    pool = pkv.Pool(1, 4, 2, 64, 4, kv_dtype=INT4)
    x, y = (torch.zeros(2, 2, 64, dtype=torch.float16, device="cuda") for _ in range(2))
    bad = torch.tensor([3, 64], device="cuda")
    monkeypatch.setenv("PKV_VALIDATE", "1")
    for call in (lambda: pkv.pkv_append(pool.handle, 0, x, y, bad, 2), lambda: pkv.pkv_gather(pool.handle, 0, bad, 2, x, y)):
        with pytest.raises(pkv.PkvError) as e:
            call()
        assert e.value.status == pkv.PKV_ERR_OUT_OF_RANGE
    assert pool.check() == 0


# ---- attention --------------------------------------------------------------------------------------------------

ROWS = [(0, 1), (1, 1), (15, 1), (16, 1), (255, 1), (511, 1), (512, 1), (700, 1), (1023, 1), (16, 3), (0, 33),
        (240, 17), (500, 12), (1020, 6)]
SHAPES = [(12, 2, 128), (4, 2, 64), (16, 4, 256), (8, 8, 128), (8, 1, 128), (16, 2, 64), (4, 1, 256), (6, 6, 64), (6, 1, 64),
          (6, 1, 256), (8, 1, 256), (2, 1, 256), (1, 1, 256), (4, 1, 128)]


def _check_batch(batch, outs, layer=0, **kw):
    rows = host_rows(batch, layer)
    for b, (q, k, v) in enumerate(rows):
        _close(row_slice(batch, outs, b), q, int4.values(k), int4.values(v), f"row {b}", **kw)


@pytest.mark.parametrize("hq,hkv,d", SHAPES)
def test_attention(cuda, built, hq, hkv, d):
    cached, qls = zip(*ROWS)
    batch = synth.custom_batch(synth.Shape(1, hq, hkv, d), cached, qls, seed=31)
    pool, ds, outs = run_batch(batch, [0], kv_dtype=INT4)
    _check_batch(batch, outs[0])


@pytest.mark.parametrize("rows", [
    [(300, 1), (17, 1), (0, 1), (255, 1), (256, 1), (700, 1), (15, 1)],     # decode rows
    [(300, 1), (40, 3), (0, 7), (255, 2), (16, 1), (900, 4), (6, 15)],      # short chunks, too many tokens to be fused
    [(300, 1), (40, 3), (0, 7), (255, 2), (16, 1), (900, 4)],               # short chunks
    [(200, 1), (0, 40), (50, 1)],                                           # a chunk of 40: append first
])
@pytest.mark.parametrize("hq,d", [(2, 64), (12, 128), (8, 256), (16, 256)])
def test_fused_equals_append_then_attention(cuda, built, rows, hq, d):
    cached, qls = zip(*rows)
    batch = synth.custom_batch(synth.Shape(2, hq, 2, d), cached, qls, seed=17)
    pa, _, oa = run_batch(batch, [0, 1], kv_dtype=INT4, fused=False)
    pb, _, ob = run_batch(batch, [0, 1], kv_dtype=INT4, fused=True)
    if sum(qls) - len(qls) < 15:
        assert pkv.pkv_last_launch_count(pb.handle) == 1   # the append ran inside the decode launch
    assert _same(pa.cache_view(), pb.cache_view())
    for layer in (0, 1):
        assert _same(oa[layer], ob[layer])
        _check_batch(batch, ob[layer], layer)
    # and what the fused call wrote is the oracle's
    want = pa.cache_view().cpu().numpy().copy()
    for layer in (0, 1):
        for b, (q, k, v) in enumerate(host_rows(batch, layer)):
            pos = np.arange(len(k))
            slots = batch.block_tables[b][pos // 16].astype(np.int64) * 16 + pos % 16
            int4.append_reference_4bit(want[layer], k, v, slots)
    assert np.array_equal(pb.cache_view().cpu().numpy(), want)


@pytest.mark.parametrize("split", [0, 17])
@pytest.mark.parametrize("d,hq", [(64, 4), (128, 6), (256, 4)])
def test_long_rows_and_batch_invariance(cuda, built, d, hq, split):
    """A token of several splits, or of more than 32 (the merge launch), alone and among others, in another order: the same
    bits."""
    shape = synth.Shape(1, hq, 1, d)
    batch = synth.custom_batch(shape, [17000, 5, 900], [1, 1, 2], seed=3, req_ids=[5, 6, 7])
    pool, _, outs = run_batch(batch, [0], kv_dtype=INT4, split_blocks=split)
    assert pkv.pkv_last_launch_count(pool.handle) == (1 if split == 0 else 2)
    _check_batch(batch, outs[0])
    alone = synth.custom_batch(shape, [17000], [1], seed=3, req_ids=[5])
    other = synth.custom_batch(shape, [900, 40, 17000, 5], [2, 1, 1, 1], seed=3, req_ids=[7, 9, 5, 6])
    _, _, oa = run_batch(alone, [0], kv_dtype=INT4, split_blocks=split)
    _, _, oo = run_batch(other, [0], kv_dtype=INT4, fused=True, split_blocks=split)
    assert _same(oa[0][0], outs[0][0]) and _same(oo[0][3], outs[0][0])
    assert _same(oo[0][:2], outs[0][2:4]) and _same(oo[0][4], outs[0][1])


@pytest.mark.parametrize("split", [1, 2, 3, 8, 32, 33, 96, 127, 128, 129, 255, 256])
def test_split_sizes(cuda, built, split):
    batch = synth.custom_batch(synth.Shape(1, 12, 2, 128), [0, 15, 16, 31, 47, 100, 333, 2047, 2048, 4200, 9000], [1] * 11, seed=8)
    _, _, outs = run_batch(batch, [0], kv_dtype=INT4, split_blocks=split, fused=True)
    _check_batch(batch, outs[0])


def test_split_size_above_the_limit_is_refused(cuda, built):
    batch = synth.tiny_decode(0)
    pool = workload.make_pool(batch, split_blocks=257, kv_dtype=INT4)
    attn = workload.Attention(pool, workload.upload(batch, pool))
    with pytest.raises(pkv.PkvError) as e:
        attn.plan()
    assert e.value.status == pkv.PKV_ERR_UNSUPPORTED


@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (12, 2, 128), (8, 1, 128), (16, 4, 256), (8, 1, 256)])
@pytest.mark.parametrize("split,rows,most,window", [(0, 24, 40000, 0), (1, 300, 700, 0), (5, 200, 3000, 0), (0, 700, 900, 0),
                                                    (64, 300, 9000, 1500), (128, 40, 30000, 20000), (0, 200, 9000, 2048),
                                                    (256, 60, 20000, 0), (256, 60, 20000, 5000)])
def test_many_tasks_to_a_streaming_multiprocessor(cuda, built, hq, hkv, d, split, rows, most, window):
    """Tens of tasks an SM, of unequal size, whose warps hand stages, queue entries and shares to each other: no wait gives up,
    launch after launch gives the same bits, and sampled rows agree with what the cache holds."""
    gen = torch.Generator(device="cuda").manual_seed(rows)
    rng = np.random.default_rng(rows)
    ctx = np.sort(rng.integers(1, most + 1, rows))[::-1].copy()
    need = -(-ctx // 16)
    total = int(need.sum())
    tables = np.zeros((rows, int(need.max())), np.int32)
    perm, at = rng.permutation(total), 0
    for b, n in enumerate(need):
        tables[b, :n], at = perm[at:at + n], at + n
    pool = pkv.Pool(1, hq, hkv, d, total, split_blocks=split, kv_dtype=INT4)
    for at in range(0, total * 16, 65536):  # every slot
        slots = torch.arange(at, min(at + 65536, total * 16), device="cuda")
        k, v = torch.randn(2, len(slots), hkv, d, device="cuda", generator=gen).half()
        pkv.pkv_append(pool.handle, 0, k, v, slots, len(slots))
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()  # noqa: E731
    bt, cl, qsl = i32(tables), i32(ctx), i32(np.arange(rows + 1))
    q = torch.randn(rows, hq, d, device="cuda", generator=gen).half()
    if window:
        need = pkv.pkv_attention_window_workspace_bytes(pool.handle, rows, rows, bt.shape[1], window, 20)
    else:
        need = pkv.pkv_attention_workspace_bytes(pool.handle, rows, rows, bt.shape[1])
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    if window:
        pkv.pkv_attention_window_plan(pool.handle, cl, qsl, rows, rows, bt.shape[1], window, 20, ws, need)
    else:
        pkv.pkv_attention_plan(pool.handle, cl, qsl, rows, rows, bt.shape[1], ws, need)
    outs = []
    for _ in range(4):
        outs.append(torch.full_like(q, float("nan")))
        pkv.pkv_attention(pool.handle, 0, q, bt, bt.shape[1], cl, qsl, rows, rows, outs[-1], ws, need)
    assert pool.check() == 0
    assert all(_same(o, outs[0]) for o in outs[1:])
    for b in sorted({0, 1, rows - 1, *rng.integers(0, rows, 10)}):
        c = int(ctx[b])
        pos = torch.arange(c, device="cuda")
        slots = bt[b].long()[pos // 16] * 16 + pos % 16
        k, v = torch.empty(2, c, hkv, d, dtype=torch.float16, device="cuda")
        pkv.pkv_gather(pool.handle, 0, slots, c, k, v)
        s = torch.einsum("hgd,chd->hgc", q[b].double().view(hkv, hq // hkv, d), k.double()) / math.sqrt(d)
        if window:
            s[..., (pos < c - window) & (pos >= 20)] = -math.inf
        w = s.softmax(-1)
        want, a = (torch.einsum("hgc,chd->hgd", w, x).view(hq, d) for x in (v.double(), v.double().abs()))
        bound = 2.0**-11 * 1.001 * (a + want.abs()) + 2.0**-13 * a + 2.0**-24
        assert ((outs[0][b].double() - want).abs() <= bound).all(), f"row {b} of {c}"


# ---- values of any size -----------------------------------------------------------------------------------------

def _run_values(q, k, v, hq, hkv, d, ctxs, qls, fused=False, window=None, sinks=0):
    """Rows of given values (lists of fp16 arrays) through a pool whose unwritten memory is NaN; out per row."""
    need = [-(-c // 16) for c in ctxs]
    perm = np.random.default_rng(1).permutation(sum(need) + 3)
    tables = np.full((len(ctxs), max(need)), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        tables[b, :n], at = perm[at:at + n], at + n
    pool = pkv.Pool(1, hq, hkv, d, len(perm), kv_dtype=INT4)
    poison(pool)
    slot = lambda b, pos: tables[b][pos // 16].astype(np.int64) * 16 + pos % 16  # noqa: E731
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()  # noqa: E731
    cat = lambda xs: torch.from_numpy(np.concatenate(xs)).cuda()  # noqa: E731
    old = [(c - n) for c, n in zip(ctxs, qls)]
    if sum(old):
        sl = cat([slot(b, np.arange(o)) for b, o in enumerate(old)])
        pkv.pkv_append(pool.handle, 0, cat([x[:o] for x, o in zip(k, old)]), cat([x[:o] for x, o in zip(v, old)]), sl, len(sl))
    sl = cat([slot(b, np.arange(o, c)) for b, (o, c) in enumerate(zip(old, ctxs))])
    kn, vn, qn = cat([x[o:] for x, o in zip(k, old)]), cat([x[o:] for x, o in zip(v, old)]), cat(q)
    T, R, W = len(qn), len(ctxs), tables.shape[1]
    starts = np.concatenate([[0], np.cumsum(qls)])
    dt, dc, dq = i32(tables), i32(ctxs), i32(starts)
    if window:
        n = pkv.pkv_attention_window_workspace_bytes(pool.handle, R, T, W, window, sinks)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        pkv.pkv_attention_window_plan(pool.handle, dc, dq, R, T, W, window, sinks, ws, n)
    else:
        n = pkv.pkv_attention_workspace_bytes(pool.handle, R, T, W)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        pkv.pkv_attention_plan(pool.handle, dc, dq, R, T, W, ws, n)
    out = torch.full_like(qn, float("nan"))
    if fused:
        pkv.pkv_attention_append(pool.handle, 0, qn, kn, vn, sl, dt, W, dc, dq, R, T, out, ws, n)
    else:
        pkv.pkv_append(pool.handle, 0, kn, vn, sl, T)
        pkv.pkv_attention(pool.handle, 0, qn, dt, W, dc, dq, R, T, out, ws, n)
    assert pool.check() == 0
    return [out[starts[b]:starts[b + 1]].cpu().numpy() for b in range(R)]


@pytest.mark.parametrize("d,hq", [(64, 2), (128, 6), (256, 4)])
@pytest.mark.parametrize("size", [-20, -14, -6, 0, 8, 13])
@pytest.mark.parametrize("fused", [False, True])
def test_values_of_any_size(cuda, built, d, hq, size, fused):
    """V scaled as a whole, down to fp16's subnormals: the weights times value scales keep their precision, with a
    uniform softmax (where each weight is a small part of the largest) as with a peaked one."""
    rng = np.random.default_rng(size + 50)
    rows = [(1, 1), (40, 1), (700, 1), (1500, 2)]
    q, k, v = [], [], []
    for i, (ctx, n) in enumerate(rows):
        q.append((rng.standard_normal((n, hq, d)) * (0 if i == 2 else 1)).astype(np.float16))
        k.append(rng.standard_normal((ctx, 1, d)).astype(np.float16))
        x = rng.uniform(0.5, 1.0, (ctx, 1, d)) * np.where(rng.random((ctx, 1, 1)) < 0.5, 1, 1 / 64)  # one sign: a mean that stays
        v.append(np.clip(x * 2.0**size, 0, 65000).astype(np.float16))
    outs = _run_values(q, k, v, hq, 1, d, [r[0] for r in rows], [r[1] for r in rows], fused)
    for b in range(len(rows)):
        _close(outs[b], q[b], int4.values(k[b]), int4.values(v[b]), f"row {b}")


@pytest.mark.parametrize("d,hq", [(64, 8), (128, 6), (256, 2)])
def test_value_sizes_that_rise_and_fall_along_a_row(cuda, built, d, hq):
    """The softmax's reference follows the largest value scale met so far: sizes rise by 2^20 over a row, fall, or jump, and
    groups of one row differ too."""
    rng = np.random.default_rng(5)
    ctxs = [900, 900, 1300, 64]
    q, k, v = [], [], []
    for i, ctx in enumerate(ctxs):
        t = np.arange(ctx) / ctx
        size = [20 * t - 12, 8 - 20 * t, rng.uniform(-14, 8, ctx), np.where(np.arange(ctx) == 37, 10, -12)][i]
        q.append(rng.standard_normal((1, hq, d)).astype(np.float16))
        k.append(rng.standard_normal((ctx, 1, d)).astype(np.float16))
        groups = np.exp2(rng.integers(-3, 4, (ctx, 1, d // 32, 1)))
        x = rng.standard_normal((ctx, 1, d // 32, 32)) * groups * np.exp2(size)[:, None, None, None]
        v.append(x.reshape(ctx, 1, d).astype(np.float16))
    outs = _run_values(q, k, v, hq, 1, d, ctxs, [1] * 4)
    for b in range(4):
        _close(outs[b], q[b], int4.values(k[b]), int4.values(v[b]), f"row {b}")


@pytest.mark.parametrize("d,hq", [(64, 8), (128, 2), (256, 8)])
def test_zero_rows_and_zero_values(cuda, built, d, hq):
    """All-zero keys (a uniform softmax), all-zero values (an output of zero), and zero groups inside rows."""
    rng = np.random.default_rng(9)
    ctxs = [50, 50, 33, 1]
    q = [rng.standard_normal((1, hq, d)).astype(np.float16) for _ in ctxs]
    k = [rng.standard_normal((c, 1, d)).astype(np.float16) for c in ctxs]
    v = [rng.standard_normal((c, 1, d)).astype(np.float16) for c in ctxs]
    k[0][:] = 0
    v[1][:] = 0
    v[2][:, :, :32] = 0
    k[2][::2, :, 32:] = 0
    v[3][:] = 0
    outs = _run_values(q, k, v, hq, 1, d, ctxs, [1] * 4, fused=True)
    assert not outs[1].any() and not outs[3].any() and not outs[2][..., :32].any()
    for b in range(4):
        _close(outs[b], q[b], int4.values(k[b]), int4.values(v[b]), f"row {b}")


@pytest.mark.parametrize("d,hq", [(64, 8), (128, 6), (256, 4)])
def test_peaked_scores(cuda, built, d, hq):
    """One key takes nearly all the weight, scores spread over hundreds of log2 units (in the decode's and the chunks'
    softmax): the weights that underflow stay zero and nothing overflows."""
    rng = np.random.default_rng(2)
    rows = [(600, 1), (600, 1), (530, 20)]
    q, k, v = [], [], []
    for i, (ctx, n) in enumerate(rows):
        kk = rng.standard_normal((ctx, 1, d)).astype(np.float16)
        at = [3, ctx - n, 100][i]
        qq = (16 * kk[at] + rng.standard_normal((n, hq, d))).astype(np.float16)
        q.append(qq), k.append(kk), v.append(rng.standard_normal((ctx, 1, d)).astype(np.float16))
    outs = _run_values(q, k, v, hq, 1, d, [r[0] for r in rows], [r[1] for r in rows], fused=True)
    for b, (ctx, n) in enumerate(rows):
        kq, vq = int4.values(k[b]), int4.values(v[b])
        want = oracle.window_attention_row(q[b], kq, vq, 1 << 30, 0)
        a = oracle.window_attention_row(q[b], kq, np.abs(vq), 1 << 30, 0)
        # the scores' own size: fp32 sums of d terms, 2^-24 sqrt(d) of sum |q k| with random signs; four of it granted
        big = np.abs(q[b].astype(np.float64)).max() * np.abs(kq).max() * d / math.sqrt(d) * 1.4427
        bound = 2.0**-11 * 1.001 * (a + np.abs(want)) + 2.0**-24 + a * (2.0**-13 + 4 * 2.0**-24 * math.sqrt(d) * big)
        assert (np.abs(outs[b].astype(np.float64) - want) <= bound).all()


# ---- windows ----------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("hq,hkv,d", [(12, 2, 128), (8, 2, 64), (4, 1, 256), (8, 1, 256)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 3), (16, 16), (100, 4), (300, 33), (5000, 4)])
@pytest.mark.parametrize("fused", [False, True])
def test_window_with_freed_blocks_and_hidden_rubbish(cuda, built, hq, hkv, d, window, sinks, fused):
    """Blocks that no new token sees are given back (table entries of -1), and hidden keys that share a block with visible
    ones hold NaN scales."""
    cached, qls = zip(*[(0, 1), (20, 1), (700, 1), (1300, 1), (90, 5), (640, 3), (64, 40), (0, 100)])
    if fused:
        cached, qls = cached[:6], qls[:6]
    batch = synth.custom_batch(synth.Shape(1, hq, hkv, d), cached, qls, seed=12)
    rows = host_rows(batch, 0)
    pool = workload.make_pool(batch, 1, kv_dtype=INT4)
    poison(pool)
    workload.prefill_cache(pool, batch, [0])
    ds = workload.upload(batch, pool)
    scales = pool.scales_view()[0]  # [block, head, slot, K or V, group]
    for b in range(batch.num_seqs):
        ctx, n = int(batch.context_lens[b]), int(batch.q_lens[b])
        low = max(0, ctx - n + 1 - window)
        for p in range(min(sinks, low), min(low, ctx - n)):
            scales[int(batch.block_tables[b, p // 16]), :, p % 16] = float("nan")
        for j in range(-(-ctx // 16)):
            if j * 16 >= sinks and j * 16 + 16 <= low:
                pool.cache_view()[0, int(batch.block_tables[b, j])] = 0xFF
                ds.block_tables[b, j] = -1
    qs, ks, vs = workload.step_inputs(ds, [0])
    n = pkv.pkv_attention_window_workspace_bytes(pool.handle, ds.num_seqs, ds.num_tokens, ds.max_blocks, window, sinks)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    pkv.pkv_attention_window_plan(pool.handle, ds.context_lens, ds.query_start_loc, ds.num_seqs, ds.num_tokens, ds.max_blocks, window,
                                  sinks, ws, n)
    out = torch.full_like(qs[0], float("nan"))
    rest = (ds.block_tables, ds.max_blocks, ds.context_lens, ds.query_start_loc, ds.num_seqs, ds.num_tokens, out, ws, n)
    if fused:
        pkv.pkv_attention_append(pool.handle, 0, qs[0], ks[0], vs[0], ds.slot_mapping, *rest)
    else:
        pkv.pkv_append(pool.handle, 0, ks[0], vs[0], ds.slot_mapping, ds.num_tokens)
        pkv.pkv_attention(pool.handle, 0, qs[0], *rest)
    assert pool.check() == 0
    for b, (q, k, v) in enumerate(rows):
        _close(row_slice(batch, out, b), q, int4.values(k), int4.values(v), f"row {b}", window=window, sinks=sinks)


@pytest.mark.parametrize("d,hq", [(64, 8), (128, 12), (256, 8)])
def test_a_window_that_holds_the_rows_gives_the_bits_of_none(cuda, built, d, hq):
    cached, qls = zip(*[(0, 1), (17, 1), (700, 1), (900, 4), (100, 40)])
    batch = synth.custom_batch(synth.Shape(1, hq, 2, d), cached, qls, seed=4)
    pool, ds, outs = run_batch(batch, [0], kv_dtype=INT4)
    qs, _, _ = workload.step_inputs(ds, [0])
    n = pkv.pkv_attention_window_workspace_bytes(pool.handle, ds.num_seqs, ds.num_tokens, ds.max_blocks, 2000, 4)
    ws, out = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty_like(qs[0])
    pkv.pkv_attention_window_plan(pool.handle, ds.context_lens, ds.query_start_loc, ds.num_seqs, ds.num_tokens, ds.max_blocks, 2000, 4, ws, n)
    pkv.pkv_attention(pool.handle, 0, qs[0], ds.block_tables, ds.max_blocks, ds.context_lens, ds.query_start_loc, ds.num_seqs,
                      ds.num_tokens, out, ws, n)
    assert pool.check() == 0 and _same(out, outs[0])


# ---- around the attention ---------------------------------------------------------------------------------------

def test_prefill_rows_that_share_blocks(cuda, built):
    """Two chunks on one prompt's blocks, in a pool with fewer blocks than their tables have entries: the shadow is addressed
    by physical block."""
    hq, hkv, d, pre, n = 4, 2, 128, 64, 20
    rng = np.random.default_rng(3)
    k, v = (rng.standard_normal((pre + 2 * n, hkv, d)).astype(np.float16) for _ in range(2))
    q = rng.standard_normal((2 * n, hq, d)).astype(np.float16)
    pool = pkv.Pool(1, hq, hkv, d, 8, kv_dtype=INT4)
    poison(pool)
    tables = np.array([[0, 1, 2, 3, 4, 5], [0, 1, 2, 3, 6, 7]], np.int32)
    new = lambda b: tables[b][(pre + np.arange(n)) // 16].astype(np.int64) * 16 + (pre + np.arange(n)) % 16  # noqa: E731
    slots = torch.from_numpy(np.concatenate([np.arange(pre), new(0), new(1)])).cuda()
    pkv.pkv_append(pool.handle, 0, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), slots, len(slots))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    dt, dc, dq = torch.from_numpy(tables).cuda(), i32([pre + n] * 2), i32([0, n, 2 * n])
    ws_n = pkv.pkv_attention_workspace_bytes(pool.handle, 2, 2 * n, 6)
    ws, qd = torch.empty(ws_n, dtype=torch.uint8, device="cuda"), torch.from_numpy(q).cuda()
    out = torch.full_like(qd, float("nan"))
    pkv.pkv_attention_plan(pool.handle, dc, dq, 2, 2 * n, 6, ws, ws_n)
    pkv.pkv_attention(pool.handle, 0, qd, dt, 6, dc, dq, 2, 2 * n, out, ws, ws_n)
    assert pool.check() == 0
    for b in range(2):
        own = slice(pre + b * n, pre + b * n + n)
        kk, vv = (int4.values(np.concatenate([x[:pre], x[own]])) for x in (k, v))
        _close(out[b * n:(b + 1) * n].cpu().numpy(), q[b * n:(b + 1) * n], kk, vv, f"row {b}")


def test_noalloc_gives_the_planned_bits(cuda, built):
    batch = synth.custom_batch(synth.Shape(1, 12, 2, 128), [300, 15, 700, 40], [1, 1, 3, 20], seed=6)
    pool, ds, outs = run_batch(batch, [0], kv_dtype=INT4)
    qs, _, _ = workload.step_inputs(ds, [0])
    out = torch.empty_like(qs[0])
    pkv.pkv_attention_noalloc(pool.handle, 0, qs[0], ds.block_tables, ds.max_blocks, ds.context_lens, ds.query_start_loc, ds.num_seqs,
                              ds.num_tokens, out)
    assert pool.check() == 0 and _same(out, outs[0])


@pytest.mark.parametrize("fused", [False, True])
def test_a_captured_step_replays(cuda, built, fused):
    """Plan, append and attention of three layers as one graph, replayed back to back, and the same step on another stream."""
    batch = synth.custom_batch(synth.Shape(3, 12, 2, 128), [300, 15, 700, 40, 1100], [1, 1, 1, 1, 1], seed=6)
    layers = [0, 1, 2]
    pool, ds, outs = run_batch(batch, layers, kv_dtype=INT4, fused=fused)
    records = pool.cache_view().clone()
    qs, ks, vs = workload.step_inputs(ds, layers)
    attn, again = workload.Attention(pool, ds), [torch.full_like(q, float("nan")) for q in qs]
    graph, _ = workload.capture_step_graph(pool, ds, attn, qs, ks, vs, again, layers, fused=fused)
    for out in again:
        out.fill_(float("nan"))
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    assert pool.check() == 0 and _same(pool.cache_view(), records)
    assert all(_same(a, b) for a, b in zip(again, outs))


def test_records_past_32_bits_of_bytes(cuda, built):
    """A pool of 5 GB: blocks whose bytes lie past 2^32, in append, attention, gather and copies."""
    hq, hkv, d, blocks = 16, 4, 256, 290000
    pool = pkv.Pool(1, hq, hkv, d, blocks, kv_dtype=INT4)
    assert pool.cfg.num_blocks * hkv * 18 * d > 2**32 + 2**29
    rng = np.random.default_rng(8)
    ctxs, ids = [100, 37], [[289999, 289990, 12, 288000, 270000, 289001, 3], [289998, 260000, 289900]]
    tables = torch.full((2, 7), -1, dtype=torch.int32)
    for b, t in enumerate(ids):
        tables[b, :len(t)] = torch.tensor(t)
    q = [rng.standard_normal((1, hq, d)).astype(np.float16) for _ in ctxs]
    k = [rng.standard_normal((c, hkv, d)).astype(np.float16) for c in ctxs]
    v = [rng.standard_normal((c, hkv, d)).astype(np.float16) for c in ctxs]
    slots = torch.cat([tables[b][torch.arange(c) // 16].long() * 16 + torch.arange(c) % 16 for b, c in enumerate(ctxs)]).cuda()
    kd, vd, qd = (torch.from_numpy(np.concatenate(x)).cuda() for x in (k, v, q))
    pkv.pkv_append(pool.handle, 0, kd, vd, slots, len(slots))
    dt, dc = tables.cuda(), torch.tensor(ctxs, dtype=torch.int32, device="cuda")
    dq = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    n = pkv.pkv_attention_workspace_bytes(pool.handle, 2, 2, 7)
    ws, out = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty_like(qd)
    pkv.pkv_attention_plan(pool.handle, dc, dq, 2, 2, 7, ws, n)
    pkv.pkv_attention(pool.handle, 0, qd, dt, 7, dc, dq, 2, 2, out, ws, n)
    ko, vo = torch.empty_like(kd), torch.empty_like(vd)
    pkv.pkv_gather(pool.handle, 0, slots, len(slots), ko, vo)
    pkv.pkv_copy_blocks(pool.handle, torch.tensor([[289999, 289995]], dtype=torch.int32, device="cuda"), 1)
    assert pool.check() == 0
    for b in range(2):
        _close(out[b:b + 1].cpu().numpy(), q[b], int4.values(k[b]), int4.values(v[b]), f"row {b}")
    assert np.array_equal(ko.cpu().numpy().astype(np.float64), int4.values(np.concatenate(k)))
    assert np.array_equal(vo.cpu().numpy().astype(np.float64), int4.values(np.concatenate(v)))
    assert torch.equal(pool.cache_view()[0, 289999], pool.cache_view()[0, 289995])


# ---- block calls ------------------------------------------------------------------------------------------------

def _rows_view(records, d):
    """Records [L, NB, H, 18 d] on the host as [L, NB, H, token, bytes of the token]."""
    lead = records.shape[:-1]
    codes = records[..., :16 * d].reshape(*lead, d // 16, 16, 16)
    scales = records[..., 16 * d:].reshape(*lead, 16, d // 8)
    return np.concatenate([np.moveaxis(codes, -3, -2).reshape(*lead, 16, d), scales], -1)


@pytest.mark.parametrize("layers,hkv,d", [(1, 1, 64), (3, 2, 128), (2, 5, 256), (28, 2, 128)])
def test_copy_fork_and_compact(cuda, built, layers, hkv, d):
    rng = np.random.default_rng(layers)
    blocks = 60
    pool = pkv.Pool(layers, hkv, hkv, d, blocks, kv_dtype=INT4)
    pool.buffer[:-256].random_(0, 256, generator=torch.Generator(device="cuda").manual_seed(1))
    host = lambda: _rows_view(pool.cache_view().cpu().numpy(), d)  # noqa: E731
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()  # noqa: E731
    want = host()
    # copies
    ids = rng.permutation(blocks)
    pairs = np.stack([ids[:9], ids[9:18]], 1)
    pairs[8, 0] = pairs[0, 0]
    pkv.pkv_copy_blocks(pool.handle, i32(np.concatenate([pairs, [[-1, 5]]])), 10)
    for s, t in pairs:
        want[:, t] = want[:, s]
    assert pool.check() == 0 and np.array_equal(host(), want)
    # forks: every tail of 1 .. 15 rows, and none
    ctx = np.array(list(range(1, 17)) + [0] * 16, np.int32)
    ids = rng.permutation(blocks)
    tables = np.full((32, 2), -1, np.int32)
    tables[:16, 0] = ids[:16]
    forks = [(b, 16 + b, int(ids[16 + b]) if b < 15 else -1) for b in range(16)]
    dt, dc = i32(tables), i32(ctx)
    pkv.pkv_fork_rows(pool.handle, dt, 2, dc, 32, i32(forks), 16)
    for b, _, t in forks[:15]:
        want[:, t, :, :b + 1] = want[:, ids[b], :, :b + 1]
    assert pool.check() == 0 and np.array_equal(host(), want)
    assert dt.cpu().numpy()[16:31, 0].tolist() == [f[2] for f in forks[:15]] and dt.cpu().numpy()[31, 0] == ids[15]
    # compaction
    tables = np.full((3, 7), -1, np.int32)
    tables.ravel()[:18] = rng.permutation(blocks)[:18]
    held = sorted(int(x) for x in tables.ravel() if x >= 0)
    moves = dict(zip([x for x in held if x >= 18], [x for x in range(18) if x not in held]))
    n = pkv.pkv_compact_workspace_bytes(pool.handle)
    new, remap, live, ws = i32(np.zeros((3, 7))), i32(np.zeros(blocks)), i32([0]), torch.empty(n, dtype=torch.uint8, device="cuda")
    pkv.pkv_compact(pool.handle, i32(tables), 7, 3, new, remap, live, ws, n)
    for s, t in moves.items():
        want[:, t] = want[:, s]
    assert pool.check() == 0 and int(live) == 18 and np.array_equal(host(), want)
    assert new.cpu().numpy().tolist() == [[moves.get(x, x) for x in r] for r in tables.tolist()]


def test_forked_rows_go_on_by_themselves(cuda, built):
    """Prompt, fork, one more token each through the fused call, compaction, another token: against the oracle."""
    hq, hkv, d = 12, 2, 128
    rng = np.random.default_rng(4)
    pool = pkv.Pool(1, hq, hkv, d, 30, kv_dtype=INT4)
    poison(pool)
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()  # noqa: E731
    tables, ctx = np.full((3, 6), -1, np.int32), np.array([0, 0, 0], np.int32)
    tables[0, :3] = [29, 11, 17]
    dt = i32(tables)
    k, v = ([rng.standard_normal((39, hkv, d)).astype(np.float16)] * 3 for _ in range(2))
    prompt = torch.from_numpy(tables[0][np.arange(39) // 16].astype(np.int64) * 16 + np.arange(39) % 16).cuda()
    pkv.pkv_append(pool.handle, 0, torch.from_numpy(k[0]).cuda(), torch.from_numpy(v[0]).cuda(), prompt, 39)
    dc = i32([39, 0, 0])
    pkv.pkv_fork_rows(pool.handle, dt, 6, dc, 3, i32([[0, 1, 5], [0, 2, 28]]), 2)
    starts = i32([0, 1, 2, 3])
    n = pkv.pkv_attention_workspace_bytes(pool.handle, 3, 3, 6)
    ws, slots = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty(3, dtype=torch.int64, device="cuda")
    for step in range(3):
        q, kn, vn = (rng.standard_normal((3, h, d)).astype(np.float16) for h in (hq, hkv, hkv))
        k = [np.concatenate([k[b], kn[b:b + 1]]) for b in range(3)]
        v = [np.concatenate([v[b], vn[b:b + 1]]) for b in range(3)]
        dc += 1
        pkv.pkv_slot_mapping(pool.handle, dt, 6, dc, starts, 3, 3, slots)
        pkv.pkv_attention_plan(pool.handle, dc, starts, 3, 3, 6, ws, n)
        qd, out = torch.from_numpy(q).cuda(), torch.empty(3, hq, d, dtype=torch.float16, device="cuda")
        pkv.pkv_attention_append(pool.handle, 0, qd, torch.from_numpy(kn).cuda(), torch.from_numpy(vn).cuda(), slots, dt, 6, dc, starts, 3, 3,
                                 out, ws, n)
        assert pool.check() == 0
        for b in range(3):
            _close(out[b:b + 1].cpu().numpy(), q[b:b + 1], int4.values(k[b]), int4.values(v[b]), f"step {step} row {b}")
        m = pkv.pkv_compact_workspace_bytes(pool.handle)
        new, remap, live, cw = torch.empty_like(dt), i32(np.zeros(30)), i32([0]), torch.empty(m, dtype=torch.uint8, device="cuda")
        pkv.pkv_compact(pool.handle, dt, 6, 3, new, remap, live, cw, m)
        dt = new
    assert int(live) == 5
