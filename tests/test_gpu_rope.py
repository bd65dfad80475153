"""GPU: pkv_rope_append and pkv_positions against a 64-bit rotation on the host.

Tolerance of a rotated value a cos - b sin: half a step of the fp16 result (2^-11 relative, 2^-25 below the smallest
normal), and in fp32 the angle (2^-25 of a half turn and 2^-32 turns: under 2^-23 rad), cos and sin (an ulp, 2^-24),
and three roundings of 2^-24, each times |a| + |b|: under 2^-21 (|a| + |b|) in all."""
import numpy as np
import pytest
import torch

from oracle import fp8
from continuous_batching_paged_ragged_gb300 import pkv

pytestmark = pytest.mark.gpu


def _rotate64(x, pos, rope):
    """x [T, H, d] fp16 -> (float64 rotated, |a| + |b| of each value's pair)."""
    c = rope.cfg
    r, d = c.rot_dim or c.head_dim, c.head_dim
    ang = pos.astype(np.float64)[:, None] * rope.frequencies()
    cos, sin = np.cos(ang)[:, None] * (c.output_scale or 1), np.sin(ang)[:, None] * (c.output_scale or 1)
    i = np.arange(r // 2)
    a, b = (2 * i, 2 * i + 1) if c.layout else (i, i + r // 2)
    y = x.astype(np.float64)
    out, amp = y.copy(), np.zeros_like(y)
    out[..., a], out[..., b] = y[..., a] * cos - y[..., b] * sin, y[..., b] * cos + y[..., a] * sin
    amp[..., a] = amp[..., b] = (np.abs(y[..., a]) + np.abs(y[..., b])) * abs(c.output_scale or 1)
    return out, amp


def _check(got, want, amp):
    err = np.abs(got.astype(np.float64) - want)
    assert np.isfinite(got.astype(np.float64)).all()
    assert (err <= 2.0**-11 * np.abs(want) * 1.001 + 2.0**-25 + 2.0**-21 * amp).all(), err.max()


def _pool(hq, hkv, d, blocks, kv_dtype=pkv.PKV_KV_F16, layers=2):
    pool = pkv.Pool(layers, hq, hkv, d, blocks, kv_dtype=kv_dtype)
    pool.buffer[:-256].random_(0, 256, generator=torch.Generator(device="cuda").manual_seed(3))
    return pool


CASES = [  # hq, hkv, d, rot, interleaved, scaling, tokens, packed
    (12, 2, 128, 128, False, "none", 1, False),
    (12, 2, 128, 64, True, "bands", 257, True),
    (4, 2, 64, 64, True, "none", 33, False),
    (4, 4, 64, 16, False, "ramp", 5, True),
    (16, 4, 256, 256, False, "linear", 100, True),
    (8, 1, 256, 64, True, "ramp", 1000, False),
    (2, 1, 64, 48, False, "none", 70, False),
    (8, 8, 128, 112, True, "bands", 2100, True),
]


@pytest.mark.parametrize("hq,hkv,d,rot,inter,scaling,T,packed", CASES)
def test_rotation_and_slots(cuda, built, hq, hkv, d, rot, inter, scaling, T, packed):
    rng = np.random.default_rng(hq * d + T)
    blocks = -(-T // 16) + 5
    pool = _pool(hq, hkv, d, blocks)
    rope = pkv.Rope(d, rot, interleaved=inter, base=10000.0, scaling=scaling, factor=4.0, original_context=4096,
                    output_scale=1.0 if scaling != "ramp" else 1.25)
    row = rng.standard_normal((T, hq + 2 * hkv, d)).astype(np.float16)
    dev = torch.from_numpy(row).cuda()
    q, k, v = dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:]
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    pos = rng.integers(0, 200000, T).astype(np.int32)
    pos[0] = 0
    if T > 2:
        pos[1], pos[2] = -7, 2**31 - 1
    slots = rng.permutation(blocks * 16)[:T].astype(np.int64)
    if T > 4:
        slots[3] = -1
    before = pool.cache_view().clone()
    out = torch.full((T, hq, d), float("nan"), dtype=torch.float16, device="cuda")
    pkv.pkv_rope_append(pool.handle, 1, rope.handle, q, q.stride(0), k, k.stride(0), v, v.stride(0),
                        torch.from_numpy(pos).cuda(), torch.from_numpy(slots).cuda(), T, out)
    torch.cuda.synchronize()
    assert pool.check() == 0 and pkv.pkv_last_launch_count(pool.handle) == 1
    # the far position's angle is good to f_i's own 2^-52: 2^31 * 2^-52 * f < 2^-21 rad, inside the tolerance's slack for
    # every other term, so that token is given twice the room
    far = np.where(pos == 2**31 - 1, 4.0, 1.0)[:, None, None]
    want, amp = _rotate64(row[:, :hq], pos, rope)
    _check(out.cpu().numpy(), want, amp * far)
    kw, ka = _rotate64(row[:, hq:hq + hkv], pos, rope)
    cache = pool.cache_view().cpu().numpy()
    want_cache = before.cpu().numpy()
    for t in range(T):
        s = slots[t]
        if s < 0:
            continue
        _check(cache[1, 0, s // 16, :, s % 16], kw[t], ka[t] * far[t])
        want_cache[1, 0, s // 16, :, s % 16] = cache[1, 0, s // 16, :, s % 16]
        want_cache[1, 1, s // 16, :, s % 16] = row[t, hq + hkv:]
    assert np.array_equal(cache.view(np.uint16), want_cache.view(np.uint16))  # values as they are, nothing else touched


@pytest.mark.parametrize("d,hq,hkv,rot,inter", [(64, 4, 2, 64, False), (128, 12, 2, 64, True), (256, 16, 4, 256, False)])
def test_8bit_is_the_rotation_followed_by_the_append(cuda, built, d, hq, hkv, rot, inter):
    """Codes and scale bytes bit for bit what pkv_append stores of the fp16 rotated keys."""
    T, blocks = 37, 4
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(T, hq, d, generator=g, device="cuda").half()
    k = (torch.randn(T, hkv, d, generator=g, device="cuda") * torch.logspace(-4, 3, T, device="cuda")[:, None, None]).half()
    v = torch.randn(T, hkv, d, generator=g, device="cuda").half()
    k[5], v[6] = 0, 0
    pos = torch.arange(T, device="cuda", dtype=torch.int32) * 911
    slots = torch.randperm(blocks * 16, generator=g, device="cuda")[:T]
    rope = pkv.Rope(d, rot, interleaved=inter)
    half = pkv.Pool(1, hq, hkv, d, blocks)
    a, b = (_pool(hq, hkv, d, blocks, pkv.PKV_KV_E4M3, 1) for _ in range(2))
    out, out8 = torch.empty_like(q), torch.empty_like(q)
    args = (rope.handle, q, hq * d, k, hkv * d, v, hkv * d, pos, slots, T)
    pkv.pkv_rope_append(half.handle, 0, *args, out)
    pkv.pkv_rope_append(a.handle, 0, *args, out8)
    kr = half.layer(0, 0)[slots // 16, :, slots % 16].contiguous()
    pkv.pkv_append(b.handle, 0, kr, v, slots, T)
    torch.cuda.synchronize()
    assert torch.equal(a.buffer, b.buffer) and torch.equal(out.view(torch.int16), out8.view(torch.int16))
    codes, scale = fp8.quantize_rows(kr.cpu().numpy())  # and the oracle's
    got = a.layer(0, 0)[slots // 16, :, slots % 16].cpu().numpy()
    assert np.array_equal(got, codes)
    assert np.array_equal(a.scales_view()[0][slots // 16, :, 0, slots % 16].cpu().numpy(), scale)


def test_in_place_keys_alone_and_far_slots(cuda, built):
    T, hq, hkv, d = 50, 12, 2, 128
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k, v = (torch.randn(T, h, d, generator=g, device="cuda").half() for h in (hq, hkv, hkv))
    pos, slots = torch.arange(T, device="cuda", dtype=torch.int32), torch.arange(T, device="cuda")
    rope = pkv.Rope(d)
    a, b = _pool(hq, hkv, d, 8), _pool(hq, hkv, d, 8)
    out, mine = torch.empty_like(q), q.clone()
    pkv.pkv_rope_append(a.handle, 0, rope.handle, q, hq * d, k, hkv * d, v, hkv * d, pos, slots, T, out)
    pkv.pkv_rope_append(b.handle, 0, rope.handle, mine, hq * d, k, hkv * d, v, hkv * d, pos, slots, T, mine)
    torch.cuda.synchronize()
    assert torch.equal(out, mine) and torch.equal(a.buffer, b.buffer)
    b.buffer.copy_(_pool(hq, hkv, d, 8).buffer)
    pkv.pkv_rope_append(b.handle, 0, rope.handle, None, 0, k, hkv * d, v, hkv * d, pos, slots, T, None)
    torch.cuda.synchronize()
    assert torch.equal(a.buffer, b.buffer)
    bad = slots.clone()
    bad[7], bad[8], bad[9] = 8 * 16, -2, 2**40  # skipped and reported; every query still rotated
    c = _pool(hq, hkv, d, 8)
    again = torch.empty_like(q)
    pkv.pkv_rope_append(c.handle, 0, rope.handle, q, hq * d, k, hkv * d, v, hkv * d, pos, bad, T, again)
    torch.cuda.synchronize()
    assert c.check() == pkv.PKV_DEVERR_SLOT_RANGE and torch.equal(out, again)
    fresh = _pool(hq, hkv, d, 8)
    want = a.cache_view().clone()
    want[0, :, 0, :, 7:10] = fresh.cache_view()[0, :, 0, :, 7:10]
    assert torch.equal(c.cache_view().view(torch.int16), want.view(torch.int16))


def test_positions(cuda, built, monkeypatch):
    pool = _pool(4, 2, 64, 4, layers=1)
    ctx, q_lens = [1, 700, 33, 16], [1, 300, 33, 2]
    starts = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    T = int(starts[-1])
    out = torch.empty(T, dtype=torch.int32, device="cuda")
    pkv.pkv_positions(pool.handle, torch.tensor(ctx, dtype=torch.int32, device="cuda"), torch.from_numpy(starts).cuda(), 4, T, out)
    want = np.concatenate([np.arange(c - n, c) for c, n in zip(ctx, q_lens)])
    assert np.array_equal(out.cpu().numpy(), want) and pool.check() == 0
    ctx[2] = 20  # fewer keys than new tokens
    pkv.pkv_positions(pool.handle, torch.tensor(ctx, dtype=torch.int32, device="cuda"), torch.from_numpy(starts).cuda(), 4, T, out)
    want[starts[2]:starts[3]] = 0
    assert np.array_equal(out.cpu().numpy(), want) and pool.check() == pkv.PKV_DEVERR_ROW_META
    monkeypatch.setenv("PKV_VALIDATE", "1")
    with pytest.raises(pkv.PkvError) as e:
        pkv.pkv_positions(pool.handle, torch.tensor(ctx, dtype=torch.int32, device="cuda"), torch.from_numpy(starts).cuda(), 4, T, out)
    assert e.value.status == pkv.PKV_ERR_INVALID_ARG


def test_refusals(cuda, built, monkeypatch):
    T, hq, hkv, d = 4, 4, 2, 64
    pool = _pool(hq, hkv, d, 4)
    rope, other = pkv.Rope(d), pkv.Rope(128)
    q, k, v = (torch.zeros(T, h, d, dtype=torch.float16, device="cuda") for h in (hq, hkv, hkv))
    pos, slots = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.arange(T, device="cuda")
    out = torch.empty_like(q)
    good = dict(layer=0, rope=rope.handle, q=q, q_stride=hq * d, k=k, k_stride=hkv * d, v=v, v_stride=hkv * d, positions=pos,
                slot_mapping=slots, num_tokens=T, q_out=out)
    for change, status in [(dict(layer=2), pkv.PKV_ERR_OUT_OF_RANGE), (dict(layer=-1), pkv.PKV_ERR_OUT_OF_RANGE),
                           (dict(rope=other.handle), pkv.PKV_ERR_INVALID_ARG), (dict(rope=None), pkv.PKV_ERR_INVALID_ARG),
                           (dict(num_tokens=-1), pkv.PKV_ERR_INVALID_ARG), (dict(k=None), pkv.PKV_ERR_INVALID_ARG),
                           (dict(q=None), pkv.PKV_ERR_INVALID_ARG), (dict(q_out=None), pkv.PKV_ERR_INVALID_ARG),
                           (dict(q_stride=hq * d - 8), pkv.PKV_ERR_INVALID_ARG), (dict(v_stride=hkv * d + 4), pkv.PKV_ERR_INVALID_ARG),
                           (dict(k=k.data_ptr() + 8), pkv.PKV_ERR_INVALID_ARG),
                           (dict(q_out=q, q_stride=hq * d + 8), pkv.PKV_ERR_INVALID_ARG), (dict(positions=None), pkv.PKV_ERR_INVALID_ARG)]:
        with pytest.raises(pkv.PkvError) as e:
            pkv.pkv_rope_append(pool.handle, **{**good, **change})
        assert e.value.status == status, change
        assert pkv.pkv_last_launch_count(pool.handle) == 0
    pkv.pkv_rope_append(pool.handle, **{**good, "num_tokens": 0})
    assert pkv.pkv_last_launch_count(pool.handle) == 0
    monkeypatch.setenv("PKV_VALIDATE", "1")
    with pytest.raises(pkv.PkvError) as e:
        pkv.pkv_rope_append(pool.handle, **{**good, "slot_mapping": slots + 4 * 16})
    assert e.value.status == pkv.PKV_ERR_OUT_OF_RANGE
    pkv.pkv_rope_append(pool.handle, **good)
