"""GPU: pkv_norm_rope_append against 64-bit norms and rotations on the host.

Tolerance: half a step of the fp16 result (2^-11 relative, 2^-25 below the smallest normal), what a rotation in fp32 costs
(2^-21 (|a| + |b|), derived beside the rotation's tests), and of the norm in fp32: the mean square is a chain of 16 fused
steps and up to four sums over lanes, 2^-24 each (under 20 * 2^-24, half of it in its root), root, quotient and three
products 2^-24 each: under 2^-19.9 of the value; 2^-19 (|a| + |b|) is granted."""
import numpy as np
import pytest
import torch

from oracle import int4
from continuous_batching_paged_ragged_gb300 import pkv

pytestmark = pytest.mark.gpu

KINDS = [pkv.PKV_KV_F16, pkv.PKV_KV_E4M3, pkv.PKV_KV_INT4]


def _bytes(x):
    return x.contiguous().view(torch.uint8)


def _want(x, w, eps, offset, pos, rope):
    """(float64 result, |a| + |b| of each value's pair) of x [T, H, d] fp16; w None: no norm."""
    y = x.astype(np.float64)
    d = y.shape[-1]
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * (offset + w.astype(np.float64))
    out, amp = y.copy(), np.abs(y)
    if rope is not None:
        c = rope.cfg
        r, scale = c.rot_dim or d, c.output_scale or 1
        ang = pos.astype(np.float64)[:, None] * rope.frequencies()
        cos, sin = np.cos(ang)[:, None] * scale, np.sin(ang)[:, None] * scale
        i = np.arange(r // 2)
        a, b = (2 * i, 2 * i + 1) if c.layout else (i, i + r // 2)
        out[..., a], out[..., b] = y[..., a] * cos - y[..., b] * sin, y[..., b] * cos + y[..., a] * sin
        amp[..., a] = amp[..., b] = (np.abs(y[..., a]) + np.abs(y[..., b])) * scale
    return out, amp


def _check(got, want, amp):
    """Within the tolerance; a result past the fp16 maximum by half a step (65520) or more rounds to infinity."""
    g = got.astype(np.float64)
    slack = (2.0**-21 + 2.0**-19) * amp
    past = np.abs(want) >= 65520
    assert np.isfinite(g[np.abs(want) < 65520 - slack]).all() and not np.isnan(g).any()
    assert (np.sign(g) == np.sign(want))[past].all() and np.isinf(g[past & (np.abs(want) > 65520 + slack)]).all()
    near = np.isfinite(g) & ~past
    err, bound = np.abs(g - want)[near], (2.0**-11 * np.abs(want) * 1.001 + 2.0**-25 + slack)[near]
    assert (err <= bound).all(), ((err / bound).max(), err.max())


CASES = [  # hq, hkv, d, rot (None: no rotation), interleaved, scaling, tokens, packed, norms, eps, offset
    (12, 2, 128, 128, False, "none", 1, False, "qk", 1e-6, 0.0),
    (12, 2, 128, 64, True, "bands", 257, True, "qk", 1e-5, 1.0),
    (4, 2, 64, 64, True, "none", 33, False, "q", 1e-6, 0.0),
    (4, 4, 64, 16, False, "ramp", 5, True, "k", 1e-6, 0.0),
    (16, 4, 256, 256, False, "linear", 100, True, "qk", 1e-6, 1.0),
    (8, 1, 256, 64, True, "ramp", 1000, False, "qk", 1e-2, 0.5),
    (2, 1, 64, 48, False, "none", 70, False, "qk", 1e-6, 0.0),
    (8, 8, 128, 112, True, "bands", 2100, True, "qk", 1e-6, 0.0),
    (6, 1, 128, None, False, "none", 3, True, "qk", 1e-6, 0.0),
    (48, 8, 256, None, False, "none", 31, False, "k", 1e-6, 1.0),
    (1, 1, 64, 32, True, "none", 2, True, "qk", 1e-6, 0.0),
]


def _inputs(rng, T, hq, hkv, d):
    row = rng.standard_normal((T, hq + 2 * hkv, d)) * np.exp2(rng.uniform(-8, 6, (T, hq + 2 * hkv, 1)))
    row = row.astype(np.float16)
    row[0, 0], row[T // 2, hq] = 0, 0                       # zero heads stay zero
    row[-1, -1] = np.float16(60000)
    if T > 2:
        row[1, 0, 1:], row[1, hq, :] = 0, np.float16(60000)  # one value alone; the largest mean square
        row[2, 0] = (rng.integers(-9, 9, d) * 2.0**-24).astype(np.float16)
    return row


def _rope(d, rot, inter, scaling):
    if rot is None:
        return None
    return pkv.Rope(d, rot, interleaved=inter, scaling=scaling, factor=4.0, original_context=4096,
                    output_scale=1.0 if scaling != "ramp" else 1.25)


@pytest.mark.parametrize("hq,hkv,d,rot,inter,scaling,T,packed,norms,eps,offset", CASES)
def test_norms_rotation_and_slots(cuda, built, hq, hkv, d, rot, inter, scaling, T, packed, norms, eps, offset):
    rng = np.random.default_rng(hq * d + T)
    blocks = -(-T // 16) + 5
    pool = pkv.Pool(2, hq, hkv, d, blocks)
    pool.buffer[:-256].random_(0, 256, generator=torch.Generator(device="cuda").manual_seed(3))
    rope = _rope(d, rot, inter, scaling)
    row = _inputs(rng, T, hq, hkv, d)
    dev = torch.from_numpy(row).cuda()
    q, k, v = dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:]
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    wq, wk = ((1 - offset + 0.3 * rng.standard_normal(d)).astype(np.float16) for _ in range(2))
    pos = rng.integers(0, 200000, T).astype(np.int32)
    if T > 2:
        pos[1] = -7
    slots = rng.permutation(blocks * 16)[:T].astype(np.int64)
    if T > 4:
        slots[3] = -1
    before = pool.cache_view().clone()
    out = torch.full((T, hq, d), float("nan"), dtype=torch.float16, device="cuda")
    pkv.pkv_norm_rope_append(pool.handle, 1, rope and rope.handle, torch.from_numpy(wq).cuda() if "q" in norms else None,
                             torch.from_numpy(wk).cuda() if "k" in norms else None, eps, offset, q, q.stride(0), k, k.stride(0), v,
                             v.stride(0), torch.from_numpy(pos).cuda() if rope else None, torch.from_numpy(slots).cuda(), T, out)
    assert pool.check() == 0 and pkv.pkv_last_launch_count(pool.handle) == 1
    want, amp = _want(row[:, :hq], wq if "q" in norms else None, eps, offset, pos, rope)
    _check(out.cpu().numpy(), want, amp)
    kw, ka = _want(row[:, hq:hq + hkv], wk if "k" in norms else None, eps, offset, pos, rope)
    cache, want_cache = pool.cache_view().cpu().numpy(), before.cpu().numpy()
    for t, s in enumerate(slots):
        if s < 0:
            continue
        _check(cache[1, 0, s // 16, :, s % 16], kw[t], ka[t])
        want_cache[1, 0, s // 16, :, s % 16] = cache[1, 0, s // 16, :, s % 16]
        want_cache[1, 1, s // 16, :, s % 16] = row[t, hq + hkv:]
    assert np.array_equal(cache.view(np.uint16), want_cache.view(np.uint16))  # values as they are, nothing else touched


@pytest.mark.parametrize("kv", KINDS[1:])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("d,hq,hkv,rot,inter", [(64, 4, 2, 64, False), (64, 2, 2, 16, False), (64, 2, 1, 48, True), (128, 12, 2, 128, False),
                                                (128, 6, 1, 80, False), (128, 4, 2, 112, False), (256, 16, 4, 256, True),
                                                (256, 4, 1, 96, False), (256, 2, 1, 240, False)])
def test_quantized_caches_hold_the_rounded_rotated_keys(cuda, built, d, hq, hkv, rot, inter, kv, norm):
    """Bit for bit what pkv_append stores of the fp16 keys that the same call leaves in an fp16 cache -- groups of 32 values that
    straddle the rotated part's halves and its end among them."""
    T, blocks = 37, 4
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(T, hq, d, generator=g, device="cuda").half()
    k = (torch.randn(T, hkv, d, generator=g, device="cuda") * torch.logspace(-4, 3, T, device="cuda")[:, None, None]).half()
    v = torch.randn(T, hkv, d, generator=g, device="cuda").half()
    k[5], v[6] = 0, 0
    pos = torch.arange(T, device="cuda", dtype=torch.int32) * 911
    slots = torch.randperm(blocks * 16, generator=g, device="cuda")[:T]
    slots[9] = -1
    rope = pkv.Rope(d, rot, interleaved=inter)
    w = torch.logspace(-1, 1, d, device="cuda").half()
    half = pkv.Pool(1, hq, hkv, d, blocks)
    a, b = (pkv.Pool(1, hq, hkv, d, blocks, kv_dtype=kv) for _ in range(2))
    for p in (a, b):
        p.buffer[:-256].fill_(0x5A)
    out, outq = torch.empty_like(q), torch.empty_like(q)

    def call(pool, dst):
        args = (q, hq * d, k, hkv * d, v, hkv * d, pos, slots, T, dst)
        if norm:
            pkv.pkv_norm_rope_append(pool.handle, 0, rope.handle, w, w, 1e-6, 0.0, *args)
        else:
            pkv.pkv_rope_append(pool.handle, 0, rope.handle, *args)
    call(half, out)
    call(a, outq)
    kr = half.layer(0, 0)[slots.clamp(min=0) // 16, :, slots.clamp(min=0) % 16].contiguous()
    pkv.pkv_append(b.handle, 0, kr, v, slots, T)
    assert a.check() == 0 and torch.equal(a.buffer, b.buffer) and torch.equal(_bytes(out), _bytes(outq))
    if kv == pkv.PKV_KV_INT4:  # and the oracle's
        want = np.full((blocks, hkv, 18 * d), 0x5A, np.uint8)
        int4.append_reference_4bit(want, kr.cpu().numpy(), v.cpu().numpy(), slots.cpu().numpy())
        assert np.array_equal(a.cache_view()[0].cpu().numpy(), want)


def test_in_place_keys_alone_and_no_tokens(cuda, built):
    T, hq, hkv, d = 50, 8, 2, 128
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k, v = (torch.randn(T, h, d, generator=g, device="cuda").half() for h in (hq, hkv, hkv))
    w = torch.rand(d, generator=g, device="cuda").half()
    pos, slots = torch.arange(T, device="cuda", dtype=torch.int32), torch.randperm(64, generator=g, device="cuda")[:T]
    rope = pkv.Rope(d)
    a, b = (pkv.Pool(1, hq, hkv, d, 4) for _ in range(2))
    a.buffer[:-256].zero_(), b.buffer[:-256].zero_()
    out = torch.empty_like(q)
    tail = (k, hkv * d, v, hkv * d, pos, slots, T)
    pkv.pkv_norm_rope_append(a.handle, 0, rope.handle, w, w, 1e-6, 0.0, q, hq * d, *tail, out)
    pkv.pkv_norm_rope_append(b.handle, 0, rope.handle, w, w, 1e-6, 0.0, None, 0, *tail, None)  # keys and values alone
    assert torch.equal(a.buffer, b.buffer)
    same = q.clone()
    pkv.pkv_norm_rope_append(b.handle, 0, rope.handle, w, w, 1e-6, 0.0, same, hq * d, *tail, same)
    assert torch.equal(a.buffer, b.buffer) and torch.equal(_bytes(same), _bytes(out))
    pkv.pkv_norm_rope_append(b.handle, 0, rope.handle, w, w, 1e-6, 0.0, None, 0, None, 0, None, 0, None, None, 0, None)
    assert pkv.pkv_last_launch_count(b.handle) == 0
    # a bad slot is skipped and reported, its query all the same
    bad = slots.clone()
    bad[7], bad[8] = 64, -2
    again = torch.full_like(q, float("nan"))
    b.buffer[:-256].zero_()
    pkv.pkv_norm_rope_append(b.handle, 0, rope.handle, w, w, 1e-6, 0.0, q, hq * d, k, hkv * d, v, hkv * d, pos, bad, T, again)
    assert b.check() == pkv.PKV_DEVERR_SLOT_RANGE and torch.equal(_bytes(again), _bytes(out))
    want = a.cache_view().clone()
    for t in (7, 8):
        want[0, :, slots[t] // 16, :, slots[t] % 16] = 0
    assert torch.equal(_bytes(b.cache_view()), _bytes(want))


def test_refusals(cuda, built):
    T, hq, hkv, d = 4, 4, 2, 64
    pool = pkv.Pool(2, hq, hkv, d, 4, kv_dtype=pkv.PKV_KV_INT4)
    rope, other = pkv.Rope(d), pkv.Rope(128)
    q, k, v = (torch.zeros(T, h, d, dtype=torch.float16, device="cuda") for h in (hq, hkv, hkv))
    w = torch.zeros(d + 8, dtype=torch.float16, device="cuda")
    pos, slots = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.arange(T, device="cuda")
    good = dict(layer=0, rope=rope.handle, qw=w, kw=w, eps=1e-6, off=0.0, q=q, qs=hq * d, k=k, ks=hkv * d, v=v, vs=hkv * d, pos=pos,
                slots=slots, T=T, out=torch.empty_like(q))
    bad = [(dict(layer=2), pkv.PKV_ERR_OUT_OF_RANGE), (dict(layer=-1), pkv.PKV_ERR_OUT_OF_RANGE)] + [
        (c, pkv.PKV_ERR_INVALID_ARG) for c in (
            dict(qw=None, kw=None), dict(qw=w[1:]), dict(kw=w.data_ptr() + 8), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
            dict(eps=float("inf")), dict(eps=1e-31), dict(off=float("inf")), dict(off=float("nan")), dict(rope=other.handle), dict(T=-1),
            dict(k=None), dict(v=None), dict(pos=None), dict(slots=None), dict(q=None), dict(out=None), dict(qs=hq * d - 8),
            dict(ks=hkv * d + 4), dict(vs=0), dict(q=q.data_ptr() + 2), dict(out=q, qs=hq * d + 8))]
    for change, status in bad:
        a = dict(good, **change)
        with pytest.raises(pkv.PkvError) as e:
            pkv.pkv_norm_rope_append(pool.handle, a["layer"], a["rope"], a["qw"], a["kw"], a["eps"], a["off"], a["q"], a["qs"], a["k"],
                                     a["ks"], a["v"], a["vs"], a["pos"], a["slots"], a["T"], a["out"])
        assert e.value.status == status and pkv.pkv_last_launch_count(pool.handle) == 0, change
    assert pool.check() == 0


@pytest.mark.parametrize("kv", KINDS)
def test_a_decode_step_of_a_model_with_norms(cuda, built, kv):
    """Positions, norms with rotation and append, plan and attention on a stream of their own and as a replayed graph: the
    outputs and the cache bit for bit, and attention over the keys that pkv_gather reads back."""
    import oracle
    hq, hkv, d, rows = 12, 2, 128, 9
    rng = np.random.default_rng(1)
    ctx = rng.integers(1, 200, rows).astype(np.int32)
    ctx[0] = 1
    width = -(-int(ctx.max()) // 16)
    tables = rng.permutation(rows * width).reshape(rows, width).astype(np.int32)
    pool = pkv.Pool(2, hq, hkv, d, rows * width, kv_dtype=kv)
    rope = pkv.Rope(d, 64)
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()  # noqa: E731
    dt, dc, ds = i32(tables), i32(ctx), i32(np.arange(rows + 1))
    packed = torch.from_numpy(rng.standard_normal((rows, hq + 2 * hkv, d)).astype(np.float16)).cuda()
    q, k, v = packed[:, :hq], packed[:, hq:hq + hkv], packed[:, hq + hkv:]
    w = torch.from_numpy((1 + 0.2 * rng.standard_normal(d)).astype(np.float16)).cuda()
    old = torch.from_numpy(rng.standard_normal((rows * width * 16, hkv, d)).astype(np.float16)).cuda()
    every = torch.arange(rows * width * 16, device="cuda")
    n = pkv.pkv_attention_workspace_bytes(pool.handle, rows, rows, width)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    pos, slots = torch.empty(rows, dtype=torch.int32, device="cuda"), torch.empty(rows, dtype=torch.int64, device="cuda")
    turned, out = (torch.empty(2, rows, hq, d, dtype=torch.float16, device="cuda") for _ in range(2))
    for layer in range(2):
        pkv.pkv_append(pool.handle, layer, old, old.flip(0).contiguous(), every, len(every))

    def step():
        pkv.pkv_positions(pool.handle, dc, ds, rows, rows, pos)
        pkv.pkv_slot_mapping(pool.handle, dt, width, dc, ds, rows, rows, slots)
        pkv.pkv_attention_plan(pool.handle, dc, ds, rows, rows, width, ws, n)
        for layer in range(2):
            pkv.pkv_norm_rope_append(pool.handle, layer, rope.handle, w, w, 1e-6, 0.0, q, q.stride(0), k, k.stride(0), v, v.stride(0),
                                     pos, slots, rows, turned[layer])
            pkv.pkv_attention(pool.handle, layer, turned[layer], dt, width, dc, ds, rows, rows, out[layer], ws, n)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            step()
    torch.cuda.synchronize()
    first, cache = out.clone(), pool.cache_view().clone()
    assert pool.check() == 0
    out.fill_(float("nan")), turned.fill_(float("nan"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for _ in range(4):
        graph.replay()
    torch.cuda.synchronize()
    assert pool.check() == 0 and torch.equal(_bytes(out), _bytes(first)) and torch.equal(_bytes(cache), _bytes(pool.cache_view()))
    ko, vo = torch.empty_like(old), torch.empty_like(old)
    pkv.pkv_gather(pool.handle, 1, every, len(every), ko, vo)
    ko, vo, tn, got = (x.cpu().numpy() for x in (ko, vo, turned[1], out[1]))
    for b in range(rows):
        s = tables[b][np.arange(ctx[b]) // 16].astype(np.int64) * 16 + np.arange(ctx[b]) % 16
        kk, vv = ko[s].astype(np.float64), vo[s].astype(np.float64)
        want = oracle.window_attention_row(tn[b:b + 1], kk, vv, 1 << 30, 0)[0]
        a = oracle.window_attention_row(tn[b:b + 1], kk, np.abs(vv), 1 << 30, 0)[0]
        # weights and output rounded to fp16, scores in fp32: derived in the 4-bit cache's tests
        assert (np.abs(got[b].astype(np.float64) - want) <= 2.0**-11 * 1.001 * (a + np.abs(want)) + 2.0**-13 * a + 2.0**-24).all()
