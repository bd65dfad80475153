"""GPU: attention calls right behind appends, on one stream and with nothing in between, give the bits of the same calls with a
synchronization after each: appends of tokens in front of the pass's own, and passes planned ahead of one another."""
import numpy as np
import pytest
import torch

import oracle
from oracle import fp8
from continuous_batching_paged_ragged_gb300 import pkv
from helpers_gpu import assert_close

pytestmark = pytest.mark.gpu

F16, E4M3 = pkv.PKV_KV_F16, pkv.PKV_KV_E4M3


class Pass:
    """One new token in each row of ctx tokens; the rows' blocks lie scattered in the pool."""

    def __init__(self, pool, tables, ctx, window=0):
        self.pool, self.n, self.ctx_host = pool, len(ctx), list(ctx)
        self.tables, self.width = torch.from_numpy(tables).cuda(), tables.shape[1]
        self.ctx = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        self.qsl = torch.arange(self.n + 1, dtype=torch.int32, device="cuda")
        self.slots = torch.tensor([int(tables[b, (c - 1) // 16]) * 16 + (c - 1) % 16 for b, c in enumerate(ctx)], device="cuda")
        self.window = window
        args = (pool.handle, self.n, self.n, self.width)
        self.ws_bytes = pkv.pkv_attention_window_workspace_bytes(*args, window, 4) if window else pkv.pkv_attention_workspace_bytes(*args)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device="cuda")
        c = pool.cfg
        self.out = torch.empty(self.n, c.num_q_heads, c.head_dim, dtype=torch.float16, device="cuda")

    def plan(self):
        if self.window:
            pkv.pkv_attention_window_plan(self.pool.handle, self.ctx, self.qsl, self.n, self.n, self.width, self.window, 4, self.ws, self.ws_bytes)
        else:
            pkv.pkv_attention_plan(self.pool.handle, self.ctx, self.qsl, self.n, self.n, self.width, self.ws, self.ws_bytes)

    def attend(self, q, k=None, v=None):
        rest = (self.tables, self.width, self.ctx, self.qsl, self.n, self.n, self.out, self.ws, self.ws_bytes)
        if k is None:
            pkv.pkv_attention(self.pool.handle, 0, q, *rest)
        else:
            pkv.pkv_attention_append(self.pool.handle, 0, q, k, v, self.slots, *rest)


def _setup(kv, shape, ctx, seed=0):
    rng = np.random.default_rng(seed)
    width = -(-(max(ctx) + 1) // 16)
    blocks = len(ctx) * width
    tables = rng.permutation(blocks).astype(np.int32).reshape(len(ctx), width)
    pool = pkv.Pool(1, *shape, blocks, kv_dtype=kv)
    pool.buffer.zero_()
    return pool, tables


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(torch.float16)


@pytest.mark.parametrize("kv", [F16, E4M3])
@pytest.mark.parametrize("shape", [(8, 2, 64), (12, 2, 128), (8, 2, 256)])
@pytest.mark.parametrize("rotary", [False, True])
@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("window", [0, 300])
def test_append_of_earlier_tokens(cuda, built, kv, shape, rotary, fused, window):
    """After the plan: the rows' whole contexts appended at once (other values every time), then the attention."""
    g = torch.Generator(device="cuda").manual_seed(1)
    ctx = [1500, 33, 700, 16, 1, 257, 1024, 90] * 3
    pool, tables = _setup(kv, shape, ctx)
    p = Pass(pool, tables, ctx, window)
    hq, hkv, d = shape
    at = [(b, t) for b, c in enumerate(ctx) for t in range(c)]
    slots = torch.tensor([int(tables[b, t // 16]) * 16 + t % 16 for b, t in at], device="cuda")
    last = torch.tensor(np.cumsum(ctx) - 1, device="cuda")
    zeros = torch.zeros(len(at), dtype=torch.int32, device="cuda")  # angle 0: rotation leaves the keys as they are
    rope = pkv.Rope(d)
    p.plan()
    for turn in range(6):
        k, v, q = _normal(g, len(at), hkv, d), _normal(g, len(at), hkv, d), _normal(g, p.n, hq, d)
        kn, vn = (k[last].contiguous(), v[last].contiguous()) if fused else (None, None)

        def append():
            if rotary:
                pkv.pkv_rope_append(pool.handle, 0, rope.handle, None, 0, k, hkv * d, v, hkv * d, zeros, slots, len(at), None)
            else:
                pkv.pkv_append(pool.handle, 0, k, v, slots, len(at))

        torch.cuda.synchronize()
        append()
        p.attend(q, kn, vn)
        got = p.out.clone()
        torch.cuda.synchronize()
        append()
        torch.cuda.synchronize()
        p.attend(q, kn, vn)
        torch.cuda.synchronize()
        assert torch.equal(got.view(torch.int16), p.out.view(torch.int16)), turn
        assert pool.check() == 0
    rows = np.concatenate([[0], np.cumsum(ctx)])
    for b, c in enumerate(ctx):
        kb, vb = (x[rows[b]:rows[b + 1]].cpu().numpy() for x in (k, v))
        if kv == E4M3:
            kb, vb = (fp8.dequantize_rows(*fp8.quantize_rows(x)) for x in (kb, vb))
        qb = q[b:b + 1].cpu().numpy()
        ref = oracle.window_attention_row(qb, kb, vb, window, 4) if window else oracle.attention_row(qb, kb, vb)
        assert_close(got[b:b + 1].cpu().numpy(), ref, f"row {b}")


@pytest.mark.parametrize("kv", [F16, E4M3])
@pytest.mark.parametrize("shape", [(8, 2, 64), (12, 2, 128), (8, 2, 256)])
@pytest.mark.parametrize("second_fused", [False, True])
def test_passes_planned_ahead(cuda, built, kv, shape, second_fused):
    """Two passes of one layer planned on two workspaces, then run one behind the other: the second attends the token that the first
    has just appended."""
    g = torch.Generator(device="cuda").manual_seed(2)
    ctx = [1 + (37 * b) % 900 for b in range(96)]
    pool, tables = _setup(kv, shape, ctx, seed=1)
    pool.cache_view().copy_(torch.randint(0, 60, pool.cache_view().shape, generator=g, device="cuda") if kv == E4M3
                            else _normal(g, *pool.cache_view().shape))
    if kv == E4M3:
        pool.scales_view().fill_(121)
    one, two = Pass(pool, tables, ctx), Pass(pool, tables, [c + 1 for c in ctx])
    hq, hkv, d = shape
    one.plan()
    two.plan()
    for turn in range(10):
        q1, q2 = _normal(g, 96, hq, d), _normal(g, 96, hq, d)
        k1, v1, k2, v2 = (_normal(g, 96, hkv, d) for _ in range(4))
        outs = []
        for sync in (False, True):
            pkv.pkv_append(pool.handle, 0, torch.zeros_like(k1), torch.zeros_like(v1), one.slots, 96)  # the first's token away
            if not second_fused:
                pkv.pkv_append(pool.handle, 0, k2, v2, two.slots, 96)
            torch.cuda.synchronize()
            one.attend(q1, k1, v1)
            if sync:
                torch.cuda.synchronize()
            two.attend(q2, *((k2, v2) if second_fused else ()))
            torch.cuda.synchronize()
            outs.append((one.out.clone(), two.out.clone()))
        assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(*outs)), turn
    assert pool.check() == 0
