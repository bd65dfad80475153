"""GPU: passes whose query_start_loc is no list of rows, or holds rows without tokens, are reported and write nothing outside the
workspace and the packed output.  (Run on kernels that bound what they derive from it.)  Tolerance as in test_gpu_parity."""
import numpy as np
import pytest
import torch

import oracle
from oracle import fp8
from continuous_batching_paged_ragged_gb300 import pkv
from helpers_gpu import assert_close

pytestmark = pytest.mark.gpu

HQ, HKV, D, BLOCKS, WIDTH, CTX = 8, 2, 64, 12, 6, 90
GUARD = 1 << 20


class Pass:
    """Rows of CTX tokens on one table; what lies around the workspace and the output is watched."""

    def __init__(self, kv, qsl, tokens, window=0):
        g = torch.Generator(device="cuda").manual_seed(3)
        self.pool = pkv.Pool(1, HQ, HKV, D, BLOCKS, kv_dtype=kv)
        self.kv, self.window, self.tokens, self.rows = kv, window, tokens, len(qsl) - 1
        self.k, self.v = (torch.randn(CTX, HKV, D, generator=g, device="cuda").half() for _ in range(2))
        row = torch.tensor([5, 3, 9, 0, 7, 1], dtype=torch.int32, device="cuda")
        slots = row[torch.arange(CTX, device="cuda") // 16].long() * 16 + torch.arange(CTX, device="cuda") % 16
        pkv.pkv_append(self.pool.handle, 0, self.k, self.v, slots, CTX)
        self.tables = row.repeat(self.rows, 1).contiguous()
        self.ctx = torch.full((self.rows,), CTX, dtype=torch.int32, device="cuda")
        self.qsl = torch.tensor(qsl, dtype=torch.int32, device="cuda")
        self.q = torch.randn(tokens, HQ, D, generator=g, device="cuda").half()
        args = (self.pool.handle, self.rows, tokens, WIDTH)
        self.n = pkv.pkv_attention_window_workspace_bytes(*args, window, 2) if window else pkv.pkv_attention_workspace_bytes(*args)
        self.memory = torch.full((GUARD + self.n + GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
        self.out_memory = torch.full((3 * tokens, HQ, D), float("nan"), dtype=torch.float16, device="cuda")

    def run(self, fused=False):
        h, ws, out = self.pool.handle, self.memory[GUARD:], self.out_memory[self.tokens:2 * self.tokens]
        meta = (self.ctx, self.qsl, self.rows, self.tokens)
        if self.window:
            pkv.pkv_attention_window_plan(h, *meta, WIDTH, self.window, 2, ws, self.n)
        else:
            pkv.pkv_attention_plan(h, *meta, WIDTH, ws, self.n)
        rest = (self.tables, WIDTH, *meta, out, ws, self.n)
        if fused:
            kv = torch.zeros(self.tokens, HKV, D, dtype=torch.float16, device="cuda")
            slots = torch.full((self.tokens,), -1, dtype=torch.int64, device="cuda")  # nothing is appended
            pkv.pkv_attention_append(h, 0, self.q, kv, kv, slots, *rest)
        else:
            pkv.pkv_attention(h, 0, self.q, *rest)
        torch.cuda.synchronize()
        assert (self.memory[:GUARD] == 0xA5).all() and (self.memory[GUARD + self.n:] == 0xA5).all()
        around = torch.cat([self.out_memory[:self.tokens], self.out_memory[2 * self.tokens:]])
        assert torch.isnan(around).all()
        return out.cpu().numpy()


EMPTY = {  # rows without tokens beside rows of 16 and more
    "few": [0, 16, 32, 48, 64] + [64] * 60, "front": [0] * 40 + [20, 20, 50], "all but one": [0] * 33 + [33],
    "short": [0, 3, 3, 7, 7, 7, 8]}
BROKEN = {  # not a list of rows
    "back and forth": [0, 60] * 31 + [0, 64], "past the end": [0, 16, 4096, 64], "below zero": [-40, 24], "not from zero": [7, 40],
    "short of the end": [0, 20], "far": [0, 2**31 - 1, -2**31, 30]}


@pytest.mark.parametrize("kv", [pkv.PKV_KV_F16, pkv.PKV_KV_E4M3])
@pytest.mark.parametrize("window", [0, 33])
@pytest.mark.parametrize("case", EMPTY)
def test_rows_without_tokens(cuda, built, kv, window, case):
    """The other rows get their results."""
    qsl = EMPTY[case]
    p = Pass(kv, qsl, qsl[-1], window)
    out = p.run()
    assert p.pool.check() == pkv.PKV_DEVERR_ROW_META
    k, v = p.k.cpu().numpy(), p.v.cpu().numpy()
    if kv == pkv.PKV_KV_E4M3:
        k, v = (fp8.dequantize_rows(*fp8.quantize_rows(x)) for x in (k, v))
    q = p.q.cpu().numpy()
    for a, b in zip(qsl, qsl[1:]):
        if b > a:
            ref = oracle.window_attention_row(q[a:b], k, v, window, 2) if window else oracle.attention_row(q[a:b], k, v)
            assert_close(out[a:b], ref, f"tokens {a} to {b}")


@pytest.mark.parametrize("kv", [pkv.PKV_KV_F16, pkv.PKV_KV_E4M3])
@pytest.mark.parametrize("window", [0, 33])
@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("case", BROKEN)
def test_no_list_of_rows(cuda, built, kv, window, fused, case):
    """Reported, no output row is written, and the pool serves the next pass."""
    p = Pass(kv, BROKEN[case], 64 if case != "far" else 30, window)
    out = p.run(fused)
    assert p.pool.check() & pkv.PKV_DEVERR_QSL and np.isnan(out).all()
    good = Pass(kv, [0, 1, 41], 41, window)
    assert np.isfinite(good.run()).all() and good.pool.check() == 0


@pytest.mark.parametrize("window", [0, 33])
@pytest.mark.parametrize("ctx", [5000, 2**31 - 1, 3, -7])
def test_contexts_rewritten_after_the_plan(cuda, built, window, ctx):
    """8-bit cache, a row of 16 and more new tokens: the pass was planned with other contexts than the call finds (which pkv.h asks
    to plan again)."""
    p = Pass(pkv.PKV_KV_E4M3, [0, 40, 41], 41, window)
    planned, plan = p.ctx.clone(), pkv.pkv_attention_window_plan if window else pkv.pkv_attention_plan
    ws, out = p.memory[GUARD:], p.out_memory[41:82]
    plan(p.pool.handle, p.ctx, p.qsl, 2, 41, WIDTH, *((window, 2) if window else ()), ws, p.n)
    p.ctx.fill_(ctx)
    pkv.pkv_attention(p.pool.handle, 0, p.q, p.tables, WIDTH, p.ctx, p.qsl, 2, 41, out, ws, p.n)
    torch.cuda.synchronize()
    assert (p.memory[:GUARD] == 0xA5).all() and (p.memory[GUARD + p.n:] == 0xA5).all()
    assert torch.isnan(p.out_memory[:41]).all() and torch.isnan(p.out_memory[82:]).all()
    p.pool.check()
    p.ctx.copy_(planned)
    p.memory.fill_(0xA5)
    p.out_memory.fill_(float("nan"))
    assert np.isfinite(p.run()).all() and p.pool.check() == 0
