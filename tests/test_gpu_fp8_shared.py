"""GPU: rows of 16 or more new tokens that share blocks on an 8-bit cache (their fp16 shadow has room for the pool's blocks,
fewer than the rows' tables name).  Tolerances as in test_gpu_fp8: the oracle over the dequantized cache."""
import numpy as np
import pytest
import torch

import oracle
from oracle import fp8
from continuous_batching_paged_ragged_gb300 import pkv
from helpers_gpu import assert_close, poison

pytestmark = pytest.mark.gpu


def _dev(x, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype).cuda()


def _rows(seed, n, heads, d):
    return np.random.default_rng([seed, 77]).standard_normal((n, heads, d)).astype(np.float16)


class Cache:
    """An 8-bit pool and passes over it; a window of 0 is none."""

    def __init__(self, shape, blocks, window=0, sinks=0, layers=1):
        self.hq, self.hkv, self.d = shape
        self.window, self.sinks = window, sinks
        self.pool = pkv.Pool(layers, *shape, blocks, kv_dtype=pkv.PKV_KV_E4M3)
        poison(self.pool)

    def attend(self, q, k, v, slots, tables, ctx, qsl, layer=0, append=True):
        h, B, T, W = self.pool.handle, len(ctx), int(qsl[-1]), tables.shape[1]
        tables, ctx, qsl, slots = _dev(tables), _dev(ctx), _dev(qsl), _dev(slots, torch.int64)
        q, k, v = (torch.from_numpy(x).cuda() for x in (q, k, v))
        out = torch.full_like(q, float("nan"))
        if self.window:
            n = pkv.pkv_attention_window_workspace_bytes(h, B, T, W, self.window, self.sinks)
        else:
            n = pkv.pkv_attention_workspace_bytes(h, B, T, W)
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        if self.window:
            pkv.pkv_attention_window_plan(h, ctx, qsl, B, T, W, self.window, self.sinks, ws, n)
        else:
            pkv.pkv_attention_plan(h, ctx, qsl, B, T, W, ws, n)
        if append:
            pkv.pkv_attention_append(h, layer, q, k, v, slots, tables, W, ctx, qsl, B, T, out, ws, n)
        else:
            pkv.pkv_attention(h, layer, q, tables, W, ctx, qsl, B, T, out, ws, n)
        torch.cuda.synchronize()
        assert self.pool.check() == 0
        return out.cpu().numpy()

    def check(self, got, q, k, v, what):
        k, v = (fp8.dequantize_rows(*fp8.quantize_rows(x)) for x in (k, v))
        ref = oracle.window_attention_row(q, k, v, self.window, self.sinks) if self.window else oracle.attention_row(q, k, v)
        assert_close(got, ref, what)


@pytest.mark.parametrize("shape", [(4, 2, 64), (12, 2, 128), (8, 2, 256)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 5)])
@pytest.mark.parametrize("children", [1, 4])
def test_forks_of_a_prompt_in_the_middle(cuda, built, shape, window, sinks, children):
    """A prompt of 300 tokens is forked after 200: the next passes hold a chunk of it in every child, on a pool that holds the
    shared blocks once and has none to spare."""
    rows = 1 + children
    blocks = 12 + rows * (20 - 12)  # 12 full blocks shared, of 20 a row
    c = Cache(shape, blocks, window, sinks)
    sched = pkv.Scheduler(rows, 200, 16, blocks)
    sched.add(0, 300, 4)
    values = {0: [_rows(s, 304, n, shape[2]) for s, n in ((0, shape[0]), (1, shape[1]), (2, shape[1]))]}
    for i in range(5 + children):
        st = sched.step()
        ids, qsl, ctx = st["req_ids"].tolist(), st["query_start_loc"], st["context_lens"]
        if not ids:
            break
        new = [np.concatenate([values[r][j][ctx[b] - st["q_lens"][b]:ctx[b]] for b, r in enumerate(ids)]) for j in range(3)]
        out = c.attend(*new, st["slot_mapping"], st["block_tables"], ctx, qsl)
        for b, r in enumerate(ids):
            q, k, v = values[r]
            c.check(out[qsl[b]:qsl[b + 1]], q[ctx[b] - st["q_lens"][b]:ctx[b]], k[:ctx[b]], v[:ctx[b]], f"pass {i} request {r}")
        if i == 0:
            assert int(ctx[0]) == 200
            for child in range(1, rows):
                block = sched.fork(0, child, 4)
                two = np.array([[*sched.tables()[1][0]], [-1] * sched.tables()[1].shape[1]], dtype=np.int32)
                pkv.pkv_fork_rows(c.pool.handle, _dev(two), two.shape[1], _dev([200, 0]), 2, _dev([[0, 1, block]]), 1)
                # its own continuation of the prompt
                values[child] = [np.concatenate([x[:200], _rows(10 * child + j, 104, x.shape[1], x.shape[2])]) for j, x in enumerate(values[0])]
    assert i > 2


@pytest.mark.parametrize("shape", [(4, 2, 64), (12, 2, 128), (8, 2, 256)])
def test_rows_of_one_table_with_different_contexts(cuda, built, shape):
    """Cached tokens attended by chunks that end at different places of the same blocks, what is behind the longest NaN; decode rows
    beside them, two layers, and the allocation-free call."""
    c = Cache(shape, 8, layers=2)
    k, v = _rows(1, 120, *shape[1:]), _rows(2, 120, *shape[1:])
    order = [5, 0, 7, 2, 6, 1, 4, 3]
    slots = np.array([order[t // 16] * 16 + t % 16 for t in range(120)], dtype=np.int64)
    for layer in (0, 1):
        pkv.pkv_append(c.pool.handle, layer, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), _dev(slots, torch.int64), 120)
    ctx, q_lens = [120, 119, 100, 97, 33, 120, 18, 64], [16, 40, 100, 17, 20, 1, 3, 64]
    qsl = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    tables = np.array([order] * len(ctx), dtype=np.int32)
    q = _rows(3, int(qsl[-1]), shape[0], shape[2])
    for layer in (0, 1):
        out = c.attend(q, k[:1], v[:1], slots[:1], tables, ctx, qsl, layer, append=False)
        for b in range(len(ctx)):
            c.check(out[qsl[b]:qsl[b + 1]], q[qsl[b]:qsl[b + 1]], k[:ctx[b]], v[:ctx[b]], f"layer {layer} row {b}")
        free = torch.full((int(qsl[-1]), shape[0], shape[2]), float("nan"), dtype=torch.float16, device="cuda")
        pkv.pkv_attention_noalloc(c.pool.handle, layer, torch.from_numpy(q).cuda(), _dev(tables), 8, _dev(ctx), _dev(qsl), len(ctx),
                                  int(qsl[-1]), free)
        assert np.array_equal(free.cpu().numpy().view(np.int16), out.view(np.int16))
