"""GPU: block calls, plans and attention enqueued one behind the other without a host synchronisation, eagerly on a stream of
their own and captured once and replayed over new contents.  Copies, forks and compaction move bytes, and a row's
result does not depend on where its blocks lie or on the rows beside it, so every output is the first one's bits."""
import numpy as np
import pytest
import torch

from continuous_batching_paged_ragged_gb300 import pkv
from helpers_gpu import poison

pytestmark = pytest.mark.gpu

LAYERS, HQ, HKV, D, ROWS = 3, 12, 2, 128, 24
F16, E4M3 = pkv.PKV_KV_F16, pkv.PKV_KV_E4M3


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


class Chain:
    """Rows of one query each over cached contexts; their blocks copied, the copies forked, everything compacted."""

    def __init__(self, kv, window, seed=0):
        rng = np.random.default_rng(seed)
        self.kv, self.window = kv, window
        ctx = rng.integers(1, 1500, ROWS)
        ctx[:4] = 1, 16, 17, 1488
        held = -(-ctx // 16)
        self.used, self.width = int(held.sum()), int(held.max()) + 1
        self.blocks = 3 * self.used + 2 * ROWS
        ids = rng.permutation(self.blocks)
        src, dst, self.spare = ids[:self.used], ids[self.used:2 * self.used], ids[2 * self.used:]
        tables, copies, at = np.full((ROWS, self.width), -1), np.full((2 * ROWS, self.width), -1), 0
        for b, n in enumerate(held):
            tables[b, :n], copies[b, :n] = src[at:at + n], dst[at:at + n]
            at += n
        self.pool = pkv.Pool(LAYERS, HQ, HKV, D, self.blocks, kv_dtype=kv)
        self.src, self.pairs = torch.from_numpy(src).cuda(), _dev(np.stack([src, dst], 1))
        self.tables, self.copies0 = _dev(tables), _dev(copies)
        self.ctx, self.ctx0 = _dev(ctx), _dev(np.concatenate([ctx, np.zeros(ROWS)]))
        self.forks = _dev([(b, ROWS + b, self.spare[b]) for b in range(ROWS)])
        self.qsl, self.qsl2 = _dev(np.arange(ROWS + 1)), _dev(np.arange(2 * ROWS + 1))
        self.copies, self.ctx2, self.compacted = self.copies0.clone(), self.ctx0.clone(), torch.empty_like(self.copies0)
        self.remap, self.live = torch.empty(self.blocks, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
        self.q = torch.empty(2 * ROWS, HQ, D, dtype=torch.float16, device="cuda")
        self.outs = [torch.empty(n, HQ, D, dtype=torch.float16, device="cuda") for n in (ROWS, ROWS, 2 * ROWS, 2 * ROWS)]
        self.ws = [self._workspace(n) for n in (ROWS, 2 * ROWS)]
        self.cws = torch.empty(pkv.pkv_compact_workspace_bytes(self.pool.handle), dtype=torch.uint8, device="cuda")

    def _workspace(self, rows):
        h = self.pool.handle
        n = (pkv.pkv_attention_window_workspace_bytes(h, rows, rows, self.width, self.window, 4) if self.window else
             pkv.pkv_attention_workspace_bytes(h, rows, rows, self.width))
        return torch.empty(n, dtype=torch.uint8, device="cuda")

    def _plan(self, ctx, qsl, rows, ws):
        head = (self.pool.handle, ctx, qsl, rows, rows, self.width)
        if self.window:
            pkv.pkv_attention_window_plan(*head, self.window, 4, ws, ws.numel())
        else:
            pkv.pkv_attention_plan(*head, ws, ws.numel())

    def _attend(self, layer, tables, ctx, qsl, rows, out, ws):
        pkv.pkv_attention(self.pool.handle, layer, self.q, tables, self.width, ctx, qsl, rows, rows, out, ws, ws.numel())

    def fill(self, seed):
        """New contents in the rows' own blocks, NaN in every other."""
        g = torch.Generator(device="cuda").manual_seed(seed)
        poison(self.pool)
        cache = self.pool.cache_view()
        shape = (LAYERS, 2, self.used, *cache.shape[3:])
        if self.kv == E4M3:
            cache[:, :, self.src] = torch.randint(0, 100, shape, generator=g, dtype=torch.uint8, device="cuda")
            scales = self.pool.scales_view()
            scales[:, self.src] = torch.randint(118, 124, (LAYERS, self.used, *scales.shape[2:]), generator=g, dtype=torch.uint8, device="cuda")
        else:
            cache[:, :, self.src] = torch.randn(shape, generator=g, device="cuda").to(cache.dtype)
        q = torch.randn(ROWS, HQ, D, generator=g, device="cuda").half()
        self.q.copy_(torch.cat([q, q]))  # a child asks what its parent asks
        for o in self.outs:
            o.fill_(float("nan"))

    def run(self):
        h, last = self.pool.handle, LAYERS - 1
        self.copies.copy_(self.copies0)
        self.ctx2.copy_(self.ctx0)
        self._plan(self.ctx, self.qsl, ROWS, self.ws[0])
        self._attend(last, self.tables, self.ctx, self.qsl, ROWS, self.outs[0], self.ws[0])
        pkv.pkv_copy_blocks(h, self.pairs, self.used)
        self._attend(last, self.copies, self.ctx, self.qsl, ROWS, self.outs[1], self.ws[0])  # on the plan of before
        pkv.pkv_fork_rows(h, self.copies, self.width, self.ctx2, 2 * ROWS, self.forks, ROWS)
        self._plan(self.ctx2, self.qsl2, 2 * ROWS, self.ws[1])
        self._attend(last, self.copies, self.ctx2, self.qsl2, 2 * ROWS, self.outs[2], self.ws[1])
        pkv.pkv_compact(h, self.copies, self.width, 2 * ROWS, self.compacted, self.remap, self.live, self.cws, self.cws.numel())
        self._attend(last, self.compacted, self.ctx2, self.qsl2, 2 * ROWS, self.outs[3], self.ws[1])

    def check(self):
        torch.cuda.synchronize()
        assert self.pool.check() == 0
        first = self.outs[0].view(torch.int16)
        assert torch.isfinite(self.outs[0]).all()
        assert torch.equal(self.outs[1].view(torch.int16), first)
        for o in self.outs[2:]:
            assert torch.equal(o.view(torch.int16), torch.cat([first, first]))
        partial = int((self.ctx % 16 > 0).sum())
        assert int(self.live) == self.used + partial and int(self.compacted.max()) == int(self.live) - 1


@pytest.mark.parametrize("kv", [F16, E4M3])
@pytest.mark.parametrize("window", [None, 200])
def test_chain_on_a_stream_and_replayed(cuda, built, kv, window):
    c = Chain(kv, window)
    side = torch.cuda.Stream()
    for seed in range(4):
        c.fill(seed)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            c.run()
        c.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    for seed in range(4, 16):
        c.fill(seed)
        graph.replay()
        c.check()
