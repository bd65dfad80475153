"""GPU: attention through a windowed plan against the float64 oracle.

Every pass runs with the blocks that no new token sees given back: their table entries are -1 and their memory
holds NaN, as do the hidden keys that share a block with visible ones (decode rows).  Outputs |o| <= max|v| =
2 sqrt(3): half an fp16 step of o and of every softmax weight is at most 2 * 3.47 * 2^-11 = 3.4e-3 together, within MAX_ABS."""
import numpy as np
import pytest
import torch

import oracle
from oracle import fp8
from continuous_batching_paged_ragged_gb300 import pkv, synth, workload
from helpers_gpu import assert_close, host_rows, poison

pytestmark = pytest.mark.gpu

F16, E4M3 = pkv.PKV_KV_F16, pkv.PKV_KV_E4M3


def _hidden(ctx, q_len, window, sinks):
    """Positions that none of the row's new tokens sees, and the blocks that hold no other."""
    low = max(0, ctx - q_len + 1 - window)
    pos = [k for k in range(min(sinks, low), low)]
    blocks = [j for j in range(-(-ctx // 16)) if j * 16 >= sinks and j * 16 + 16 <= low]
    return pos, blocks


class Pass:
    """One pass through a windowed plan on a pool whose hidden memory is NaN."""

    def __init__(self, batch, window, sinks, kv_dtype=F16, split_blocks=0, rows=None):
        self.batch, self.window, self.sinks, self.kv = batch, window, sinks, kv_dtype
        self.rows = rows or host_rows(batch, 0)
        self.pool = workload.make_pool(batch, 1, split_blocks, kv_dtype=kv_dtype)
        poison(self.pool)
        cached = batch.cached_lens
        have = np.nonzero(cached > 0)[0]
        if have.size:
            bt = torch.from_numpy(np.ascontiguousarray(batch.block_tables[have])).cuda()
            ctx = torch.from_numpy(cached[have].astype(np.int32)).cuda()
            starts = np.concatenate([[0], np.cumsum(cached[have])]).astype(np.int32)
            total = int(starts[-1])
            slots = torch.empty(total, dtype=torch.int64, device="cuda")
            pkv.pkv_slot_mapping(self.pool.handle, bt, bt.shape[1], ctx, torch.from_numpy(starts).cuda(), int(have.size), total, slots)
            k, v = (torch.from_numpy(np.concatenate([self.rows[b][i][:cached[b]] for b in have])).cuda() for i in (1, 2))
            pkv.pkv_append(self.pool.handle, 0, k, v, slots, total)
        self.ds = workload.upload(batch, self.pool)
        nan = 0x7F if kv_dtype == E4M3 else float("nan")
        for b in range(batch.num_seqs):
            ctx, ql = int(batch.context_lens[b]), int(batch.q_lens[b])
            pos, blocks = _hidden(ctx, ql, window, sinks)
            if ql < 16:  # a chunk's own tile may hold its hidden values: they have to be finite (pkv.h)
                for p in pos:
                    if p < ctx - ql:
                        self.pool.cache_view()[0, :, int(batch.block_tables[b, p // 16]), :, p % 16] = nan
            for j in blocks:
                self.pool.cache_view()[0, :, int(batch.block_tables[b, j])] = nan
                if kv_dtype == E4M3:
                    self.pool.scales_view()[0, int(batch.block_tables[b, j])] = 255
                self.ds.block_tables[b, j] = -1
        cat = lambda i: torch.from_numpy(np.concatenate([r[i][0 if i == 0 else cached[b]:] for b, r in enumerate(self.rows)])).cuda()  # noqa: E731
        self.q, self.k, self.v = cat(0), cat(1), cat(2)
        d = self.ds
        self.ws_bytes = pkv.pkv_attention_window_workspace_bytes(self.pool.handle, d.num_seqs, d.num_tokens, d.max_blocks, window, sinks)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device="cuda")

    def plan(self):
        d = self.ds
        pkv.pkv_attention_window_plan(self.pool.handle, d.context_lens, d.query_start_loc, d.num_seqs, d.num_tokens, d.max_blocks,
                                      self.window, self.sinks, self.ws, self.ws_bytes)

    def run(self, fused=False):
        d = self.ds
        out = torch.full_like(self.q, float("nan"))
        rest = (d.block_tables, d.max_blocks, d.context_lens, d.query_start_loc, d.num_seqs, d.num_tokens, out, self.ws, self.ws_bytes)
        if fused:
            pkv.pkv_attention_append(self.pool.handle, 0, self.q, self.k, self.v, d.slot_mapping, *rest)
        else:
            pkv.pkv_append(self.pool.handle, 0, self.k, self.v, d.slot_mapping, d.num_tokens)
            pkv.pkv_attention(self.pool.handle, 0, self.q, *rest)
        return out

    def check(self, out, sample=None):
        torch.cuda.synchronize()
        assert self.pool.check() == 0
        got, starts = out.cpu().numpy(), self.batch.query_start_loc
        for b in range(self.batch.num_seqs):
            q, k, v = self.rows[b]
            if self.kv == E4M3:
                k, v = (fp8.dequantize_rows(*fp8.quantize_rows(x)) for x in (k, v))
            mine = got[starts[b]:starts[b + 1]]
            ql, ctx = q.shape[0], k.shape[0]
            at = range(ql) if sample is None or ql <= sample else sorted({0, 1, ql - 1, *np.linspace(0, ql - 1, sample).astype(int)})
            for i in ([None] if len(at) == ql else at):
                s = slice(0, ql) if i is None else slice(i, i + 1)
                end = ctx if i is None else ctx - ql + i + 1
                ref = oracle.window_attention_row(q[s], k[:end], v[:end], self.window, self.sinks)
                assert_close(mine[s], ref, f"row {b} query {i}")


def _run(shape, cached, q_lens, window, sinks, kv=F16, split_blocks=0, fused=False, sample=None, seed=5):
    batch = synth.custom_batch(synth.Shape(1, *shape), cached, q_lens, seed=seed)
    p = Pass(batch, window, sinks, kv, split_blocks)
    p.plan()
    out = p.run(fused)
    p.check(out, sample)
    return p, out


SHAPES = [(4, 4, 64), (4, 2, 128), (8, 2, 64), (12, 2, 128), (16, 2, 256)]
WINDOWS = [(1, 0), (2, 1), (15, 16), (16, 0), (17, 4), (100, 17), (300, 4), (5000, 3)]


@pytest.mark.parametrize("kv", [F16, E4M3])
@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_decode_rows(cuda, built, kv, fused, window, sinks):
    cached = [0, 1, 14, 15, 16, 17, 31, 100, 115, 116, 117, 300, 301, 515, 999, 2500]
    _run((12, 2, 128), cached, [1] * len(cached), window, sinks, kv, fused=fused)


@pytest.mark.parametrize("kv", [F16, E4M3])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("split_blocks", [0, 2])
def test_decode_head_layouts_and_short_chunks(cuda, built, kv, shape, split_blocks):
    for window, sinks in ((40, 5), (333, 0)):
        _run(shape, [0, 700, 33, 90, 1200, 0], [1, 3, 15, 7, 1, 9], window, sinks, kv, split_blocks, fused=split_blocks == 2)


@pytest.mark.parametrize("kv", [F16, E4M3])
def test_many_splits(cuda, built, kv):
    """Splits of one block: a window of 900 keys is more than 32 of them (the merge of its own launch), 200 fewer."""
    for window in (900, 200):
        _run((8, 2, 128), [3000, 80, 1024, 150], [1, 1, 2, 1], window, 4, kv, split_blocks=1)


@pytest.mark.parametrize("kv", [F16, E4M3])
@pytest.mark.parametrize("shape", [(4, 4, 64), (4, 2, 128), (8, 2, 128), (12, 2, 128), (16, 2, 64), (6, 1, 256), (2, 2, 256)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (50, 4), (128, 0), (129, 130), (700, 1), (9000, 0)])
def test_chunks(cuda, built, kv, shape, window, sinks):
    """Chunks on their own and on cached tokens, with decode rows among them."""
    _run(shape, [0, 500, 37, 1000, 2000, 5], [300, 40, 16, 1, 131, 2], window, sinks, kv, fused=True, sample=24)


@pytest.mark.parametrize("kv", [F16, E4M3])
@pytest.mark.parametrize("shape", [(12, 2, 128), (4, 1, 256)])
def test_long_windows_split_items(cuda, built, kv, shape):
    """A short chunk far into its row, its window long enough that its work runs in two parts."""
    _run(shape, [9000], [40], 6000, 100, kv, sample=10)
    _run(shape, [7000], [16], 4500, 0, kv, sample=16)


@pytest.mark.parametrize("kv", [F16, E4M3])
@pytest.mark.parametrize("shape", [(12, 2, 128), (8, 2, 256), (4, 4, 64)])
@pytest.mark.parametrize("window", [100000, 1024])
def test_rows_that_the_window_holds_whole_give_the_unwindowed_bits(cuda, built, kv, shape, window):
    batch = synth.custom_batch(synth.Shape(1, *shape), [0, 3000, 40, 900, 600, 1023, 700], [1, 1, 5, 1, 50, 1, 300], seed=3)
    p = Pass(batch, 100000, 7, kv)  # every block stays
    p.window = window
    p.plan()
    out = p.run()
    attn = workload.Attention(p.pool, p.ds)
    attn.plan()
    full = torch.empty_like(out)
    attn.run(0, p.q, full)
    torch.cuda.synchronize()
    for b in range(batch.num_seqs):
        if batch.context_lens[b] <= window and (shape[2] != 64 or batch.q_lens[b] >= 16):
            rows = slice(int(batch.query_start_loc[b]), int(batch.query_start_loc[b + 1]))
            assert torch.equal(out[rows].view(torch.int16), full[rows].view(torch.int16)), b
    p.check(out, sample=8)


def test_non_finite_new_tokens_reach_only_those_that_see_them(cuda, built):
    """Short chunks (decode path), fused and not: NaN and infinite keys and values of new tokens."""
    batch = synth.custom_batch(synth.Shape(1, 12, 2, 128), [100, 3, 60], [12, 10, 15], seed=4)
    for fused in (False, True):
        rows = host_rows(batch, 0)
        bad = {0: 105, 1: 6, 2: 70}  # row -> the position of its bad token
        for b, pos in bad.items():
            rows[b][1][pos], rows[b][2][pos] = (np.nan, np.inf)[b % 2], (np.inf, np.nan, -np.inf)[b]
        p = Pass(batch, 3, 2, rows=rows)
        p.plan()
        got = p.run(fused).cpu().numpy()
        assert p.pool.check() == 0
        for b, (q, k, v) in enumerate(rows):
            ql, ctx = q.shape[0], k.shape[0]
            for i in range(ql):
                at = ctx - ql + i
                if bad[b] <= at < bad[b] + 3:
                    continue  # sees it
                ref = oracle.window_attention_row(q[i:i + 1], k[:at + 1], v[:at + 1], 3, 2)
                assert_close(got[int(batch.query_start_loc[b]) + i][None], ref, f"row {b} query {i}")


@pytest.mark.parametrize("seed", range(12))
def test_random_passes(cuda, built, seed):
    rng = np.random.default_rng(seed)
    hkv, group, d = int(rng.choice([1, 2, 4])), int(rng.choice([1, 2, 4, 6, 8])), int(rng.choice([64, 128, 256]))
    n = int(rng.integers(1, 12))
    cached = [int(rng.choice([0, rng.integers(0, 40), rng.integers(0, 1500)])) for _ in range(n)]
    q_lens = [int(rng.choice([1, 1, 1, rng.integers(1, 16), rng.integers(16, 150)])) for _ in range(n)]
    window, sinks = int(2 ** rng.uniform(0, 10)), int(rng.choice([0, 1, 4, 15, 16, 33, 200]))
    _run((hkv * group, hkv, d), cached, q_lens, window, sinks, int(rng.choice([F16, E4M3])), int(rng.choice([0, 0, 1, 5, 13])),
         fused=bool(rng.integers(2)), sample=16, seed=seed)


@pytest.mark.parametrize("kv", [F16, E4M3])
def test_peaked_scores(cuda, built, kv):
    """Queries scaled by 8, a dominant key hidden just outside the window, one at its first position and one among the sinks."""
    batch = synth.custom_batch(synth.Shape(1, 12, 2, 128), [900, 900, 900, 640], [1, 1, 1, 100], seed=8)
    rows = host_rows(batch, 0)
    for b, (q, k, v) in enumerate(rows):
        q *= np.float16(8)
        if b < 3:
            p = k.shape[0] - 1
            at = (p - 256, p - 255, 1)[b]  # just outside, first inside, a sink
            k[at] = np.clip(q[0].reshape(2, 6, 128).mean(1) / 2, -30, 30)
    p = Pass(batch, 256, 4, kv, rows=rows)
    p.plan()
    p.check(p.run(), sample=12)


def test_batch_and_order_do_not_matter(cuda, built):
    cached, q_lens = [700, 3, 90, 2000, 1500, 64], [1, 1, 4, 1, 200, 1]
    whole, out = _run((12, 2, 128), cached, q_lens, 300, 4, sample=4)
    starts = whole.batch.query_start_loc
    for b in range(6):
        batch = synth.custom_batch(synth.Shape(1, 12, 2, 128), [cached[b]], [q_lens[b]], seed=5, req_ids=[int(whole.batch.req_ids[b])])
        p = Pass(batch, 300, 4)
        p.plan()
        alone = p.run()
        torch.cuda.synchronize()
        assert torch.equal(alone.view(torch.int16), out[int(starts[b]):int(starts[b + 1])].view(torch.int16)), b


def test_two_plans_one_graph(cuda, built):
    """A windowed and a full layer on two workspaces, captured and replayed with the plans, beside eager calls."""
    batch = synth.custom_batch(synth.Shape(1, 12, 2, 128), [700, 3, 90, 2000], [1, 1, 4, 60], seed=6)
    p = Pass(batch, 5000, 0)
    p.window, p.sinks = 200, 4  # the pool keeps every block, the plan sees few
    full = workload.Attention(p.pool, p.ds)
    outs = [torch.empty_like(p.q) for _ in range(2)]
    d = p.ds

    def step():
        p.plan()
        full.plan()
        pkv.pkv_attention_append(p.pool.handle, 0, p.q, p.k, p.v, d.slot_mapping, d.block_tables, d.max_blocks, d.context_lens,
                                 d.query_start_loc, d.num_seqs, d.num_tokens, outs[0], p.ws, p.ws_bytes)
        full.run(0, p.q, outs[1])

    step()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    p.check(outs[0], sample=8)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for o in outs:
            o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(outs, want))
    assert p.pool.check() == 0


def test_refusals_and_validation(cuda, built, monkeypatch):
    batch = synth.custom_batch(synth.Shape(1, 4, 2, 64), [400, 30], [1, 2], seed=6)
    p = Pass(batch, 100, 4)
    h, d = p.pool.handle, p.ds
    size = lambda *a: pkv.pkv_attention_window_workspace_bytes(h, *a)  # noqa: E731
    assert size(2, 3, 26, 0, 0) == 0 and size(2, 3, 26, 1, -1) == 0 and size(2, 3, 0, 1, 0) == 0
    assert size(2, 3, 26, 100, 4) <= pkv.pkv_attention_workspace_bytes(h, 2, 3, 26)
    for window, sinks, ws_bytes in [(0, 4, p.ws_bytes), (-5, 4, p.ws_bytes), (100, -1, p.ws_bytes), (100, 4, p.ws_bytes - 1)]:
        with pytest.raises(pkv.PkvError) as e:
            pkv.pkv_attention_window_plan(h, d.context_lens, d.query_start_loc, 2, 3, d.max_blocks, window, sinks, p.ws, ws_bytes)
        assert e.value.status == pkv.PKV_ERR_INVALID_ARG
    with pytest.raises(pkv.PkvError):
        p.run()  # no plan on this workspace
    monkeypatch.setenv("PKV_VALIDATE", "1")
    p.plan()
    p.check(p.run(fused=True))  # the blocks given back pass the validation
    pkv.pkv_slot_mapping(h, d.block_tables, d.max_blocks, d.context_lens, d.query_start_loc, 2, 3, d.slot_mapping)
    bad = d.block_tables.clone()
    bad[0, 20] = -1  # inside row 0's window
    out = torch.empty_like(p.q)
    args = (d.max_blocks, d.context_lens, d.query_start_loc, 2, 3, out, p.ws, p.ws_bytes)
    with pytest.raises(pkv.PkvError) as e:
        pkv.pkv_attention(h, 0, p.q, bad, *args)
    assert e.value.status == pkv.PKV_ERR_OUT_OF_RANGE
    bad[0, 20], bad[0, 25] = d.block_tables[0, 20], -1  # the block of the new token itself
    with pytest.raises(pkv.PkvError) as e:
        pkv.pkv_slot_mapping(h, bad, d.max_blocks, d.context_lens, d.query_start_loc, 2, 3, d.slot_mapping)
    assert e.value.status == pkv.PKV_ERR_OUT_OF_RANGE
    full = workload.Attention(p.pool, d)
    with pytest.raises(pkv.PkvError) as e:  # a full plan needs the blocks that were given back
        full.plan()
        full.run(0, p.q, out)
    assert e.value.status == pkv.PKV_ERR_OUT_OF_RANGE
    assert p.pool.check() == 0


def test_a_block_missing_inside_the_window_is_reported(cuda, built):
    batch = synth.custom_batch(synth.Shape(1, 4, 2, 64), [400, 600], [1, 20], seed=6)
    for row, block in ((0, 20), (1, 36)):
        p = Pass(batch, 100, 4)
        p.ds.block_tables[row, block] = -1
        p.plan()
        p.run()
        torch.cuda.synchronize()
        assert p.pool.check() == pkv.PKV_DEVERR_BLOCK_RANGE
