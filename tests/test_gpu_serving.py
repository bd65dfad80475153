"""GPU: the cache's operators together, as a serving loop uses them -- scheduled passes whose keys are rotated on their way
into the cache and attended through a window, requests forked between passes, the pool compacted under them -- every
row against the float64 oracle over its own history."""
import random

import numpy as np
import pytest
import torch

import oracle
from oracle import fp8
from continuous_batching_paged_ragged_gb300 import pkv
from helpers_gpu import assert_close, poison

pytestmark = pytest.mark.gpu

HQ, HKV, D, BLOCKS, WINDOW, SINKS = 4, 2, 64, 60, 50, 5


def _values(tag, pos):
    """q, k, v of the token that the history `tag` computed at a position."""
    r = np.random.default_rng([tag, pos]).standard_normal((HQ + 2 * HKV, D)).astype(np.float16)
    return r[:HQ], r[HQ:HQ + HKV], r[HQ + HKV:]


def _rotate(x, pos, freq):
    """Half layout, float64, rounded once: [T, H, D]."""
    a = pos[:, None, None] * freq
    y, h = x.astype(np.float64), len(freq)
    out = y.copy()
    out[..., :h], out[..., h:2 * h] = y[..., :h] * np.cos(a) - y[..., h:2 * h] * np.sin(a), y[..., h:2 * h] * np.cos(a) + y[..., :h] * np.sin(a)
    return out.astype(np.float16)


def _dev(x, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype).cuda()


def _serve(kv_dtype, seed=3):
    rng = random.Random(seed)
    sched = pkv.Scheduler(8, 64, 16, BLOCKS, prefix_caching=True)
    pool = pkv.Pool(1, HQ, HKV, D, BLOCKS, kv_dtype=kv_dtype)
    poison(pool)
    h = pool.handle
    rope = pkv.Rope(D, 32, base=10000.0, scaling="ramp", factor=4.0, original_context=64)
    freq = rope.frequencies()
    history, next_id, forked, compacted, passes = {}, 0, 0, 0, 0
    while passes < 60:
        if next_id < 25 and rng.random() < 0.5:
            sched.add(next_id, rng.choice([1, 5, 16, 33, 70, 120]), rng.randint(2, 40))
            history[next_id] = {}
            next_id += 1
        st = sched.step()
        passes += 1
        T = int(st["query_start_loc"][-1])
        if T == 0:
            continue
        B, W = len(st["req_ids"]), st["max_blocks_per_seq"]
        rows = []
        for rid, n, c in zip(st["req_ids"].tolist(), st["q_lens"].tolist(), st["context_lens"].tolist()):
            for p in range(c - n, c):
                history[rid].setdefault(p, rid)
            rows.append([_values(history[rid][p], p) for p in range(c)])
        new = [x[c - n:] for x, n, c in zip(rows, st["q_lens"].tolist(), st["context_lens"].tolist())]
        packed = _dev(np.stack([np.concatenate(t) for x in new for t in x]), torch.float16)  # [T, HQ + 2 HKV, D]
        bt, ctx, qsl = _dev(st["block_tables"]), _dev(st["context_lens"]), _dev(st["query_start_loc"])
        pos, slots = torch.empty(T, dtype=torch.int32, device="cuda"), torch.empty(T, dtype=torch.int64, device="cuda")
        pkv.pkv_positions(h, ctx, qsl, B, T, pos)
        pkv.pkv_slot_mapping(h, bt, W, ctx, qsl, B, T, slots)
        q = torch.empty(T, HQ, D, dtype=torch.float16, device="cuda")
        out = torch.empty_like(q)
        s = packed.stride(0)
        pkv.pkv_rope_append(h, 0, rope.handle, packed, s, packed[:, HQ:], s, packed[:, HQ + HKV:], s, pos, slots, T, q)
        n = pkv.pkv_attention_window_workspace_bytes(h, B, T, W, WINDOW, SINKS)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        pkv.pkv_attention_window_plan(h, ctx, qsl, B, T, W, WINDOW, SINKS, ws, n)
        pkv.pkv_attention(h, 0, q, bt, W, ctx, qsl, B, T, out, ws, n)
        torch.cuda.synchronize()
        assert pool.check() == 0
        assert np.array_equal(slots.cpu().numpy(), st["slot_mapping"])
        got = out.cpu().numpy()
        for b in range(B):
            c, nq = int(st["context_lens"][b]), int(st["q_lens"][b])
            p = np.arange(c)
            k = _rotate(np.stack([t[1] for t in rows[b]]), p, freq)
            v = np.stack([t[2] for t in rows[b]])
            if kv_dtype == pkv.PKV_KV_E4M3:
                k, v = (fp8.dequantize_rows(*fp8.quantize_rows(x)) for x in (k, v))
            ql = _rotate(np.stack([t[0] for t in rows[b]])[c - nq:], p[c - nq:], freq)
            ref = oracle.window_attention_row(ql, k, v, WINDOW, SINKS)
            q0 = int(st["query_start_loc"][b])
            assert_close(got[q0:q0 + nq], ref, f"pass {passes} row {b}")
        running, tables = sched.tables()
        if running.size and rng.random() < 0.35:
            i = rng.randrange(running.size)
            parent, child = int(running[i]), next_id
            done = max(history[parent]) + 1
            try:
                block = sched.fork(parent, child, rng.randint(20, 60))
            except pkv.PkvError:
                pass
            else:
                next_id += 1
                forked += 1
                history[child] = dict(history[parent])
                computed = int(st["context_lens"][st["req_ids"].tolist().index(parent)]) if parent in st["req_ids"] else done
                two = np.full((2, tables.shape[1]), -1, np.int32)
                two[0] = tables[i]
                dt, dc = _dev(two), _dev([computed, 0])
                pkv.pkv_fork_rows(h, dt, two.shape[1], dc, 2, _dev([[0, 1, block]]), 1)
                ids, now = sched.tables()
                mine = now[ids.tolist().index(child)]
                child_row = dt[1].cpu().numpy()
                w = min(len(mine), len(child_row))
                assert np.array_equal(child_row[:w], mine[:w]) and dc.tolist() == [computed, computed]
        if rng.random() < 0.3:
            ids, tables = sched.tables()
            if ids.size:
                dt = _dev(tables)
                remap, live = torch.empty(BLOCKS, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
                nb = pkv.pkv_compact_workspace_bytes(h)
                cws = torch.empty(nb, dtype=torch.uint8, device="cuda")
                pkv.pkv_compact(h, dt, tables.shape[1], len(ids), dt, remap, live, cws, nb)
                sched.remap(remap.cpu().numpy())
                assert np.array_equal(sched.tables()[1], dt.cpu().numpy())
                assert sched.free_list() == list(range(int(live), BLOCKS))
                compacted += 1
    assert pool.check() == 0
    return forked, compacted


@pytest.mark.parametrize("kv_dtype", [pkv.PKV_KV_F16, pkv.PKV_KV_E4M3])
def test_serving_with_forks_and_compactions(cuda, built, kv_dtype):
    forked, compacted = _serve(kv_dtype)
    assert forked >= 3 and compacted >= 3
