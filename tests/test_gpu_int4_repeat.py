"""GPU: the 4-bit decode's hand-over of shares between warps, launch after launch: rows whose warps finish at very different
times give the same bits every time.  (What orders the shares' reads is in the source; a run can only fail to show it missing.)"""
import numpy as np
import pytest
import torch

from continuous_batching_paged_ragged_gb300 import pkv, synth, workload
from helpers_gpu import run_batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,d", [(8, 1, 64), (12, 2, 128), (8, 1, 256)])
@pytest.mark.parametrize("window", [0, 700])
def test_a_hundred_launches_give_the_same_bits(cuda, built, hq, hkv, d, window):
    rng = np.random.default_rng(d)
    cached = np.concatenate([rng.integers(1, 200, 400), rng.integers(1000, 3000, 100)])
    batch = synth.custom_batch(synth.Shape(1, hq, hkv, d), cached[rng.permutation(500)], np.ones(500, np.int64), seed=4)
    pool, ds, outs = run_batch(batch, [0], kv_dtype=pkv.PKV_KV_INT4)
    qs, _, _ = workload.step_inputs(ds, [0])
    shape = (ds.num_seqs, ds.num_tokens, ds.max_blocks)
    if window:
        n = pkv.pkv_attention_window_workspace_bytes(pool.handle, *shape, window, 4)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        pkv.pkv_attention_window_plan(pool.handle, ds.context_lens, ds.query_start_loc, *shape, window, 4, ws, n)
    else:
        n = pkv.pkv_attention_workspace_bytes(pool.handle, *shape)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        pkv.pkv_attention_plan(pool.handle, ds.context_lens, ds.query_start_loc, *shape, ws, n)
    got = [torch.full_like(qs[0], float("nan")) for _ in range(100)]
    for out in got:
        pkv.pkv_attention(pool.handle, 0, qs[0], ds.block_tables, ds.max_blocks, ds.context_lens, ds.query_start_loc, ds.num_seqs,
                          ds.num_tokens, out, ws, n)
    assert pool.check() == 0
    first = got[0] if window else outs[0]
    assert all(torch.equal(g.view(torch.int16), first.view(torch.int16)) for g in got)
