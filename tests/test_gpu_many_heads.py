"""GPU: as many KV heads as a task can name, and the refusal of more."""
import pytest
import torch

from continuous_batching_paged_ragged_gb300 import pkv, synth
from helpers_gpu import assert_close, host_rows, oracle_row, oracle_row_8bit, row_slice, run_batch

pytestmark = pytest.mark.gpu

KINDS = [pkv.PKV_KV_F16, pkv.PKV_KV_E4M3, pkv.PKV_KV_INT4]


@pytest.mark.parametrize("kv", KINDS)
def test_256_kv_heads(cuda, built, kv):
    batch = synth.custom_batch(synth.Shape(1, 256, 256, 64), [40, 0, 17], [1, 1, 3], seed=2)
    pool, ds, outs = run_batch(batch, [0], kv_dtype=kv, split_blocks=2)
    for b in range(3):
        if kv == pkv.PKV_KV_INT4:
            import oracle
            from oracle import int4
            q, k, v = host_rows(batch, 0)[b]
            want = oracle.attention_row(q, int4.values(k), int4.values(v))
        else:
            want = (oracle_row_8bit if kv == pkv.PKV_KV_E4M3 else oracle_row)(batch, 0, b)
        assert_close(row_slice(batch, outs[0], b), want, f"row {b}")


@pytest.mark.parametrize("kv", KINDS)
def test_more_are_refused(cuda, built, kv):
    pool = pkv.Pool(1, 257, 257, 64, 2, kv_dtype=kv)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ctx, starts, tables = i32(3), i32(0, 1), torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    x = torch.zeros(1, 257, 64, dtype=torch.float16, device="cuda")
    out, slots = torch.empty_like(x), torch.tensor([2], device="cuda")
    n = pkv.pkv_attention_workspace_bytes(pool.handle, 1, 1, 1)
    ws = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
    tail = (tables, 1, ctx, starts, 1, 1, out)
    for call in (lambda: pkv.pkv_attention_plan(pool.handle, ctx, starts, 1, 1, 1, ws, n),
                 lambda: pkv.pkv_attention_window_plan(pool.handle, ctx, starts, 1, 1, 1, 2, 0, ws, n),
                 lambda: pkv.pkv_attention(pool.handle, 0, x, *tail, ws, n),
                 lambda: pkv.pkv_attention_append(pool.handle, 0, x, x, x, slots, *tail, ws, n),
                 lambda: pkv.pkv_attention_noalloc(pool.handle, 0, x, *tail)):
        with pytest.raises(pkv.PkvError) as e:
            call()
        assert e.value.status == pkv.PKV_ERR_UNSUPPORTED and "256 KV heads" in pkv.pkv_last_error()
        assert pkv.pkv_last_launch_count(pool.handle) == 0
    # what does not attend still serves them
    pkv.pkv_append(pool.handle, 0, x, x, slots, 1)
    ko, vo = torch.full_like(x, 1.0), torch.full_like(x, 1.0)
    pkv.pkv_gather(pool.handle, 0, slots, 1, ko, vo)
    assert pool.check() == 0 and not ko.any() and not vo.any()
