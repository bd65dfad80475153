"""GPU: what the window hides has no part in a result, whatever its memory holds -- the bytes that a program which restored only
the sinks and the window into fresh memory has never written.  Tolerances as in test_gpu_window."""
import pytest

from continuous_batching_paged_ragged_gb300 import pkv, synth
from test_gpu_window import Pass, _hidden

pytestmark = pytest.mark.gpu

F16, E4M3 = pkv.PKV_KV_F16, pkv.PKV_KV_E4M3


def _spoil(p, codes=0x7F, scale=255):
    """Every hidden token of the pass, those that share a block with visible ones too: its codes (or values: NaN) and scale bytes."""
    batch = p.batch
    for b in range(batch.num_seqs):
        ctx, ql = int(batch.context_lens[b]), int(batch.q_lens[b])
        for pos in _hidden(ctx, ql, p.window, p.sinks)[0]:
            if pos >= ctx - ql:
                continue  # a new token: appended by the pass
            block, slot = int(batch.block_tables[b, pos // 16]), pos % 16
            p.pool.cache_view()[0, :, block, :, slot] = codes if p.kv == E4M3 else float("nan")
            if p.kv == E4M3:
                p.pool.scales_view()[0, block, :, :, slot] = scale


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("shape", [(8, 2, 64), (12, 2, 128), (16, 4, 256), (2, 2, 256)])
@pytest.mark.parametrize("window,sinks", [(100, 4), (1, 0), (333, 17), (700, 1)])
def test_hidden_scale_bytes(cuda, built, shape, window, sinks, fused):
    """8-bit cache, rows of fewer than 16 new tokens: a scale byte of 255 decodes to infinity, beside NaN and beside ordinary codes."""
    cached, q_lens = [1200, 40, 333, 899, 2000, 17], [1, 1, 3, 15, 1, 1]
    batch = synth.custom_batch(synth.Shape(1, *shape), cached, q_lens, seed=9)
    for codes in (0x7F, 0x38):
        p = Pass(batch, window, sinks, E4M3)
        _spoil(p, codes)
        p.plan()
        p.check(p.run(fused))


@pytest.mark.parametrize("kv", [F16, E4M3])
@pytest.mark.parametrize("shape", [(4, 4, 64), (4, 2, 128), (12, 2, 128), (16, 2, 64), (6, 1, 256), (2, 2, 256)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (50, 4), (129, 130), (475, 15), (700, 1), (9, 33)])
def test_chunks_beside_hidden_values(cuda, built, kv, shape, window, sinks):
    """Rows of 16 or more new tokens whose hidden keys and values are NaN, those in partly visible blocks too: of the sinks' last
    block, of the window's first, or of one block that is both."""
    cached, q_lens = [0, 500, 37, 1000, 2000, 5, 513], [300, 40, 16, 1, 131, 2, 17]
    batch = synth.custom_batch(synth.Shape(1, *shape), cached, q_lens, seed=12)
    for codes in ((0x7F, 0x38) if kv == E4M3 else (None,)):
        p = Pass(batch, window, sinks, kv)
        _spoil(p, codes)
        p.plan()
        p.check(p.run(fused=True), sample=24)


@pytest.mark.parametrize("kv", [F16, E4M3])
@pytest.mark.parametrize("shape", [(12, 2, 128), (4, 1, 256)])
def test_split_chunks_beside_hidden_values(cuda, built, kv, shape):
    """A short chunk far into its row, whose work runs in two parts."""
    for cached, new, window, sinks in ((9000, 40, 6000, 100), (7000, 16, 4500, 0), (9000, 20, 5001, 1001)):
        p = Pass(synth.custom_batch(synth.Shape(1, *shape), [cached], [new], seed=13), window, sinks, kv)
        _spoil(p)
        p.plan()
        p.check(p.run(), sample=8)
