"""GPU: calls on a 4-bit cache and of the normalising append as a serving program makes them: two passes at once on two streams,
captured and replayed with other inputs, with bad block tables beside good ones, and with another device current."""
import os
import re
import subprocess
import sys

import numpy as np
import pytest
import torch

import test_gpu_int4 as int4_tests
import test_gpu_other_device as other
from continuous_batching_paged_ragged_gb300 import pkv, synth, workload
from helpers_gpu import run_batch, row_slice

pytestmark = pytest.mark.gpu

INT4 = pkv.PKV_KV_INT4


def _bits(x):
    return x.contiguous().view(torch.uint8)


def _same(a, b):
    return torch.equal(_bits(a), _bits(b))


@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (12, 2, 128), (16, 4, 256)])
def test_two_passes_at_once_on_one_pool(cuda, built, hq, hkv, d):
    """Two plans in workspaces of their own, launched on two streams, each with its layer: the bits of one after the other."""
    rng = np.random.default_rng(d)
    batch = synth.custom_batch(synth.Shape(2, hq, hkv, d), rng.integers(1, 2500, 90), np.ones(90, np.int64), seed=4)
    pool, ds, outs = run_batch(batch, [0, 1], kv_dtype=INT4)
    qs, _, _ = workload.step_inputs(ds, [0, 1])
    plans = [workload.Attention(pool, ds) for _ in range(2)]
    for p in plans:
        p.plan()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[torch.full_like(qs[i], float("nan")) for _ in range(8)] for i in range(2)]
    for n in range(8):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                plans[i].run(i, qs[i], got[i][n])
    torch.cuda.synchronize()
    assert pool.check() == 0
    for i in range(2):
        assert all(_same(g, outs[i]) for g in got[i])


def test_bad_block_ids_are_reported_and_other_rows_served(cuda, built):
    batch = synth.custom_batch(synth.Shape(1, 12, 2, 128), [300, 2000, 50, 700], [1, 1, 1, 1], seed=9)
    pool, ds, outs = run_batch(batch, [0], kv_dtype=INT4)
    qs, _, _ = workload.step_inputs(ds, [0])
    good = ds.block_tables.clone()
    for bad in (-3, batch.num_blocks, 2**31 - 1):
        ds.block_tables.copy_(good)
        ds.block_tables[1, 77] = bad
        attn, out = workload.Attention(pool, ds), torch.full_like(qs[0], float("nan"))
        attn.plan()
        attn.run(0, qs[0], out)
        assert pool.check() == pkv.PKV_DEVERR_BLOCK_RANGE
        for b in (0, 2, 3):
            assert np.array_equal(row_slice(batch, out, b), row_slice(batch, outs[0], b))


@pytest.mark.parametrize("kv", [pkv.PKV_KV_F16, pkv.PKV_KV_E4M3, INT4])
def test_captured_norms_append_and_gather(cuda, built, kv):
    """The graph reads what its buffers hold when it is replayed: inputs, weights, positions and slots."""
    T, hq, hkv, d = 300, 8, 2, 128
    gen = torch.Generator(device="cuda").manual_seed(1)
    pool, twin = (pkv.Pool(1, hq, hkv, d, 40, kv_dtype=kv) for _ in range(2))
    rope = pkv.Rope(d)
    x = torch.randn(T, hq + 2 * hkv, d, device="cuda", generator=gen).half()
    wq, wk = (1 + 0.2 * torch.randn(2, d, device="cuda", generator=gen)).half()
    pos = torch.randint(0, 9000, (T,), dtype=torch.int32, device="cuda", generator=gen)
    slots = torch.randperm(40 * 16, device="cuda", generator=gen)[:T]
    out, ko, vo = torch.empty(T, hq, d, dtype=torch.float16, device="cuda"), *torch.empty(2, T, hkv, d, dtype=torch.float16, device="cuda")

    def step(pool, out, ko, vo):
        n = x.stride(0)
        pkv.pkv_norm_rope_append(pool.handle, 0, rope.handle, wq, wk, 1e-6, 0.0, x, n, x[:, hq:], n, x[:, hq + hkv:], n, pos, slots, T,
                                 out)
        pkv.pkv_gather(pool.handle, 0, slots, T, ko, vo)

    step(pool, out, ko, vo)
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            step(pool, out, ko, vo)
    for n in range(3):
        x.copy_(torch.randn(x.shape, device="cuda", generator=gen).half())
        wk.mul_(-0.5)
        pos.add_(1000)
        slots.copy_(slots.roll(7))
        graph.replay()
        want, kw, vw = torch.empty_like(out), torch.empty_like(ko), torch.empty_like(vo)
        step(twin, want, kw, vw)
        assert pool.check() == 0 and twin.check() == 0
        assert _same(out, want) and _same(ko, kw) and _same(vo, vw)


def test_new_calls_with_another_device_current(cuda, built, tmp_path):
    calls = """calls = [
    lambda: pkv.pkv_gather(pool, 0, ptr, 1, ptr, ptr + 4096, 0),
    lambda: pkv.pkv_norm_rope_append(pool, 0, rope, ptr, ptr, 1e-6, 0.0, None, 0, ptr, 128, ptr, 128, ptr, ptr, 1, None, 0),
    lambda: pkv.pkv_norm_rope_append(pool, 0, None, None, ptr, 1e-6, 0.0, None, 0, ptr, 128, ptr, 128, None, ptr, 1, None, 0),
]
"""
    probe, n = re.subn(r"calls = \[\n.*?\n\]\n", calls, other._PROBE, flags=re.S)
    assert n == 1
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    (tmp_path / "shim.c").write_text(other._SHIM)
    shim = str(tmp_path / "shim.so")
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", shim, str(tmp_path / "shim.c"), "-ldl"], check=True)
    r = subprocess.run([sys.executable, "-c", probe, root, shim], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, LD_PRELOAD=shim))
    assert r.returncode == 0 and "REFUSED 3" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("hq,hkv,d", int4_tests.SHAPES)
def test_a_window_at_every_head_layout(cuda, built, hq, hkv, d):
    int4_tests.test_window_with_freed_blocks_and_hidden_rubbish(cuda, built, hq, hkv, d, 100, 4, False)
