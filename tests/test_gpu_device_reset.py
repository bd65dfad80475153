"""GPU: what the library remembers of a device's context does not outlive it.  A process of its own, without torch: every call that
asks for more shared memory than a kernel gets by default, before and after cudaDeviceReset, to the same bits.  (A second device is
the same case: function attributes belong to a context.)"""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

_PROBE = r"""
import ctypes, sys
sys.path.insert(0, sys.argv[1])
import numpy as np
from continuous_batching_paged_ragged_gb300 import pkv

pkv.load()
rt = ctypes.CDLL("libcudart.so.13")

def ok(e):
    assert e == 0, e

def dev(x=None, nbytes=None):
    p = ctypes.c_void_p()
    ok(rt.cudaMalloc(ctypes.byref(p), ctypes.c_size_t(nbytes or x.nbytes)))
    ok(rt.cudaMemset(p, 0, ctypes.c_size_t(nbytes or x.nbytes)))
    if x is not None:
        ok(rt.cudaMemcpy(p, x.ctypes.data_as(ctypes.c_void_p), ctypes.c_size_t(x.nbytes), 1))
    return p.value

def host(p, shape, dtype):
    x = np.empty(shape, dtype)
    ok(rt.cudaDeviceSynchronize())
    ok(rt.cudaMemcpy(x.ctypes.data_as(ctypes.c_void_p), ctypes.c_void_p(p), ctypes.c_size_t(x.nbytes), 2))
    return x

def everything():
    results = []
    rng = np.random.default_rng(0)
    for kv in (pkv.PKV_KV_F16, pkv.PKV_KV_E4M3):
        blocks, hq, hkv, d = 64, 12, 2, 128
        cfg = pkv.pkv_config(1, hq, hkv, d, 16, blocks, 0, kv)
        n = pkv.pkv_pool_bytes(cfg)
        pool = pkv.pkv_pool_init(cfg, dev(nbytes=n), n)
        ctx, ql = np.array([300, 120, 40], np.int32), np.array([1, 20, 40], np.int32)
        qsl = np.concatenate([[0], np.cumsum(ql)]).astype(np.int32)
        tables = rng.permutation(blocks)[:60].reshape(3, 20).astype(np.int32)
        T, bt, dc, dq = int(qsl[-1]), dev(tables), dev(ctx), dev(qsl)
        at = [(b, t) for b in range(3) for t in range(ctx[b])]
        slots = dev(np.array([tables[b, t // 16] * 16 + t % 16 for b, t in at], np.int64))
        k, v = (dev(rng.standard_normal((len(at), hkv, d)).astype(np.float16)) for _ in range(2))
        q, out = dev(rng.standard_normal((T, hq, d)).astype(np.float16)), dev(nbytes=T * hq * d * 2)
        pkv.pkv_append(pool, 0, k, v, slots, len(at), 0)
        for window in (0, 90):
            size = pkv.pkv_attention_window_workspace_bytes(pool, 3, T, 20, window, 4) if window else pkv.pkv_attention_workspace_bytes(pool, 3, T, 20)
            ws = dev(nbytes=size)
            if window:
                pkv.pkv_attention_window_plan(pool, dc, dq, 3, T, 20, window, 4, ws, size, 0)
            else:
                pkv.pkv_attention_plan(pool, dc, dq, 3, T, 20, ws, size, 0)
            pkv.pkv_attention(pool, 0, q, bt, 20, dc, dq, 3, T, out, ws, size, 0)
            results.append(host(out, (T, hq, d), np.uint16))
        pkv.pkv_attention_noalloc(pool, 0, q, bt, 20, dc, dq, 3, T, out, 0)
        results.append(host(out, (T, hq, d), np.uint16))
        pkv.pkv_copy_blocks(pool, dev(np.array([[tables[0, 0], next(b for b in range(blocks) if b not in tables)]], np.int32)), 1, 0)
        for wide in (20, 400):  # the small compaction, and the one in two launches
            wt = np.full((3, wide), -1, np.int32)
            wt[:, :20] = tables
            remap, live, new = dev(nbytes=4 * blocks), dev(nbytes=4), dev(nbytes=wt.nbytes)
            size = pkv.pkv_compact_workspace_bytes(pool)
            pkv.pkv_compact(pool, dev(wt), wide, 3, new, remap, live, dev(nbytes=size), size, 0)
            results.append(host(remap, (blocks,), np.int32))
        assert pkv.pkv_pool_check(pool) == 0
        results.append(host(pkv.pkv_pool_layer_ptr(pool, 0, 1), (n // 4,), np.uint8))
        pkv.pkv_pool_destroy(pool)
    return results

first = everything()
ok(rt.cudaDeviceReset())
second = everything()
assert len(first) == len(second) == 12 and all(np.array_equal(a, b) for a, b in zip(first, second))
print("SAME")
"""


def test_calls_after_a_device_reset(cuda, built):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _PROBE, root], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "SAME" in r.stdout, r.stderr[-2000:]
