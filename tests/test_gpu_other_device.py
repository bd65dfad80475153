"""GPU: every call that launches refuses to while another device than the pool's is current.  One device is enough: in a process of
its own, a preloaded cudaGetDevice names another one while the calls are made, all of them refused on the host."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

_SHIM = r"""
#define _GNU_SOURCE
#include <dlfcn.h>
int shim_device = -1;  /* named instead of the current one */
int cudaGetDevice(int* device) {
  int (*real)(int*) = (int (*)(int*))dlsym(dlopen("libcudart.so.13", RTLD_NOW | RTLD_NOLOAD), "cudaGetDevice");
  int e = real(device);
  if (shim_device >= 0) *device = shim_device;
  return e;
}
"""

_PROBE = r"""
import ctypes, sys
sys.path.insert(0, sys.argv[1])
shim = ctypes.CDLL(sys.argv[2])
from continuous_batching_paged_ragged_gb300 import pkv
rt = ctypes.CDLL("libcudart.so.13")
p = ctypes.c_void_p()
assert rt.cudaMalloc(ctypes.byref(p), ctypes.c_size_t(1 << 26)) == 0 and rt.cudaMemset(p, 0, ctypes.c_size_t(1 << 26)) == 0
at = p.value
cfg = pkv.pkv_config(1, 4, 2, 64, 16, 8, 0, 0)
n = pkv.pkv_pool_bytes(cfg)
pool = pkv.pkv_pool_init(cfg, at, n)
rope = pkv.pkv_rope_create(pkv.pkv_rope_config(64, 0, 0, 0, 1e4, 1.0, 0.0, 0.0, 0.0, 0.0))
ptr = at + (1 << 25)  # zeros, for every argument
ws, size = at + (1 << 24), 1 << 22
pkv.pkv_attention_plan(pool, ptr, ptr, 1, 1, 4, ws, size, 0)
rest = (ptr, 4, ptr, ptr, 1, 1, ptr + 4096)
calls = [
    lambda: pkv.pkv_slot_mapping(pool, ptr, 4, ptr, ptr, 1, 1, ptr, 0),
    lambda: pkv.pkv_append(pool, 0, ptr, ptr, ptr, 1, 0),
    lambda: pkv.pkv_attention_plan(pool, ptr, ptr, 1, 1, 4, ws, size, 0),
    lambda: pkv.pkv_attention_window_plan(pool, ptr, ptr, 1, 1, 4, 16, 0, ws, size, 0),
    lambda: pkv.pkv_attention(pool, 0, ptr, *rest, ws, size, 0),
    lambda: pkv.pkv_attention_append(pool, 0, ptr, ptr, ptr, ptr, *rest, ws, size, 0),
    lambda: pkv.pkv_attention_noalloc(pool, 0, ptr, *rest, 0),
    lambda: pkv.pkv_positions(pool, ptr, ptr, 1, 1, ptr, 0),
    lambda: pkv.pkv_rope_append(pool, 0, rope, None, 0, ptr, 128, ptr, 128, ptr, ptr, 1, None, 0),
    lambda: pkv.pkv_copy_blocks(pool, ptr, 1, 0),
    lambda: pkv.pkv_fork_rows(pool, ptr, 4, ptr, 1, ptr, 1, 0),
    lambda: pkv.pkv_compact(pool, ptr, 4, 1, ptr + 4096, ptr + 8192, ptr + 12288, ws, size, 0),
]
ctypes.c_int.in_dll(shim, "shim_device").value = 1
for i, call in enumerate(calls):
    try:
        call()
    except pkv.PkvError as e:
        assert e.status == pkv.PKV_ERR_INVALID_ARG and "current device" in str(e), (i, str(e))
    else:
        raise AssertionError(f"call {i} was not refused")
    assert pkv.pkv_last_launch_count(pool) in (0, 1)
ctypes.c_int.in_dll(shim, "shim_device").value = -1
pkv.pkv_positions(pool, ptr, ptr, 1, 1, ptr, 0)
print("REFUSED", len(calls))
"""


def test_calls_with_another_device_current(cuda, built, tmp_path):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    (tmp_path / "shim.c").write_text(_SHIM)
    shim = str(tmp_path / "shim.so")
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", shim, str(tmp_path / "shim.c"), "-ldl"], check=True)
    r = subprocess.run([sys.executable, "-c", _PROBE, root, shim], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, LD_PRELOAD=shim))
    assert r.returncode == 0 and "REFUSED 12" in r.stdout, r.stderr[-2000:]
