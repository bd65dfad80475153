"""GPU: pkv_norm_rope_append at the ends of its arguments' ranges."""
import numpy as np
import pytest
import torch

from continuous_batching_paged_ragged_gb300 import pkv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", [pkv.PKV_KV_F16, pkv.PKV_KV_INT4])
@pytest.mark.parametrize("offset", [1e20, -1e20, 65504.0, 0.0])
def test_zeros_stay_zeros_under_the_largest_factor(cuda, built, kv, offset):
    """The root's reciprocal is 1e15 for a head of zeros at the least eps; its product with the weights has to be finite."""
    T, hq, hkv, d = 5, 4, 2, 128
    pool = pkv.Pool(1, hq, hkv, d, 2, kv_dtype=kv)
    pool.buffer[:-256].zero_()
    rope = pkv.Rope(d, 64)
    rng = np.random.default_rng(1)
    q = np.zeros((T, hq, d), np.float16)
    q[1, 0] = rng.standard_normal(d).astype(np.float16)
    q[1, 0, ::3] = 0
    q[2, 1, 5] = np.float16(2.0**-24)
    k = torch.zeros(T, hkv, d, dtype=torch.float16, device="cuda")
    w = torch.full((d,), 65504.0 if offset >= 0 else -65504.0, dtype=torch.float16, device="cuda")
    pos, slots = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.arange(T, device="cuda")
    dq, out = torch.from_numpy(q).cuda(), torch.full((T, hq, d), float("nan"), dtype=torch.float16, device="cuda")
    pkv.pkv_norm_rope_append(pool.handle, 0, rope.handle, w, w, 1e-30, offset, dq, hq * d, k, hkv * d, k, hkv * d, pos, slots, T, out)
    assert pool.check() == 0
    got = out.cpu().numpy()
    assert not np.isnan(got).any()
    assert (got[q == 0] == 0).all()  # position 0 turns nothing
    live = got[q != 0].astype(np.float64) * np.sign(q[q != 0].astype(np.float64)) * (1 if offset >= 0 else -1)
    assert (live > 0).all()
    ko, vo = torch.full_like(k, 1.0), torch.full_like(k, 1.0)
    pkv.pkv_gather(pool.handle, 0, slots, T, ko, vo)
    assert not ko.any() and not vo.any()


def test_larger_offsets_are_refused(cuda, built):
    T, hq, hkv, d = 2, 2, 1, 64
    pool = pkv.Pool(1, hq, hkv, d, 2)
    q, k = (torch.zeros(T, h, d, dtype=torch.float16, device="cuda") for h in (hq, hkv))
    w, slots = torch.ones(d, dtype=torch.float16, device="cuda"), torch.arange(T, device="cuda")
    for offset in (1.001e20, -1.001e20, 1e30, -3e38, float("inf"), float("-inf"), float("nan")):
        with pytest.raises(pkv.PkvError) as e:
            pkv.pkv_norm_rope_append(pool.handle, 0, None, w, w, 1e-6, offset, q, hq * d, k, hkv * d, k, hkv * d, None, slots, T,
                                     torch.empty_like(q))
        assert e.value.status == pkv.PKV_ERR_INVALID_ARG and "weight_offset" in pkv.pkv_last_error()
        assert pkv.pkv_last_launch_count(pool.handle) == 0
