"""GPU: pkv_gather at every head size and cache format, and the normalising append of many tokens into each cache."""
import numpy as np
import pytest
import torch

from oracle import fp8, int4
from continuous_batching_paged_ragged_gb300 import pkv

pytestmark = pytest.mark.gpu

KINDS = [pkv.PKV_KV_F16, pkv.PKV_KV_E4M3, pkv.PKV_KV_INT4]


def _held(x, kv):
    """What fp16 rows stand for in a cache of this format (magnitudes here are far from the fp16 maximum)."""
    if kv == pkv.PKV_KV_F16:
        return x
    values = fp8.dequantize_rows(*fp8.quantize_rows(x)) if kv == pkv.PKV_KV_E4M3 else int4.values(x)
    return values.astype(np.float16)


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hkv,T", [(1, 1), (3, 37), (8, 700)])
def test_rows_come_back_as_what_they_stand_for(cuda, built, kv, d, hkv, T):
    rng = np.random.default_rng(d + T)
    blocks = -(-T // 16) + 3
    pool = pkv.Pool(2, hkv, hkv, d, blocks, kv_dtype=kv)
    pool.buffer[:-256].random_(0, 256, generator=torch.Generator(device="cuda").manual_seed(T))
    k, v = ((rng.standard_normal((T, hkv, d)) * np.exp2(rng.uniform(-18, 8, (T, hkv, 1)))).astype(np.float16) for _ in range(2))
    slots = torch.from_numpy(rng.permutation(blocks * 16)[:T]).cuda()
    pkv.pkv_append(pool.handle, 1, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), slots, T)
    before = pool.buffer.clone()
    order = torch.from_numpy(rng.integers(0, T, 2 * T + 5)).cuda()  # any slot any number of times
    ko, vo = torch.full((2, len(order), hkv, d), float("nan"), dtype=torch.float16, device="cuda")
    pkv.pkv_gather(pool.handle, 1, slots[order], len(order), ko, vo)
    assert pool.check() == 0 and torch.equal(pool.buffer, before)
    at = order.cpu().numpy()
    for got, x in ((ko, k), (vo, v)):
        assert np.array_equal(got.cpu().numpy(), _held(x, kv)[at])


@pytest.mark.parametrize("kv", KINDS[1:])
@pytest.mark.parametrize("hq,hkv,d,rot", [(12, 2, 128, 128), (8, 4, 64, 32), (6, 1, 256, 64)])
def test_many_tokens_normalised_into_a_quantized_cache(cuda, built, kv, hq, hkv, d, rot):
    """Thousands of tokens, more than a warp's run each: bit for bit the fp16 keys of the same call, appended."""
    T, blocks = 5003, 320
    g = torch.Generator(device="cuda").manual_seed(d)
    x = torch.randn(T, hq + 2 * hkv, d, generator=g, device="cuda").half()
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    n = x.stride(0)
    pos = torch.randint(0, 100000, (T,), generator=g, device="cuda", dtype=torch.int32)
    slots = torch.randperm(blocks * 16, generator=g, device="cuda")[:T]
    w = torch.rand(2, d, generator=g, device="cuda").half()
    rope = pkv.Rope(d, rot)
    pools = [pkv.Pool(1, hq, hkv, d, blocks, kv_dtype=t) for t in (pkv.PKV_KV_F16, kv, kv)]
    outs = [torch.empty(T, hq, d, dtype=torch.float16, device="cuda") for _ in range(2)]
    for p in pools:
        p.buffer[:-256].fill_(0x33)
    for p, out in zip(pools, outs):
        pkv.pkv_norm_rope_append(p.handle, 0, rope.handle, w[0], w[1], 1e-6, 0.0, q, n, k, n, v, n, pos, slots, T, out)
    keys = pools[0].layer(0, 0)[slots // 16, :, slots % 16].contiguous()
    pkv.pkv_append(pools[2].handle, 0, keys, v.contiguous(), slots, T)
    assert all(p.check() == 0 for p in pools)
    assert torch.equal(pools[1].buffer, pools[2].buffer) and torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16))
