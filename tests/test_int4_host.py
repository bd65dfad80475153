"""The 4-bit cache and the normalising append without a GPU: sizes, and refusals that need no pool."""
from continuous_batching_paged_ragged_gb300 import pkv


def test_pool_bytes_follow_the_header_layout(built):
    """18 head_dim bytes a (layer, block, KV head), padded to 256, then the status area."""
    for layers, hkv, d, nb in [(1, 2, 64, 64), (3, 4, 128, 10), (2, 1, 256, 7), (1, 1, 64, 1)]:
        cfg = pkv.pkv_config(layers, 2 * hkv, hkv, d, 16, nb, 0, pkv.PKV_KV_INT4)
        assert pkv.pkv_pool_bytes(cfg) == (layers * nb * hkv * 18 * d + 255) // 256 * 256 + 256
    # past 32 bits of bytes
    cfg = pkv.pkv_config(80, 64, 8, 128, 16, 100000, 0, pkv.PKV_KV_INT4)
    assert pkv.pkv_pool_bytes(cfg) == 80 * 100000 * 8 * 2304 + 256
    for kv in (2, 3, 5, -1):
        assert pkv.pkv_pool_bytes(pkv.pkv_config(1, 4, 2, 64, 16, 64, 0, kv)) == 0


def test_calls_without_a_pool_are_refused(built):
    assert built.pkv_gather(None, 0, None, 1, None, None, None) == pkv.PKV_ERR_INVALID_ARG
    assert b"pool" in built.pkv_last_error()
    assert built.pkv_norm_rope_append(None, 0, None, None, None, 1e-6, 0.0, None, 0, None, 0, None, 0, None, None, 1, None,
                                      None) == pkv.PKV_ERR_INVALID_ARG
    assert b"pool" in built.pkv_last_error()
