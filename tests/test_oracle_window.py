"""CPU: the windowed oracle against the unwindowed one, hand-worked masks and keys it must not touch."""
import numpy as np
import pytest

import oracle


def _row(q_len, ctx, hq, hkv, d, seed=0):
    rng = np.random.default_rng(seed)
    return [rng.standard_normal(s).astype(np.float16) for s in ((q_len, hq, d), (ctx, hkv, d), (ctx, hkv, d))]


def test_visible_keys_by_hand():
    assert oracle.visible_keys(0, 1, 0).tolist() == [0]
    assert oracle.visible_keys(5, 1, 0).tolist() == [5]
    assert oracle.visible_keys(5, 3, 0).tolist() == [3, 4, 5]
    assert oracle.visible_keys(5, 3, 2).tolist() == [0, 1, 3, 4, 5]
    assert oracle.visible_keys(5, 3, 4).tolist() == [0, 1, 2, 3, 4, 5]
    assert oracle.visible_keys(2, 9, 9).tolist() == [0, 1, 2]


@pytest.mark.parametrize("window,sinks", [(40, 0), (1000, 7), (1, 40)])
def test_everything_visible_is_the_unwindowed_oracle(window, sinks):
    q, k, v = _row(9, 40, 6, 2, 16)
    np.testing.assert_allclose(oracle.window_attention_row(q, k, v, window, sinks), oracle.attention_row(q, k, v), rtol=1e-12, atol=1e-14)


def test_a_window_without_sinks_is_attention_over_a_slice():
    q, k, v = _row(1, 50, 4, 4, 16)
    got = oracle.window_attention_row(q, k, v, 20, 0)
    np.testing.assert_allclose(got, oracle.attention_row(q, k[30:], v[30:]), rtol=1e-12, atol=1e-14)


def test_one_key_is_its_value_and_hidden_keys_are_not_read():
    q, k, v = _row(3, 30, 2, 1, 16)
    k[:27], v[:27] = np.nan, np.inf
    got = oracle.window_attention_row(q, k, v, 1, 0)
    assert np.array_equal(got, np.repeat(v[27:].astype(np.float64), 2, axis=1))


def test_uniform_scores_average_the_visible_values():
    q, k, v = _row(2, 12, 1, 1, 8)
    got = oracle.window_attention_row(np.zeros_like(q), k, v, 4, 2)
    for i, keys in enumerate(([0, 1, 7, 8, 9, 10], [0, 1, 8, 9, 10, 11])):
        np.testing.assert_allclose(got[i, 0], v[keys, 0].astype(np.float64).mean(0), rtol=1e-12)
