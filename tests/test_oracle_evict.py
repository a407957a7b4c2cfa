"""Pins of the eviction oracle and of the delta rule's oracle from a given state."""
import numpy as np
import pytest

from oracle import evict
from oracle.gated_deltanet import gated_delta_rule, gated_deltanet


def test_weights_sum_to_the_heads_and_follow_one_softmax():
    rng = np.random.default_rng(0)
    q, keys = rng.standard_normal((24, 128)), rng.standard_normal((2, 43, 128))
    w = evict.block_weights(q, keys, 43, [0, 3, 7])
    assert abs(w.sum() - 24) < 1e-12
    # one dense softmax over the same tokens
    tok = [0, 1, 2, 3, 12, 13, 14, 15, 28, 29, 30, 31, 40, 41, 42]
    want = np.zeros(4)
    for h in range(24):
        x = keys[h // 12][tok] @ q[h] / np.sqrt(128)
        p = np.exp(x - x.max())
        p /= p.sum()
        want += [p[:4].sum(), p[4:8].sum(), p[8:12].sum(), p[12:].sum()]
    assert np.allclose(w, want, rtol=1e-12)


def test_weights_own_block_alone():
    q, keys = np.ones((24, 128)), np.ones((2, 2, 128))
    assert np.allclose(evict.block_weights(q, keys, 2, []), [24.0])


def test_kept_ties_protection_and_nan():
    assert evict.kept_blocks([1, 1, 1, 1], 4, 2, 0, 0) == [0, 1]
    assert evict.kept_blocks([0, 5, 1, 9, 2], 5, 3, 1, 1) == [0, 3, 4]
    assert evict.kept_blocks([np.nan, 0.0, -0.0, np.nan], 4, 2, 0, 0) == [1, 2]
    assert evict.kept_blocks([3, 2], 2, 4, 0, 0) == [0, 1]
    assert evict.kept_blocks([9, 9, 9, 9], 4, 2, 1, 1) == [0, 3]


@pytest.mark.parametrize("heads,key_heads", [(1, 1), (4, 2)])
def test_delta_rule_continues_a_state(heads, key_heads):
    rng = np.random.default_rng(1)
    T = 12
    q, k = (rng.standard_normal((T, key_heads, 8)) / 3 for _ in range(2))
    v = rng.standard_normal((T, heads, 8))
    la, beta = np.log(rng.uniform(0.5, 1, (T, heads))), rng.uniform(0, 1, (T, heads))
    rep = heads // key_heads
    want, ws = gated_deltanet(np.repeat(q, rep, 1), np.repeat(k, rep, 1), v, la, beta, [0, T],
                              with_state=True)
    S = np.zeros((heads, 8, 8))
    o1, S = gated_delta_rule(q[:5], k[:5], v[:5], la[:5], beta[:5], S)
    o2, S = gated_delta_rule(q[5:], k[5:], v[5:], la[5:], beta[5:], S)
    assert np.allclose(np.concatenate([o1, o2]), want, atol=1e-12)
    assert np.allclose(S, ws[0], atol=1e-12)
