"""CPU tests of the latent oracles: against each other and plain cases."""

import numpy as np
import pytest

import oracle

RNG = np.random.default_rng(11)


def test_absorbed_and_expanded_are_the_same():
    """W_k's product taken to the queries or to the keys, W_v's after the mean or
    before it."""
    H, L, R, nope, prefix, n = 3, 32, 8, 16, 5, 4
    c, r = RNG.normal(size=(prefix + n, L)), RNG.normal(size=(prefix + n, R))
    q = RNG.normal(size=(n, H, nope + R))
    wk, wv = RNG.normal(size=(2, H, nope, L))
    out, lse, *_ = oracle.latent_prefill(q, wk, wv, c, r, prefix, 0.2)
    ql = np.einsum("nha,hal->nhl", q[..., :nope], wk)
    mean, lse2, *_ = oracle.latent_attention(ql, q[..., nope:], c, r, prefix, None, 0.2)
    assert np.allclose(np.einsum("nhl,hal->nha", mean, wv), out, rtol=1e-10, atol=1e-12)
    assert np.allclose(lse, lse2, rtol=1e-12)


def test_latent_attention_is_attention_of_one_shared_head():
    H, L, R, prefix, n = 4, 16, 8, 6, 5
    c, r = RNG.normal(size=(prefix + n, L)), RNG.normal(size=(prefix + n, R))
    ql, qr = RNG.normal(size=(n, H, L)), RNG.normal(size=(n, H, R))
    parents = [0, 0, 1, 1]
    out, lse, *_ = oracle.latent_attention(ql, qr, c, r, prefix, parents, -0.3)
    k = np.concatenate([c, r], 1)[None]
    v = np.concatenate([c, 0 * r], 1)[None]
    want, lse2, *_ = oracle.tree_attention(np.concatenate([ql, qr], 2), k, v, prefix, parents, -0.3)
    assert np.allclose(out, want[..., :L], rtol=1e-10, atol=1e-12)
    assert np.allclose(lse, lse2, rtol=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_equal_positions_on_all_axes_are_one(interleaved):
    rot, D = 16, 24
    table = RNG.normal(size=(9, rot))
    x, w = RNG.normal(size=D), RNG.normal(size=D)
    axis = [i % 3 for i in range(rot // 2)]
    got = oracle.axes_turn(x, w, 1e-6, table, (5, 5, 5), axis, interleaved)
    assert np.allclose(got, oracle.norm_rope(x, w, 1e-6, table[5], rot, interleaved))
    # one pair alone turns by its own axis
    got = oracle.axes_turn(x, None, 1e-6, table, (5, 7, 5), axis, interleaved)
    one = oracle.norm_rope(x, None, 1e-6, table[7], rot, interleaved)
    a, b = (2, 3) if interleaved else (1, 1 + rot // 2)
    assert got[a] == one[a] and got[b] == one[b]


def test_latent_e4m3_has_an_exponent_for_each_group():
    x = np.concatenate([RNG.normal(size=128) * 1e-4, RNG.normal(size=128) * 1e4])
    y = oracle.latent_e4m3(x)
    assert np.all(np.abs(y - x) <= np.maximum(2.0 ** -4 * np.abs(x),
                                              np.repeat([1e-4, 1e4], 128) * 2.0 ** -8))
