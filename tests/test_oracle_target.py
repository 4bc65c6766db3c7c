"""The target-pass oracle against closed forms and independent restatements."""

import numpy as np
import pytest
import torch

import oracle


def test_tree_paths_and_checks():
    # rows: 0 - 1 - 3, 0 - 2 - 4 - 5
    parents = [0, 0, 1, 2, 4]
    assert oracle.tree_paths(parents, 6) == [[0], [0, 1], [0, 2], [0, 1, 3], [0, 2, 4], [0, 2, 4, 5]]
    assert oracle.tree_paths([0, 1, 2], 4)[-1] == [0, 1, 2, 3]  # the chain
    assert oracle.tree_ok(parents, 6)
    assert not oracle.tree_ok([0, 2], 3)  # its own parent
    assert not oracle.tree_ok([-1], 2)
    assert oracle.tree_ok([0, 9], 2)  # entries past the rows do not count


def test_e4m3_values_are_torchs():
    ref = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oracle.e4m3_values(), ref, equal_nan=True)


def test_e4m3_round_is_torchs_on_a_grid():
    x = np.concatenate([np.linspace(-470, 470, 9001), np.ldexp(np.linspace(1, 2, 33), -8),
                        np.ldexp(np.arange(40) / 4.0, -9)])
    got = oracle.e4m3_round(x[None], np.zeros(1, np.int64))[0]
    ref = torch.from_numpy(np.clip(x, -448, 448)).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(got, ref)


@pytest.mark.parametrize("top,e", [(448.0, 0), (448.0001, 1), (224.0, -1), (0.0, 0), (1.0, -8),
                                   (1.75, -8), (1.7500001, -7), (3e38, 119), (1e-45, -100)])
def test_e4m3_exponent(top, e):
    assert oracle.e4m3_exponent(np.array([[0.0, -top, top / 3]]))[0] == e


def test_e4m3_nonfinite():
    x = np.array([[np.nan, np.inf, -2.0, 1.0]])
    e = oracle.e4m3_exponent(x)
    y = oracle.e4m3_round(x, e)
    assert np.isnan(y[0, :2]).all() and np.array_equal(y[0, 2:], x[0, 2:])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_relative_angles(interleaved):
    rng = np.random.default_rng(0)
    D, rot = 64, 32
    f = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    table = lambda p: np.concatenate([np.cos(p * f), np.sin(p * f)])
    a, b = rng.normal(size=D), rng.normal(size=D)
    ra = lambda p: oracle.norm_rope(a, None, 0, table(p), rot, interleaved)
    rb = lambda p: oracle.norm_rope(b, None, 0, table(p), rot, interleaved)
    assert np.isclose(np.linalg.norm(ra(17)), np.linalg.norm(a))
    assert np.array_equal(ra(5)[rot:], a[rot:])
    assert np.isclose(ra(7) @ rb(3), ra(104) @ rb(100))


def test_norm_gives_unit_mean_square():
    x = np.random.default_rng(1).normal(0, 3, 128)
    y = oracle.norm_rope(x, np.ones(128), 0.0, None, 0, False)
    assert np.isclose(np.mean(y * y), 1.0)


def test_tree_attention_is_each_paths_own_attention():
    """A row of a tree gets what the last row of its path's chain gets."""
    rng = np.random.default_rng(2)
    D, prefix, n = 8, 5, 6
    parents = [0, 0, 1, 2, 4]
    k, v = rng.normal(size=(2, 2, prefix + n, D))
    q = rng.normal(size=(n, 4, D))
    out, lse, _, _ = oracle.tree_attention(q, k, v, prefix, parents, 0.3)
    for j, path in enumerate(oracle.tree_paths(parents, n)):
        seen = list(range(prefix)) + [prefix + i for i in path]
        o, l, _, _ = oracle.tree_attention(q[path], k[:, seen], v[:, seen], prefix, None, 0.3)
        assert np.allclose(o[-1], out[j]) and np.allclose(l[-1], lse[j])
    # one key: its value
    o, l, _, _ = oracle.tree_attention(q[:1], k[:, :1], v[:, :1], 0, None, 0.3)
    assert np.allclose(o[0, 0], v[0, 0]) and np.allclose(l[0, 0], 0.3 * q[0, 0] @ k[0, 0])


def test_tree_accept_on_chains_is_accept():
    rng = np.random.default_rng(3)
    B, gamma, V = 9, 5, 40
    lens = rng.integers(1, gamma + 2, B)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    rows = rng.normal(size=(int(cu[-1]), V)).astype(np.float32)
    am = oracle.row_argmax(rows)
    drafts = rng.integers(0, V, (B, gamma)).astype(np.int32)
    for r in range(B):
        for j in range(1, lens[r]):
            if rng.random() < 0.8:
                drafts[r, j - 1] = am[cu[r] + j - 1]
    prefix = rng.integers(0, 99, B).astype(np.int32)
    t = oracle.tree_accept(B, gamma, rows, "f32", cu, drafts, None, prefix)
    a = oracle.accept(B, gamma, rows, "f32", cu, drafts, prefix)
    for x, y in (("num_correct", "num_correct"), ("bonus", "bonus"), ("commit", "commit"),
                 ("new_seq", "new_seq"), ("row_argmax", "row_argmax"), ("meta", "meta")):
        assert np.array_equal(t[x], a[y]), x
    for r in range(B):
        c = int(t["num_correct"][r])
        assert np.array_equal(t["out_tokens"][r, :c + 1], a["out_tokens"][r, :c + 1])
        assert t["path_rows"][r].tolist() == list(range(c + 1)) + [-1] * (gamma - c)


def test_tree_accept_by_hand():
    V = 10
    says = [3, 5, 7, 1, 9]  # what rows 0..4 predict
    rows = np.zeros((5, V), np.float32)
    rows[np.arange(5), says] = 1
    # rows 1 and 2 are children of the root, 3 of 2, 4 of 3; drafts 4, 3, 7, 2
    r = oracle.tree_accept(1, 4, rows, "f32", [0, 5], [[4, 3, 7, 2]], [[0, 0, 2, 3]], [10])
    assert r["path_rows"][0].tolist() == [0, 2, 3, -1, -1]
    assert r["out_tokens"][0].tolist() == [3, 7, 1, -1, -1]
    assert (r["num_correct"][0], r["bonus"][0], r["new_seq"][0]) == (2, 1, 13)
    assert oracle.commit_moves(r["path_rows"][0], 2, 10, 4) == [(12, 11), (13, 12)]
    # equal siblings: the lower row
    r = oracle.tree_accept(1, 2, rows, "f32", [0, 3], [[3, 3]], [[0, 0]])
    assert r["path_rows"][0].tolist() == [0, 1, -1]


def test_commit_moves_refuses_what_is_no_path():
    f = oracle.commit_moves
    assert f([0, 1, 2, -1], 2, 5, 3) == []
    assert f([0, 2, 2, -1], 2, 5, 3) is None
    assert f([1, 2, -1, -1], 1, 5, 3) is None
    assert f([0, 4, -1, -1], 1, 5, 3) is None
    assert f([0, 1, 2, 3], 4, 5, 3) is None
    assert f([-1, -1], 0, 5, 1) is None
