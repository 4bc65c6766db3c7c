"""Oracles of the target pass over a latent cache, and of the rotation by
positions on several axes.

Test infrastructure only (see ``oracle/__init__.py``). Everything is computed in
float64 from the definitions, a request at a time. A cache is a dense array per
request here; the paging is undone by the caller.
"""

from __future__ import annotations

import numpy as np

from .target import e4m3_exponent, e4m3_round, tree_paths

GROUP = 128  # elements of an 8-bit latent that share an exponent


def axes_turn(x, weight, eps, table, positions, pair_axis, interleaved):
    """One head x [D]: norm (weight None: none), then the rotation of pair i by the
    entry i of table row positions[pair_axis[i]]."""
    x = np.asarray(x, np.float64)
    if weight is not None:
        x = x / np.sqrt(np.mean(x * x) + eps) * np.asarray(weight, np.float64)
    y, h = x.copy(), len(pair_axis)
    for i, axis in enumerate(pair_axis):
        row = table[int(positions[axis])]
        c, s = float(row[i]), float(row[h + i])
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
        y[a] = x[a] * c - x[b] * s
        y[b] = x[b] * c + x[a] * s
    return y


def latent_e4m3(x):
    """The values that 8 bits keep of latents [..., L], an exponent for each GROUP."""
    y = np.asarray(x, np.float64).reshape(*x.shape[:-1], -1, GROUP)
    return e4m3_round(y, e4m3_exponent(y)).reshape(x.shape)


def _softmax(s, seen, v, size, scale):
    """s [H, n, T] scores, seen [n, T], v [H or 1, T, d]: outputs [n, H, d], log sums
    [n, H], the weighted means of |v| [n, H, d]; and `size` [H, n, T] (sums of
    magnitudes of the scores' terms) at its largest over the keys seen [n, H]."""
    s = np.where(seen, scale * s, -np.inf)
    m = s.max(-1, keepdims=True)
    w = np.exp(s - m)
    total = w.sum(-1, keepdims=True)
    lse = (m + np.log(total))[..., 0]
    w = w / total
    top = abs(scale) * np.where(seen, size, 0.0).max(-1)
    t = lambda a: np.swapaxes(a, 0, 1)  # noqa: E731
    return t(w @ v), t(lse), t(w @ np.abs(v)), t(top)


def latent_attention(ql, qr, c, r, prefix, parents, scale):
    """ql [n, H, L], qr [n, H, R], c [T, L], r [T, R] of one request with T = prefix
    + n; parents None: chain. Returns what _softmax does."""
    n, T = ql.shape[0], c.shape[0]
    seen = np.zeros((n, T), bool)
    seen[:, :prefix] = True
    for j, path in enumerate(tree_paths(list(range(n - 1)) if parents is None else parents, n)):
        seen[j, [prefix + i for i in path]] = True
    q = np.swapaxes(np.concatenate([ql, qr], -1), 0, 1)
    k = np.concatenate([c, r], -1)
    return _softmax(q @ k.T, seen, c[None], np.abs(q) @ np.abs(k).T, scale)


def latent_prefill(q, wk, wv, c, r, prefix, scale):
    """q [n, H, nope + R], wk and wv [H, nope, L], c [T, L], r [T, R] of one request
    with T = prefix + n. Returns what _softmax does, and the magnitudes behind the
    expansion: the sums sum |q| |k| of its rounded part and sum |q| (|wk| |c|), at
    their largest over the keys seen [n, H], and the weighted means of |wv| |c|
    [n, H, nope]."""
    n, T, nope = q.shape[0], c.shape[0], wk.shape[1]
    seen = np.arange(T) <= prefix + np.arange(n)[:, None]
    qh = np.swapaxes(q, 0, 1)
    kn, v = c @ np.swapaxes(wk, 1, 2), c @ np.swapaxes(wv, 1, 2)  # [H, T, nope]
    s = qh[..., :nope] @ np.swapaxes(kn, 1, 2) + qh[..., nope:] @ r.T
    qa, ka = np.abs(qh), np.abs(kn)
    rounded = qa[..., :nope] @ np.swapaxes(ka, 1, 2)
    size = rounded + qa[..., nope:] @ np.abs(r).T
    out = _softmax(s, seen, v, size, scale)
    deep_k = np.abs(c) @ np.swapaxes(np.abs(wk), 1, 2)
    deep_v = np.abs(c) @ np.swapaxes(np.abs(wv), 1, 2)
    spread = qa[..., :nope] @ np.swapaxes(deep_k, 1, 2)
    most = lambda a: np.swapaxes(abs(scale) * np.where(seen, a, 0.0).max(-1), 0, 1)  # noqa: E731
    w = np.exp(np.where(seen, scale * s, -np.inf) - np.swapaxes(out[1], 0, 1)[..., None])
    return out + (most(rounded), most(spread), np.swapaxes(w @ deep_v, 0, 1))
