"""Target-pass oracles: cache append and read, tree attention, tree accept, commit.

Test infrastructure only (see ``oracle/__init__.py``). Everything is computed
in float64 from the definitions, one request, row and head at a time.

A tree is a list of parent rows: ``parents[j - 1]`` in [0, j - 1] is the parent
of row j, and row 0 the root. A cache is a dense array per request here; the
paging is undone by the caller's ``slots`` (page, offset) lists.

Readings (also in the design notes):

* The pages draft chains only. A tree's rows stay in the packed order, parents
  before children, so the planner's lengths cut trees to trees.
* Row j's position is prefix + depth(j); its cache index is prefix + j until
  the commit moves the accepted path together.
* Of several children with the predicted token the lowest row is taken.
"""

from __future__ import annotations

import numpy as np

from .accept import as_f32_rows, row_argmax
from .pack import DATA_BAD_LENS

DATA_BAD_TREE, DATA_BAD_PAGE, DATA_BAD_POS = 16, 32, 64


def tree_paths(parents, n):
    """For the n rows of a tree, each row's path from the root, itself included."""
    paths = [[0]]
    for j in range(1, n):
        paths.append(paths[int(parents[j - 1])] + [j])
    return paths


def tree_ok(parents, n):
    return all(0 <= int(parents[j - 1]) < j for j in range(1, n))


def e4m3_values():
    """The value of every code: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[c] = np.nan if c & 127 == 127 else (-x if c & 128 else x)
    return out


def e4m3_exponent(x):
    """Per row of x [..., D]: the least e with max |x| <= 448 * 2^e over the
    finite elements, held to [-100, 119]; 0 for a row of zeros."""
    top = np.abs(np.where(np.isfinite(x), x, 0.0)).max(-1)
    m, e = np.frexp(top / 448.0)  # m in [0.5, 1)
    e = np.where(m == 0.5, e - 1, e)
    return np.where(top == 0, 0, np.clip(e, -100, 119)).astype(np.int64)


def e4m3_round(x, e):
    """x [..., D] to the nearest value code * 2^e (ties to even), saturating."""
    y = np.clip(np.ldexp(np.where(np.isfinite(x), x, 0.0), -e[..., None]), -448.0, 448.0)
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6))) - 3)
    return np.where(np.isfinite(x), np.ldexp(np.rint(y / step) * step, e[..., None]), np.nan)


def norm_rope(x, weight, eps, table_row, rot, interleaved):
    """One head x [D]: norm (weight None: none), then rotation by a table row of
    rot / 2 cosines and rot / 2 sines (None: none)."""
    x = np.asarray(x, np.float64)
    if weight is not None:
        x = x / np.sqrt(np.mean(x * x) + eps) * np.asarray(weight, np.float64)
    if table_row is None:
        return x
    y = x.copy()
    h = rot // 2
    for i in range(h):
        c, s = float(table_row[i]), float(table_row[h + i])
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
        y[a] = x[a] * c - x[b] * s
        y[b] = x[b] * c + x[a] * s
    return y


def tree_attention(q, k, v, prefix, parents, scale):
    """q [n, Hq, D], k and v [Hkv, prefix + n, D] of one request; parents None:
    chain. Returns out [n, Hq, D], lse [n, Hq], and what error bounds need: the
    weighted mean of |v| [n, Hq, D] and the largest scale * sum |q||k| [n, Hq]."""
    n, hq, D = q.shape
    group = hq // k.shape[0]
    parents = list(range(n - 1)) if parents is None else parents
    out, mean_abs = np.zeros((n, hq, D)), np.zeros((n, hq, D))
    lse, top = np.zeros((n, hq)), np.zeros((n, hq))
    for j, path in enumerate(tree_paths(parents, n)):
        seen = list(range(prefix)) + [prefix + i for i in path]
        for h in range(hq):
            kk, vv = k[h // group][seen], v[h // group][seen]
            s = scale * (kk @ q[j, h])
            m = s.max()
            w = np.exp(s - m)
            lse[j, h] = m + np.log(w.sum())
            w = w / w.sum()
            out[j, h] = w @ vv
            mean_abs[j, h] = w @ np.abs(vv)
            top[j, h] = abs(scale) * (np.abs(kk) @ np.abs(q[j, h])).max()
    return out, lse, mean_abs, top


def tree_accept(B, gamma, rows, dtype, cu_seqlens, drafts, parents, prefix_lens=None,
                max_rows=None):
    """Greedy accept along trees; rows [>= total, V] packed logits."""
    B, gamma = int(B), int(gamma)
    cu = [int(c) for c in cu_seqlens]
    max_rows = rows.shape[0] if max_rows is None else int(max_rows)
    total = cu[B]
    total_eff = min(max(total, 0), max_rows)
    am = row_argmax(as_f32_rows(rows[:total_eff], dtype))
    prefix = [0] * B if prefix_lens is None else [int(p) for p in prefix_lens]
    status = 0 if total == total_eff else DATA_BAD_LENS
    num, bonus = np.zeros(B, np.int32), np.full(B, -1, np.int32)
    commit, new_seq = np.zeros(B, np.int32), np.array(prefix, np.int32)
    out = np.full((B, gamma + 1), -1, np.int32)
    paths = np.full((B, gamma + 1), -1, np.int32)
    for r in range(B):
        n = cu[r + 1] - cu[r]
        if not (cu[r] >= 0 and 1 <= n <= gamma + 1 and cu[r + 1] <= total_eff):
            status |= DATA_BAD_LENS
            continue
        par = list(range(gamma)) if parents is None else [int(p) for p in parents[r]]
        if not tree_ok(par, n):
            status |= DATA_BAD_TREE
            continue
        path, node = [0], 0
        while True:
            word = int(am[cu[r] + node])
            nxt = [j for j in range(1, n) if par[j - 1] == node and int(drafts[r][j - 1]) == word]
            if not nxt:
                break
            node = nxt[0]
            path.append(node)
        num[r], bonus[r] = len(path) - 1, am[cu[r] + node]
        commit[r], new_seq[r] = len(path), prefix[r] + len(path)
        out[r, :len(path)] = [int(drafts[r][j - 1]) for j in path[1:]] + [bonus[r]]
        paths[r, :len(path)] = path
    return {"row_argmax": am.astype(np.int32), "num_correct": num, "bonus": bonus,
            "commit": commit, "new_seq": new_seq, "out_tokens": out, "path_rows": paths,
            "meta": np.array([total, status], np.int32)}


def commit_moves(path_rows, num_correct, prefix, gamma):
    """(source, destination) cache indices of one request, or None where its
    path is not one."""
    c = int(num_correct)
    path = [int(p) for p in path_rows[:c + 1]] if 0 <= c <= gamma else []
    if not path or prefix < 0 or path[0] != 0:
        return None
    if any(b <= a for a, b in zip(path, path[1:])) or path[-1] > gamma:
        return None
    return [(prefix + p, prefix + k) for k, p in enumerate(path) if p != k]
