"""GPU tests of the latent cache's calls on batches at the edge of what they take: words
of cu_seqlens out of order, requests that claim others' rows. Tolerances as in
test_gpu_latent.py."""

import numpy as np
import pytest
import torch

import dspark_verify_scheduling_amd as dv
from _gpu import DEV, say
from test_gpu_latent import R, latent_setup, prefill_check, typed
from test_gpu_target import TYPES, Batch, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu(hip):
    return hip


# ------------------------------------------------------------------ lengths out of order

def disorder(cu, ctx, most=10 ** 9):
    """A batch of these words, whose last is the largest, and who has which rows: the
    lengths of those that have any, and the requests that are well formed but have rows in
    common with a well-formed one ahead."""
    total, mine, lost, own = cu[-1], [], [], set()
    for r, c in enumerate(ctx):
        rows = set(range(cu[r], cu[r + 1]))
        good = 0 <= cu[r] <= cu[r + 1] <= total and c >= 0 and len(rows) <= most
        if good and any(m & rows for m in mine):
            lost.append(r)
        mine.append(rows if good else set())
    lens = [0 if r in lost else len(m) for r, m in enumerate(mine)]
    # pages for everybody's rows, as if they were in order
    b = Batch(3, [max(0, e - s) for s, e in zip(cu, cu[1:])], [max(c, 0) for c in ctx], 1, 16, False)
    b.cu, b.lens, b.rows = np.asarray(cu, np.int32), lens, total + 3
    for r, n in enumerate(lens):
        own |= mine[r] if n else set()
    return b, lost, torch.tensor([n not in own for n in range(b.rows)], device=DEV)


OUT_OF_ORDER = [  # words, contexts
    ([0, 300, 0, 300, 301], [0, 0, 0, 0]),     # one row behind others that two claim
    ([0, 384] * 10, [5] * 19),                 # thirty tiles claim three tiles' rows
    ([7, 100, 50, 120, 110, 130], [30, 0, 9, 0, 64]),
    ([40, 90, 0, 40, 20, 90, 95], [3, 0, 70, 0, 8, 0]),
    ([0, 60, 60, 0, 60, 61], [-1, 0, 0, 12, 0]),  # a malformed one claims nothing
    ([0] + [2, 1] * 150 + [3, 200], [1] * 302),
]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", range(len(OUT_OF_ORDER)))
def test_latent_prefill_where_lengths_go_back(case, kind):
    """Rows that several well-formed requests claim are the first one's; the others are
    left out, and nobody loses rows that none of these claims."""
    cu, ctx = OUT_OF_ORDER[case]
    say(f"latent prefill, words out of order, case {case} {kind}")
    H, n, L = 3, 64, 256
    b, lost, nobody = disorder(cu, ctx)
    full, b.lens = b.lens, [max(0, e - s) for s, e in zip(cu, cu[1:])]
    cache, _, _ = latent_setup(b, kind, 1, L)
    b.lens = full
    rng, dt = np.random.default_rng(1), TYPES[kind][1]
    q = typed(rng, (b.rows, H, n + R), dt).to(DEV)
    w = typed(rng, (H, 2 * n, L), dt, L ** -0.5).to(DEV)
    keys = sum(c + max(0, e - s) for c, s, e in zip(b.ctx, cu, cu[1:]))
    o = dv.alloc_latent_prefill_outputs(b.B, b.rows, keys, H, n, cache, lse=True)
    for _ in range(3):
        o.workspace.fill_(0xFF)
        o.out.fill_(-7)
        o.lse.fill_(-7)
        dv.dspark_latent_prefill(b.B, q, w[:, :n], w[:, n:], b.rows, keys, i32(cu), i32(ctx),
                                 i32(b.table), cache, 0.07, o)
        torch.cuda.synchronize()
        assert o.attention_meta.tolist() == [cu[-1], dv.DATA_BAD_LENS]
        prefill_check(b, kind, H, n, L, 0.07, cache, q, w[:, :n], w[:, n:], o)
        assert bool((o.out[nobody] == -7).all()) and bool((o.lse[nobody] == -7).all())
