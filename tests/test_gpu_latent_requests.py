"""GPU tests of the latent cache's calls on batches at the edge of what they take: words
of cu_seqlens out of order, requests that claim others' rows. Tolerances as in
test_gpu_latent.py."""

import numpy as np
import pytest
import torch

import dspark_verify_scheduling_amd as dv
import oracle
from _gpu import DEV, say
from test_gpu_latent import R, attention_bound, latent_setup, lget, prefill_check, typed
from test_gpu_target import TYPES, Batch, W, f64, i32, make_cache, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu(hip):
    return hip


# ------------------------------------------------------------------ requests that start late

@pytest.mark.parametrize("B", [1, 3, 300])
def test_axes_positions_of_nobody_do_not_count(B):
    """Requests of a part of the packed rows: positions before the first one's rows are not
    looked at; a bad one of theirs still counts where words are out of order."""
    say(f"append axes, rows that start late, B={B}")
    start, D = 40, 64
    b = Batch(B, [3] * B, [7] * B, 1, 16, False)
    b.cu = b.cu + start
    b.rows += start
    cache = make_cache("bf16", b.nb, 1, 16, D)
    x = typed(b.rng, (b.rows, 1, D), torch.bfloat16).to(DEV)
    pos = torch.zeros(2, b.rows, dtype=torch.int32, device=DEV)
    pos[:, :start] = -1
    rope = torch.zeros(5, D, device=DEV)

    def call(cu):
        o = dv.alloc_append_outputs(b.rows, 1, cache)
        o.q_out.fill_(-7)
        dv.dspark_kv_append_axes(B, x, x, x, b.rows, i32(cu), i32(b.ctx), pos, [i % 2 for i in range(D // 2)],
                                 i32(b.table), cache, o, rope)
        torch.cuda.synchronize()
        return o

    total = int(b.cu[-1])
    o = call(b.cu)
    assert o.append_meta.tolist() == [total, 0]
    assert bool((o.q_out[:start] == -7).all()) and bool((o.q_out[start:total] == 0).all())
    pos[1, total - 1] = 5
    assert call(b.cu).append_meta.tolist() == [total, dv.DATA_BAD_POS]
    pos[1, total - 1] = 0
    pos[0, start + 4 if B > 1 else start] = -2
    assert call(b.cu).append_meta.tolist() == [total, dv.DATA_BAD_POS]
    if B > 1:  # the first request's word is beyond the others'
        for word in (total, 2 ** 31 - 1):
            cu = b.cu.copy()
            cu[0] = word
            assert call(cu).append_meta.tolist() == [total, dv.DATA_BAD_LENS | dv.DATA_BAD_POS]


# ------------------------------------------------------------------ lengths out of order

def disorder(cu, ctx, most=10 ** 9):
    """A batch of these words, whose last is the largest, the lengths of its requests as
    far as they are well formed and have no rows of a well-formed one ahead, and which
    rows are nobody's."""
    cu, total = [int(c) for c in cu], int(cu[-1])
    lens, seen, nobody = [], [], torch.ones(total + 3, dtype=torch.bool)
    for s, e, c in zip(cu, cu[1:], ctx):
        good = 0 <= s <= e <= total and c >= 0 and e - s <= most
        free = good and not any(s < y and x < e for x, y in seen)
        if good:
            seen.append((s, e))
        lens.append(e - s if free else 0)
        if free:
            nobody[s:e] = False
    # pages for everybody's rows, as if they were in order
    b = Batch(3, [max(0, e - s) for s, e in zip(cu, cu[1:])], [max(c, 0) for c in ctx], 8, 16, False)
    b.cu, b.rows = np.asarray(cu, np.int32), total + 3
    return b, lens, nobody.to(DEV)


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
    b, lens, nobody = disorder(cu, ctx)
    cache, _, _ = latent_setup(b, kind, 1, L)
    keys, b.lens = sum(b.ctx) + sum(b.lens), lens
    rng, dt = np.random.default_rng(1), TYPES[kind][1]
    q = typed(rng, (b.rows, H, n + R), dt).to(DEV)
    w = typed(rng, (H, 2 * n, L), dt, L ** -0.5).to(DEV)
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


def test_latent_prefill_of_more_keys_than_32_bits_count():
    """A request whose last cache index passes 2^31 is left out for its keys, as any that
    passes max_keys; the one ahead of it is not."""
    say("latent prefill, keys past 2^31")
    H, n, L, page = 2, 64, 256, 256
    b = Batch(2, [20, 10], [30, 0], 1, page, False)
    cache, _, _ = latent_setup(b, "bf16", 1, L)
    q = typed(b.rng, (b.rows, H, n + R), torch.bfloat16).to(DEV)
    w = typed(b.rng, (H, 2 * n, L), torch.bfloat16, L ** -0.5).to(DEV)
    table = torch.zeros(2, 2 ** 31 // page + 1, dtype=torch.int32, device=DEV)
    table[:, :b.width] = i32(np.maximum(b.table, 0))
    o = dv.alloc_latent_prefill_outputs(2, b.rows, 60, H, n, cache, lse=True)
    for prefix, rows in ((2 ** 31 - 5, (0,)), (2 ** 31 - 11, (0,)), (0, (0, 1))):
        o.out.fill_(-7)
        o.lse.fill_(-7)
        dv.dspark_latent_prefill(2, q, w[:, :n], w[:, n:], b.rows, 60, i32(b.cu), i32([30, prefix]), table,
                                 cache, 0.07, o)
        torch.cuda.synchronize()
        assert o.attention_meta.tolist() == [30, dv.DATA_BAD_LENS if prefix else 0]
        prefill_check(b, "bf16", H, n, L, 0.07, cache, q, w[:, :n], w[:, n:], o,
                      [r for r in (0, 1) if r not in rows])


def swapped(B, gamma, seed):
    """Words in order but for some that have changed places with one a few further."""
    rng = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(rng.integers(1, gamma + 2, B))])
    for i in rng.integers(0, B - 4, max(1, B // 20)):
        j = i + int(rng.integers(1, 4))
        cu[i], cu[j] = cu[j], cu[i]
    return cu.tolist(), rng.integers(0, 60, B).tolist()


SHORT_OUT_OF_ORDER = [  # words, contexts; up to 9 rows a request
    ([0, 5, 0, 5, 6], [40, 3, 100, 0]),
    ([0, 9] * 12, [70] * 23),
    ([3, 9, 5, 12, 10, 14], [30, 0, 9, 0, 64]),
    ([4, 9, 0, 4, 2, 9, 11], [3, 0, 70, 0, 8, 0]),
    ([0, 6, 6, 0, 6, 7], [-1, 0, 0, 12, 0]),      # malformed ones claim nothing:
    ([0, 20, 12, 20, 21], [50, 0, 31, 64]),       # too many rows
    ([0] + [2, 1] * 150 + [3, 8], [1] * 302),
    swapped(64, 8, 1), swapped(65, 8, 2), swapped(300, 4, 3), swapped(2500, 2, 4),
]


@pytest.mark.parametrize("kind,L,H", [("bf16", 512, 5), ("f16", 256, 33), ("e4m3", 512, 40)])
@pytest.mark.parametrize("case", range(len(SHORT_OUT_OF_ORDER)))
def test_latent_attention_where_lengths_go_back(case, kind, L, H):
    cu, ctx = SHORT_OUT_OF_ORDER[case]
    say(f"latent attention, words out of order, case {case} {kind} L={L}")
    if len(ctx) > 400:
        H = 2
    b, lens, nobody = disorder(cu, ctx, 9)
    assert 0 < sum(lens) and len(lens) > sum(n > 0 for n in lens)
    if len(ctx) > 400:  # pages of others' will do
        b.nb = b.nb // 4
        b.table = np.where(b.table >= 0, b.table % b.nb, b.table)
    cache, ql, qr = latent_setup(b, kind, H, L)
    o = dv.alloc_latent_attention_outputs(b.B, 8, b.rows, H, cache, lse=True)
    for _ in range(3):
        o.workspace.fill_(0xFF)
        o.out.fill_(-7)
        o.lse.fill_(-7)
        dv.dspark_latent_attention(b.B, 8, ql, qr, b.rows, i32(cu), i32(ctx), i32(b.table), cache, 0.05, o)
        torch.cuda.synchronize()
        assert o.attention_meta.tolist() == [cu[-1], dv.DATA_BAD_LENS]
        assert bool((o.out[nobody] == -7).all()) and bool((o.lse[nobody] == -7).all())
    got, got_lse, u = f64(o.out), f64(o.lse), TYPES[kind][2]
    for r, n in enumerate(lens):
        if not n:
            continue
        T, s = ctx[r] + n, slice(cu[r], cu[r + 1])
        lat, rope = lget(cache, b.slots(r, 0, T))
        ref, lse, mean_abs, top = oracle.latent_attention(f64(ql[s]), f64(qr[s]), lat, rope, ctx[r], None, 0.05)
        bound, lse_bound = attention_bound(ref, lse, mean_abs, (L + R + 16) * W * top,
                                           np.abs(lat).max(), T, u, kind)
        within(got[s], ref, bound, (r, "out"))
        within(got_lse[s], lse, lse_bound, (r, "lse"))


# ------------------------------------------------------------------ orders of rows and heads

@pytest.mark.parametrize("kind,L,H", [("bf16", 512, 20), ("f16", 256, 3), ("e4m3", 512, 128)])
def test_queries_of_a_product_for_each_head(kind, L, H):
    """Queries as a product for each head leaves them, a head's rows together, give what
    the same queries in rows do, bit for bit; so does the append, in place too."""
    say(f"latent queries by head {kind} L={L} H={H}")
    b = Batch(4, [5, 1, 3], [100, 0, 700], 4, 16, True)
    cache, ql, qr = latent_setup(b, kind, H, L)
    n = int(b.cu[-1])
    ql[n:], qr[n:] = 0, 0
    rope = torch.randn(800, R, device=DEV)
    kv = typed(b.rng, (b.rows, L + R), ql.dtype).to(DEV)
    by_head = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (ql, qr)]
    assert by_head[0].stride(0) == L and by_head[1].stride(1) == b.rows * R
    got = []
    for latent, turned, place in ((ql, qr.contiguous(), False), (*by_head, False), (*by_head, True)):
        ap = dv.alloc_latent_append_outputs(b.rows, H, cache)
        if place:
            ap = ap._replace(q_rope=turned)
        elif latent is not ql:
            ap = ap._replace(q_rope=torch.empty_like(turned.transpose(0, 1)).transpose(0, 1))
            assert ap.q_rope.stride(0) == R
        if not place:
            ap.q_rope.fill_(-7)
        dv.dspark_latent_append(b.B, kv, b.rows, *b.args(), cache, ap, q_rope=turned, rope=rope, gamma=4,
                                tree_parents=b.par())
        o = dv.alloc_latent_attention_outputs(b.B, 4, b.rows, H, cache, lse=True)
        dv.dspark_latent_attention(b.B, 4, latent, ap.q_rope, b.rows, *b.args(), cache, 0.05, o,
                                   tree_parents=b.par())
        torch.cuda.synchronize()
        assert ap.append_meta.tolist() == [n, 0] and o.attention_meta.tolist() == [n, 0]
        assert bool((ap.q_rope[n:] == (0 if place else -7)).all())
        got.append([ap.q_rope[:n].clone(), o.out[:n].clone(), o.lse[:n].clone()])
    for other in got[1:]:
        for x, y in zip(got[0], other):
            assert torch.equal(x, y)


@pytest.mark.parametrize("which", ["w_k", "w_v"])
def test_weights_of_other_heads_are_refused(which):
    """A share of the heads needs its share of the weights: more than q has heads would be
    the first heads' without a word."""
    say(f"latent prefill, {which} of other heads")
    n, L = 64, 256
    b = Batch(2, [5], [0], 1, 16, False)
    cache, _, _ = latent_setup(b, "bf16", 1, L)
    q = torch.zeros(b.rows, 2, n + R, dtype=torch.bfloat16, device=DEV)
    w = torch.zeros(4, n, L, dtype=torch.bfloat16, device=DEV)
    o = dv.alloc_latent_prefill_outputs(1, b.rows, 5, 2, n, cache)
    for heads in (4, 1):
        weights = {"w_k": w[:2], "w_v": w[:2], which: w[:heads]}
        with pytest.raises(ValueError, match=which):
            dv.dspark_latent_prefill(1, q, weights["w_k"], weights["w_v"], b.rows, 5, *b.args(), cache, 0.1, o)
    dv.dspark_latent_prefill(1, q, w[:2], w[2:], b.rows, 5, *b.args(), cache, 0.1, o)
    torch.cuda.synchronize()
    assert o.attention_meta.tolist() == [5, 0]


@pytest.mark.parametrize("kind,H,cuts", [("bf16", 8, (0, 3, 8)), ("e4m3", 5, (0, 1, 2, 5))])
def test_prompts_by_shares_of_the_heads(kind, H, cuts):
    """A call for some heads at a time, in a workspace of their size, gives what one call
    for all does, bit for bit."""
    say(f"latent prefill by shares of heads {kind}")
    n, L = 64, 256
    b = Batch(6, [150, 1, 40], [30, 200, 0], 1, 16, False)
    cache, _, _ = latent_setup(b, kind, 1, L)
    dt = TYPES[kind][1]
    q = typed(b.rng, (b.rows, H, n + R), dt).to(DEV)
    w = typed(b.rng, (H, 2 * n, L), dt, L ** -0.5).to(DEV)
    keys = sum(b.ctx) + sum(b.lens)
    whole = dv.alloc_latent_prefill_outputs(3, b.rows, keys, H, n, cache, lse=True)
    parts = torch.full_like(whole.out, -7)
    for o in (whole.out, whole.lse):
        o.fill_(-7)
    dv.dspark_latent_prefill(3, q, w[:, :n], w[:, n:], b.rows, keys, *b.args(), cache, 0.07, whole)
    for lo, hi in zip(cuts, cuts[1:]):
        o = dv.alloc_latent_prefill_outputs(3, b.rows, keys, hi - lo, n, cache, lse=True)
        assert o.workspace.numel() < whole.workspace.numel()
        o.lse.fill_(-7)
        o = o._replace(out=parts[:, lo:hi])
        dv.dspark_latent_prefill(3, q[:, lo:hi], w[lo:hi, :n], w[lo:hi, n:], b.rows, keys, *b.args(), cache,
                                 0.07, o)
        torch.cuda.synchronize()
        assert o.attention_meta.tolist() == [int(b.cu[-1]), 0]
        assert torch.equal(o.lse, whole.lse[:, lo:hi])
    assert torch.equal(parts, whole.out)
