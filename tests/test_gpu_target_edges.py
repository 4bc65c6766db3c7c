"""GPU tests of the target pass at the edges of what its calls take: lengths that
start late or are out of order, weights and exponents at the ends of their types,
buffers and views of unusual sizes.

Tolerances as in test_gpu_target.py unless a test says otherwise.
"""

import numpy as np
import pytest
import torch

import dspark_verify_scheduling_amd as dv
import oracle
from _gpu import DEV, say
from test_gpu_target import Batch, bits, i32, make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu(hip):
    return hip


# ------------------------------------------------------------------ requests of a read

def filled(B, seed=3, D=64, page=16):
    """A batch of short chains in a cache, and the rows appended to it."""
    rng = np.random.default_rng(B)
    lens = rng.integers(2, 5, B).tolist()
    b = Batch(seed, lens, rng.integers(0, 40, B).tolist(), 4, page, False)
    cache = make_cache("bf16", b.nb, 1, page, D)
    rows = torch.randn(b.rows, 1, D, device=DEV).bfloat16()
    ap = dv.alloc_append_outputs(b.rows, 1, cache)
    dv.dspark_kv_append(B, 4, rows, rows, rows, b.rows, *b.args(), cache, ap)
    torch.cuda.synchronize()
    assert ap.append_meta.tolist() == [int(b.cu[-1]), 0]
    return b, cache, rows


@pytest.mark.parametrize("B,lo", [(6, 2), (300, 17), (300, 299)])
def test_read_of_the_later_part_of_a_batch(B, lo):
    """Lengths that start above 0: the rows before them belong to no request."""
    say(f"read of requests {lo}..{B - 1}")
    b, cache, rows = filled(B)
    rd = dv.alloc_kv_read_outputs(b.rows, cache)
    for t in rd[:2]:
        t.fill_(-7)
    dv.dspark_kv_read(B - lo, b.rows, i32(b.cu[lo:]), i32(b.ctx[lo:]), i32(b.table[lo:]), cache, rd)
    torch.cuda.synchronize()
    c0, c1 = int(b.cu[lo]), int(b.cu[-1])
    assert rd.read_meta.tolist() == [c1, 0]
    for t in rd[:2]:
        assert torch.equal(t[c0:c1], rows[c0:c1])
        assert bool((t[:c0] == -7).all()) and bool((t[c1:] == -7).all())


@pytest.mark.parametrize("B", [5, 300])
def test_read_stays_inside_its_arrays_where_lengths_are_out_of_order(B):
    say(f"read, one length out of order, B={B}")
    b, cache, rows = filled(B)
    total = int(b.cu[-1])
    for at in (0, B // 2, B - 1):
        for value in (10 ** 6, -5, total, 1):
            cu = b.cu.copy()
            cu[at] = value
            rd = dv.alloc_kv_read_outputs(b.rows, cache)
            rd.k_out.fill_(-7)
            dv.dspark_kv_read(B, b.rows, i32(cu), i32(b.ctx), i32(b.table), cache, rd)
            torch.cuda.synchronize()
            meta = rd.read_meta.tolist()
            bad = any(s < 0 or e < s or e > total for s, e in zip(cu[:-1], cu[1:]))
            assert meta[0] == total and bool(meta[1] & oracle.DATA_BAD_LENS) == bad, (at, value)
            assert bool((rd.k_out[total:] == -7).all())


@pytest.mark.parametrize("kind,hkv,D,B", [("bf16", 1, 64, 4), ("e4m3", 8, 128, 70), ("f16", 2, 64, 300)])
def test_read_leaves_other_requests_alone_where_lengths_are_out_of_order(kind, hkv, D, B):
    """Every row that one well-formed request claims comes back, whatever the other
    lengths are; a row that none claims is not written, and one that several claim
    is a row of one of them."""
    say(f"read beside malformed lengths {kind} hkv={hkv} D={D} B={B}")
    rng = np.random.default_rng(B)
    lens = rng.integers(1, 5, B).tolist()
    b = Batch(2, lens, rng.integers(0, 40, B).tolist(), 4, 16, False)
    cache = make_cache(kind, b.nb, hkv, 16, D)
    x = torch.randn(b.rows, hkv, D, device=DEV).to(cache.row_dtype)
    ap = dv.alloc_append_outputs(b.rows, hkv, cache)
    dv.dspark_kv_append(B, 4, x, x, x, b.rows, *b.args(), cache, ap)
    total, reach = int(b.cu[-1]), b.width * b.page
    per_slot = {}  # what the cache holds at (page, offset), as bits
    pages = bits(cache.k).cpu()
    scales = None if cache.k_scale is None else cache.k_scale.cpu()
    ctx = np.array(b.ctx)

    def want(r, j):
        i = int(ctx[r]) + j
        pg, of = int(b.table[r, i // 16]), i % 16
        if pg < 0:
            return None
        if (pg, of) not in per_slot:
            v = pages[pg, :, of]
            if scales is not None:
                e = scales[pg, :, of].double() - 127
                v = v.view(torch.float8_e4m3fn).double() * torch.exp2(e)[:, None]
            per_slot[pg, of] = v.to(cache.row_dtype)
        return per_slot[pg, of]

    shuffled = rng.permutation(b.cu[:-1])
    trials = [(at, w) for at in (B // 3, B // 2) for w in (10 ** 6, -5, total, 0)] + [(None, None)]
    alone = 0
    for at, w in trials:
        cu = b.cu.copy()
        if at is None:
            cu[:-1] = shuffled
        else:
            cu[at] = w
        claims = {}
        for r in range(B):
            s, e = int(cu[r]), int(cu[r + 1])
            if 0 <= s <= e <= total and ctx[r] + e - s <= reach:
                for row in range(s, e):
                    claims.setdefault(row, []).append(want(r, row - s))
        outs = []
        for _ in range(2):
            rd = dv.alloc_kv_read_outputs(b.rows, cache)
            rd.k_out.fill_(-7)
            dv.dspark_kv_read(B, b.rows, i32(cu), i32(ctx), i32(b.table), cache, rd)
            torch.cuda.synchronize()
            outs.append(rd.k_out.cpu())
        assert torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16))
        for row in range(b.rows):
            got = outs[0][row]
            may = [torch.full_like(got, -7) if v is None else v for v in claims.get(row, [None])]
            assert any(torch.equal(got.nan_to_num(9), v.nan_to_num(9)) for v in may), (at, w, row)
            alone += len(claims.get(row, [])) == 1
    assert alone >= total // 2
