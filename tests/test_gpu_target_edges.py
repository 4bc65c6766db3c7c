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
from test_gpu_target import (TYPES, W, Batch, attention_check, bits, f64, get, i32, make_cache, put,
                             within)
from test_gpu_target_steps import ref_long

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


# ------------------------------------------------------------------ scores at the ends of their range

@pytest.mark.parametrize("kind,D,size", [
    ("bf16", 128, 3e4), ("bf16", 64, 1e9), ("f16", 64, 9e3), ("f16", 256, 3e4), ("e4m3", 128, 3e4)])
def test_equal_scores_of_any_size_give_the_mean(kind, D, size):
    """Keys all alike: the weights are equal however large the scores are, and the
    output is the mean of the values. Equal scores have equal weights p, so sum p v
    / sum p errs by the rounding of p, of n float32 additions each and of the
    output; the scores' own errors cancel."""
    say(f"equal scores of size {size:g}^2 {kind} D={D}")
    code, dt, u = TYPES[kind]
    b = Batch(1, [3, 1], [500, 40], 4, 16, False)
    cache = make_cache(kind, b.nb, 1, 16, D)
    rng = np.random.default_rng(0)
    key = (rng.uniform(0.5, 1, (1, 1, D)) * size).astype(np.float32)
    vals = []
    for r in range(2):
        T = b.ctx[r] + b.lens[r]
        vals.append(rng.normal(1, 1, (T, 1, D)).astype(np.float32))
        put(cache, b.slots(r, 0, T), np.repeat(key, T, 0), vals[r])
    q = torch.full((b.rows, 4, D), size, device=DEV).to(dt)
    q[:, 1] *= -1
    o = dv.alloc_attention_outputs(2, 4, b.rows, 4, cache, lse=True)
    dv.dspark_tree_attention(2, 4, q, b.rows, *b.args(), cache, D ** -0.5, o)
    torch.cuda.synchronize()
    assert o.attention_meta.tolist() == [4, 0]
    got, lse = f64(o.out), f64(o.lse)
    assert np.isfinite(lse[:4]).all()
    for r in range(2):
        v = get(cache, b.slots(r, 0, b.ctx[r] + b.lens[r]), "v")[:, 0]
        for j in range(b.lens[r]):
            n = b.ctx[r] + j + 1
            mean, size_v = v[:n].mean(0), np.abs(v[:n]).mean(0)
            within(got[b.cu[r] + j], np.broadcast_to(mean, (4, D)),
                   u * np.abs(mean) + (u + 2 * (n + 32) * W) * size_v, (r, j))


@pytest.mark.parametrize("kind,size", [("bf16", 3e4), ("f16", 9e3), ("e4m3", 3e4)])
def test_a_key_far_above_the_others_takes_everything(kind, size):
    """Scores that rise by thousands of their float32 steps from key to key: all of
    the weight is the last key's, whichever part of the keys holds it."""
    say(f"rising scores {kind}")
    code, dt, u = TYPES[kind]
    D, T = 64, 900
    b = Batch(1, [1], [T - 1], 1, 16, False)
    cache = make_cache(kind, b.nb, 1, 16, D)
    rng = np.random.default_rng(0)
    k = np.zeros((T, 1, D), np.float32)
    # element i holds a digit of the key's number: exact in every type
    for i in range(2):
        k[:, 0, i] = (np.arange(T) // 30 ** i % 30)
    v = rng.normal(0, 1, (T, 1, D)).astype(np.float32)
    if kind == "e4m3":
        k = np.minimum(k, 16)  # integers up to 16 are codes
    put(cache, b.slots(0, 0, T), k, v)
    q = torch.zeros(b.rows, 2, D, device=DEV, dtype=dt)
    q[:, :, 0] = size
    q[:, :, 1] = size
    o = dv.alloc_attention_outputs(1, 1, b.rows, 2, cache)
    for scale in (size, -size):
        dv.dspark_tree_attention(1, 1, q, b.rows, *b.args(), cache, scale, o)
        torch.cuda.synchronize()
        kk, vv = get(cache, b.slots(0, 0, T), "k")[:, 0], get(cache, b.slots(0, 0, T), "v")[:, 0]
        s = (kk[:, 0] + kk[:, 1]) * np.sign(scale)
        top = vv[s == s.max()]
        mean = top.mean(0)
        within(f64(o.out[0]), np.broadcast_to(mean, (2, D)),
               u * np.abs(mean) + (u + 2 * (len(top) + 32) * W) * np.abs(top).mean(0), scale)


@pytest.mark.parametrize("below", [12.0, 18.0, 22.0])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_the_tail_under_large_weights_counts(D, below):
    """One key in a hundred, whose value is zero, and keys of e^-below of its weight
    between them (every share of the keys has some of both): what the small ones
    add up to is the output. In float16 a weight is off by half of 2^-24 where the
    largest are 2^11 at least, so by 2^-36 of one of those, besides u, and the
    output by half of 2^-24 where it is small."""
    say(f"a long tail, e^-{below:g} each, D={D}")
    code, dt, u = TYPES["f16"]
    T, page, every = 20_000, 64, 100
    b = Batch(1, [1], [T - 1], 1, page, False)
    cache = make_cache("f16", b.nb, 1, page, D)
    rng = np.random.default_rng(0)
    k = np.zeros((T, 1, D), np.float32)
    k[:, 0, 0] = -below / 2
    k[::every, 0, 0] = 0
    v = rng.normal(1000, 500, (T, 1, D)).astype(np.float32)
    v[::every] = 0
    put(cache, b.slots(0, 0, T), k, v)
    q = torch.zeros(b.rows, 2, D, device=DEV, dtype=dt)
    q[:, :, 0] = 2
    o = dv.alloc_attention_outputs(1, 1, b.rows, 2, cache, lse=True)
    dv.dspark_tree_attention(1, 1, q, b.rows, *b.args(), cache, 1.0, o)
    torch.cuda.synchronize()
    kk, vv = (get(cache, b.slots(0, 0, T), n).transpose(1, 0, 2) for n in "kv")
    ref, rl, mean_abs, top = oracle.tree_attention(f64(q[:1]), kk, vv, T - 1, None, 1.0)
    t = (D + 16) * W * top[..., None] + 2 * W
    bound = (u * np.abs(ref) + (u + 2 * t + (T + 32) * W) * mean_abs +
             every * 2.0 ** -36 * np.abs(vv).max() + 2.0 ** -25)
    within(f64(o.out[:1]), ref, bound, "out")
    within(f64(o.lse[:1]), rl, t[..., 0] + (T + 32) * W + 4 * W * np.abs(rl), "lse")


# ------------------------------------------------------------------ bytes of a row that is not there

@pytest.mark.parametrize("D,hq", [(64, 4), (128, 4), (128, 32), (256, 4), (256, 32)])
def test_exponent_bytes_of_an_unseen_row_do_not_matter(D, hq):
    """A row of the step that append left out (its page holds whatever was there) has
    any codes and exponent bytes: the rows that do not see it keep their outputs to
    the bit."""
    say(f"any exponent byte in a sibling's row D={D} hq={hq}")
    b = Batch(3, [5, 1], [61, 30], 6, 16, True)
    b.parents[0, :4] = [0, 0, 1, 2]  # 0-1-3, 0-2-4
    cache = make_cache("e4m3", b.nb, 2, 16, D)
    rng = np.random.default_rng(1)
    for r in range(2):
        T = b.ctx[r] + b.lens[r]
        put(cache, b.slots(r, 0, T), *rng.normal(0, 1, (2, T, 2, D)).astype(np.float32))
    q = torch.from_numpy(rng.normal(0, 1, (b.rows, hq, D)).astype(np.float32)).bfloat16().to(DEV)
    o = dv.alloc_attention_outputs(2, 6, b.rows, hq, cache)
    args, par = b.args(), b.par()
    pg, of = b.slots(0, 62, 63)[0]  # row 1: rows 1 and 3 see it
    want = None
    for byte in (120, 0, 246, 247, 254, 255):
        for t in (cache.k_scale, cache.v_scale):
            t[pg, :, of] = byte
        o.out.fill_(-7)
        dv.dspark_tree_attention(2, 6, q, b.rows, *args, cache, 0.1, o, tree_parents=par)
        torch.cuda.synchronize()
        got = o.out[[0, 2, 4, 5]].clone()
        want = got if want is None else want
        assert torch.isfinite(got.float()).all() and torch.equal(got, want), byte


# ------------------------------------------------------------------ large reads

@pytest.mark.parametrize("rows", [8 * 2 ** 20 + 777, 8 * 2 ** 23 + 4096])
def test_read_of_more_rows_than_a_launch_holds(rows):
    """8.4 and 67 million rows, the latter with more than 2^32 threads' work (137 GB
    of outputs): the first and the last rows, and those around every 2^23, are
    those of the cache."""
    say(f"read of {rows} rows")
    hkv, D, page = 2, 256, 256
    if torch.cuda.mem_get_info()[0] < 2.2 * rows * hkv * D * 2:
        pytest.skip("needs more memory")
    cache = dv.alloc_kv_cache(5, hkv, page, D, dv.BF16, DEV)
    cache.k.normal_()
    cache.v.normal_()
    ids = (torch.arange(rows // page + 1, device=DEV, dtype=torch.int32) * 3 % 5).view(1, -1)
    rd = dv.alloc_kv_read_outputs(rows + 100, cache)
    spans = [(0, 4096), (rows - 8192, rows)]
    spans += [(x - 2048, x + 2048) for x in range(2 ** 23, rows - 2048, 2 ** 23)]
    for t in rd[:2]:
        t[rows:] = -7
        for lo, hi in spans:
            t[lo:hi] = -7
    dv.dspark_kv_read(1, rows + 100, i32([0, rows]), i32([0]), ids, cache, rd)
    torch.cuda.synchronize()
    assert rd.read_meta.tolist() == [rows, 0]
    for t, pool in ((rd.k_out, cache.k), (rd.v_out, cache.v)):
        assert bool((t[rows:] == -7).all())
        for lo, hi in spans:
            i = torch.arange(lo, hi, device=DEV)
            assert torch.equal(t[lo:hi], pool[i // page * 3 % 5, :, i % page]), lo
    del rd
    torch.cuda.empty_cache()


def test_read_into_buffers_of_any_number_of_rows():
    """The launch does not grow with the rows that the buffers are said to hold."""
    say("read with max_rows 2^31 - 1")
    b, cache, rows = filled(6)
    total = int(b.cu[-1])
    rd = dv.alloc_kv_read_outputs(b.rows, cache)
    for t in rd[:2]:
        t.fill_(-7)
    cu, pre, table = b.args()
    for most in (80_000_000, 2 ** 31 - 1):
        st = dv._lib.lib().dspark_kv_read(
            b.B, most, cu.data_ptr(), pre.data_ptr(), table.data_ptr(), b.width, cache._ref,
            rd.k_out.data_ptr(), rd.v_out.data_ptr(), 64, rd.read_meta.data_ptr(),
            torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert st == dv._lib.OK
        assert rd.read_meta.tolist() == [total, 0]
        for t in rd[:2]:
            assert torch.equal(t[:total], rows[:total]) and bool((t[total:] == -7).all())


# ------------------------------------------------------------------ views of a pool

@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_caches_whose_dimensions_of_one_have_any_stride(kind):
    """One head stored as [page][1][dim], and a single page cut from two pools of
    different page strides: the strides of dimensions of one do not matter."""
    say(f"cache views {kind}")
    D, page = 64, 16
    el = torch.float8_e4m3fn if kind == "e4m3" else torch.bfloat16
    e8 = kind == "e4m3"

    def pool(*shape, dtype=el):
        return torch.zeros(shape, device=DEV).to(dtype)

    token_major = [pool(3, page, 1, D).transpose(1, 2) for _ in range(2)]
    scales = [pool(3, page, 1, dtype=torch.uint8).transpose(1, 2) for _ in range(2)] if e8 else []
    one_page = [pool(4, 2, 1, page, D)[1:2, 0], pool(4, 1, page, D)[2:3]]
    one_scale = [pool(4, 2, 1, page, dtype=torch.uint8)[1:2, 0],
                 pool(4, 1, page, dtype=torch.uint8)[2:3]] if e8 else []
    one_layer = [pool(2, 5, 1, page, D)[:1], pool(1, 5, 1, page, D)]
    layer_scale = [pool(2, 5, 1, page, dtype=torch.uint8)[:1],
                   pool(1, 5, 1, page, dtype=torch.uint8)] if e8 else []
    x = torch.randn(5, 1, D, device=DEV).bfloat16()
    if e8:
        x = x.to(el).to(torch.bfloat16)  # codes: exact in 8 bits under an exponent of 0
        x[:, :, 0] = 448
    for k_v, sc in ((token_major, scales), (one_page, one_scale), (one_layer, layer_scale)):
        cache = dv.KvCache(*k_v, *sc)
        lay = cache.layer(0) if k_v[0].dim() == 5 else cache
        ap = dv.alloc_append_outputs(5, 1, lay)
        rd = dv.alloc_kv_read_outputs(5, lay)
        args = i32([0, 5]), i32([3]), i32([[0]])
        dv.dspark_kv_append(1, 4, x, x, x, 5, *args, lay, ap)
        dv.dspark_kv_read(1, 5, *args, lay, rd)
        cm = torch.empty(2, dtype=torch.int32, device=DEV)
        dv.dspark_kv_commit(1, 4, i32([[0, 2, 4, -1, -1]]), i32([2]), i32([3]), i32([[0]]), cache, cm)
        torch.cuda.synchronize()
        assert ap.append_meta.tolist() == rd.read_meta.tolist() == [5, 0] and cm.tolist() == [2, 0]
        assert torch.equal(rd.k_out, x) and torch.equal(rd.v_out, x)
        for t in k_v:
            t = t[0] if t.dim() == 5 else t
            assert torch.equal(t[0, 0, 3:8].float(), x[[0, 2, 4, 3, 4], 0].float())
    # what is not dense is refused as before
    with pytest.raises(ValueError, match="dense"):
        dv.KvCache(*[pool(3, page, 2, D).transpose(1, 2) for _ in range(2)],
                   *[pool(3, 2, page, dtype=torch.uint8) for _ in sc])
    with pytest.raises(ValueError, match="strides"):
        dv.KvCache(pool(4, 2, 1, page, D)[:, 0], pool(4, 1, page, D),
                   *[pool(4, 1, page, dtype=torch.uint8) for _ in sc])


# ------------------------------------------------------------------ workspace

@pytest.mark.parametrize("kind,gamma,hq,hkv,D", [
    ("bf16", 3, 4, 2, 64), ("e4m3", 3, 4, 2, 128), ("f16", 31, 16, 2, 128), ("e4m3", 31, 16, 2, 256),
    ("bf16", 3, 4, 1, 256)])
def test_attention_keeps_to_its_workspace(kind, gamma, hq, hkv, D):
    """Contexts that every workgroup has a part of, in a workspace of just the size
    asked for: the bytes behind it stay, the rows are right."""
    say(f"workspace {kind} gamma={gamma} hq={hq} hkv={hkv} D={D}")
    _, dt, u = TYPES[kind]
    b = Batch(1, [gamma + 1, 2], [30_000, 9_000], gamma, 64, False)
    cache = make_cache(kind, b.nb, hkv, 64, D)
    torch.manual_seed(0)
    for t in (cache.k, cache.v):
        t.copy_(torch.randn(t.shape, device=DEV).to(t.dtype))
    if kind == "e4m3":
        cache.k_scale.fill_(127)
        cache.v_scale.fill_(127)
    q = torch.randn(b.rows, hq, D, device=DEV).to(dt)
    o = dv.alloc_attention_outputs(b.B, gamma, b.rows, hq, cache)
    size = dv.dspark_tree_attention_workspace_size(b.B, gamma, hq, hkv, D)
    buf = torch.full((size + 2 ** 20,), 0xA5, dtype=torch.uint8, device=DEV)
    o = o._replace(workspace=buf[:size])
    dv.dspark_tree_attention(b.B, gamma, q, b.rows, *b.args(), cache, D ** -0.5, o)
    torch.cuda.synchronize()
    assert o.attention_meta.tolist() == [int(b.cu[-1]), 0]
    assert bool((buf[size:] == 0xA5).all())
    for r in range(2):
        T = b.ctx[r] + b.lens[r]
        pages = torch.tensor(b.table[r][:-(-T // 64)].tolist(), device=DEV)
        k, v = (t[pages].to(torch.float32).transpose(0, 1).reshape(hkv, -1, D)[:, :T]
                .repeat_interleave(hq // hkv, 0) for t in (cache.k, cache.v))
        c0, c1 = int(b.cu[r]), int(b.cu[r + 1])
        ref, mean_abs, top = ref_long(q[c0:c1], k, v, b.ctx[r], D ** -0.5)
        t = (D + 16) * W * top[..., None] + 2 * W
        bound = u * np.abs(ref) + (u + 2 * t + (T + 32) * W) * mean_abs
        if kind == "f16":
            bound = bound + T * 2.0 ** -36 * float(v.abs().max()) + 2.0 ** -25
        within(f64(o.out[c0:c1]), ref, bound, f"request {r}")


# ------------------------------------------------------------------ every kernel of the attention

@pytest.mark.parametrize("kind,lens,ctx,gamma,hq,hkv,D,page,tree,joint", [
    # eight waves at heads of 256, 8 and 16 bits: a wave's share of a tile is two copies
    ("e4m3", [17, 3, 17], [63, 5, 400], 16, 10, 2, 256, 32, True, False),
    ("e4m3", [65, 1, 33], [1000, 2000, 0], 64, 16, 2, 256, 16, True, True),
    ("e4m3", [17], [9000], 16, 8, 1, 256, 256, False, False),
    ("f16", [17, 3, 17], [63, 5, 400], 16, 10, 2, 256, 32, True, False),
    ("f16", [65, 20], [5000, 31], 64, 8, 4, 256, 64, True, True),
    # 8 bits in batches beyond a wave's lanes, few rows and many, each head size
    ("e4m3", [3] * 90, [7 * i for i in range(90)], 2, 8, 2, 128, 16, True, False),
    ("e4m3", [1 + i % 17 for i in range(70)], [11 * i for i in range(70)], 16, 16, 2, 128, 32, True, True),
    ("e4m3", [1 + i % 5 for i in range(300)], [i % 97 for i in range(300)], 4, 3, 1, 64, 16, True, False),
    ("e4m3", [2] * 65, [301] * 65, 1, 4, 2, 256, 64, False, False),
    ("e4m3", [1 + i % 33 for i in range(66)], [200 - i for i in range(66)], 32, 4, 1, 256, 16, True, False),
])
def test_attention_kernels(kind, lens, ctx, gamma, hq, hkv, D, page, tree, joint):
    say(f"attention {kind} B={len(lens)} lens={lens[:4]} hq={hq} hkv={hkv} D={D}")
    b = Batch(len(lens) + D, lens, ctx, gamma, page, tree)
    attention_check(b, kind, hq, hkv, D, D ** -0.5, seed=D, joint=joint, repeat=2)


@pytest.mark.parametrize("kind", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_rows_ignore_what_they_do_not_see(kind, D):
    """A tree of 33 rows, eight query heads to each of two key/value heads (more than
    64 rows to a head): NaN and infinities of two siblings' rows, in keys, in
    values, in both, reach the rows that see them and no other."""
    say(f"non-finite rows of a large tree {kind} D={D}")
    _, dt, u = TYPES[kind]
    n, hq, hkv, page = 33, 16, 2, 16
    b = Batch(3, [n, 2], [61, 30], n - 1, page, True)
    rng = b.rng
    cache = make_cache(kind, b.nb, hkv, page, D)
    T = b.ctx[0] + n
    paths = oracle.tree_paths(b.parents[0], n)
    k, v = rng.normal(0, 1, (2, T, hkv, D)).astype(np.float32)
    inf = np.nan if kind == "e4m3" else np.inf
    leaves = [j for j in range(1, n) if j not in set(b.parents[0, :n - 1].tolist())]
    k[61 + leaves[0], 0, 3] = np.nan
    v[61 + leaves[1], 1, D - 1] = inf
    v[61 + 5, :, 0] = np.nan
    v[61 + 5, :, D // 2] = inf
    put(cache, b.slots(0, 0, T), k, v)
    put(cache, b.slots(1, 0, 32), *rng.normal(0, 1, (2, 32, hkv, D)).astype(np.float32))
    q = torch.from_numpy(rng.normal(0, 1, (b.rows, hq, D)).astype(np.float32)).to(dt).to(DEV)
    o = dv.alloc_attention_outputs(2, n - 1, b.rows, hq, cache)
    dv.dspark_tree_attention(2, n - 1, q, b.rows, *b.args(), cache, 0.1, o, tree_parents=b.par())
    torch.cuda.synchronize()
    assert o.attention_meta.tolist() == [n + 2, 0]
    got = o.out[:n + 2].float().cpu().numpy()
    for j in range(n):
        bad = np.zeros((hq, D), bool)
        if leaves[0] in paths[j]:
            bad[:8] = True  # a NaN score: the whole row of that head's queries
        if leaves[1] in paths[j]:
            bad[8:, D - 1] = True
        if 5 in paths[j]:
            bad[:, [0, D // 2]] = True
        assert np.array_equal(~np.isfinite(got[j]), bad), j
    assert np.isfinite(got[n:]).all()


# ------------------------------------------------------------------ lengths out of order

@pytest.mark.parametrize("B", [6, 80])
def test_attention_and_append_beside_lengths_out_of_order(B):
    """A word out of place leaves out the two requests that it bounds, or makes them
    others; every request that it does not touch has the rows that it has without."""
    say(f"attention and append beside malformed lengths B={B}")
    b, cache, rows = filled(B)
    rng = np.random.default_rng(B)
    for r in range(B):
        put(cache, b.slots(r, 0, b.ctx[r] + b.lens[r]),
            *rng.normal(0, 1, (2, b.ctx[r] + b.lens[r], 1, 64)).astype(np.float32))
    q = torch.randn(b.rows, 2, 64, device=DEV).bfloat16()
    o = dv.alloc_attention_outputs(B, 4, b.rows, 2, cache)
    dv.dspark_tree_attention(B, 4, q, b.rows, *b.args(), cache, 0.125, o)
    torch.cuda.synchronize()
    want, total, at = o.out.clone(), int(b.cu[-1]), B // 2
    # the shares of the keys differ: each side is within 2.1 u mean |v|, and |v| < 5
    tol = 2 * 2.1 * 2.0 ** -8 * 5
    other = make_cache("bf16", b.nb, 1, 16, 64)
    for value in (10 ** 6, -5, total, 0):
        cu = b.cu.copy()
        cu[at] = value
        o.out.fill_(-7)
        dv.dspark_tree_attention(B, 4, q, b.rows, i32(cu), i32(b.ctx), i32(b.table), cache, 0.125, o)
        ap = dv.alloc_append_outputs(b.rows, 1, other)
        ap.q_out.fill_(-7)
        dv.dspark_kv_append(B, 4, rows, rows, rows, b.rows, i32(cu), i32(b.ctx), i32(b.table), other, ap)
        torch.cuda.synchronize()
        for meta in (o.attention_meta, ap.append_meta):
            assert meta.tolist() == [total, oracle.DATA_BAD_LENS], value
        taken = set()  # rows of the request that the word makes out of others'
        for r in (at - 1, at):
            s, e = int(cu[r]), int(cu[r + 1])
            if 0 <= s < e <= total and e - s <= 5:
                taken |= set(range(s, e))
        for r in range(B):
            c = range(int(b.cu[r]), int(b.cu[r + 1]))
            if taken & set(c):
                continue
            c = slice(c.start, c.stop)
            if r in (at - 1, at):
                assert bool((o.out[c] == -7).all()) and bool((ap.q_out[c] == -7).all())
            else:
                assert float((o.out[c].float() - want[c].float()).abs().max()) <= tol
                assert torch.equal(ap.q_out[c], rows[c])
