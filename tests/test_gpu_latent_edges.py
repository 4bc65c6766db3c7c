"""GPU tests of the latent cache's calls where they change their way of working:
exponents far apart in a tile, large batches of many heads, row tiles past what
their plan sorts, workspaces with neighbours. Tolerances as in test_gpu_latent.py."""

import numpy as np
import pytest
import torch

import dspark_verify_scheduling_amd as dv
from _gpu import DEV, say, up
from test_gpu_latent import (R, latent_check, latent_run, latent_setup, lput, make_latent, prefill_check,
                             prefill_run, turns, typed)
from test_gpu_target import TYPES, Batch, bits, f64, i32, make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu(hip):
    return hip


@pytest.mark.parametrize("L", [512, 256])
@pytest.mark.parametrize("where", ["draft", "cache", "everywhere"])
def test_exponents_far_apart_in_a_tile(L, where):
    """In 8 bits a tile's exponents differ by up to 219: a key that a row does not see,
    or whose weight is nothing, takes nothing from the others' bits."""
    say(f"latent attention far exponents L={L} {where}")
    H, gamma = 6, 9
    b = Batch(4, [10, 3], [170, 64], gamma, 16, True)
    b.parents[0] = [0, 1, 0, 3, 3, 2, 6, 0, 8]
    dt = TYPES["e4m3"][1]
    rng = np.random.default_rng(3)
    cache = make_latent("e4m3", b.nb, 16, L)
    ql = typed(rng, (b.rows, H, L), dt).to(DEV)
    qr = typed(rng, (b.rows, H, R), dt).to(DEV)
    # the columns with the exponents take no part in the scores
    ql[..., 128:256] = 0
    qr[..., 0] = 1.0
    for r in range(2):
        T = b.ctx[r] + b.lens[r]
        lat, rope = rng.normal(0, 1, (T, L)), rng.normal(0, 1, (T, R))
        size = np.full(T, -85.0)
        rope[:, 0] = 0
        if where == "draft":
            size[b.ctx[r] + 2] = 108  # seen by its descendants only
        elif where == "cache":
            size[[5, 40, 63]] = [60, 105, 20]  # in whole tiles
            rope[[5, 40, 63], 0] = -4000.0     # weights of 2^-288
        else:
            size = rng.integers(-85, 109, T).astype(np.float64)
        lat[:, 128:256] *= 2.0 ** size[:, None]
        lput(cache, b.slots(r, 0, T), lat, rope)
    o = dv.alloc_latent_attention_outputs(b.B, gamma, b.rows, H, cache, lse=True)
    o.out.fill_(-7)
    o.lse.fill_(-7)
    dv.dspark_latent_attention(b.B, gamma, ql, qr, b.rows, *b.args(), cache, 0.05, o,
                               tree_parents=b.par())
    torch.cuda.synchronize()
    assert o.attention_meta.tolist() == [13, 0]
    latent_check(b, "e4m3", H, L, 0.05, cache, ql, qr, o)


@pytest.mark.parametrize("kind,H,L", [("bf16", 128, 512), ("f16", 65, 256), ("e4m3", 33, 512)])
def test_latent_attention_of_large_batches_and_many_heads(kind, H, L):
    """More requests than a wave has lanes, several segments each."""
    say(f"latent attention of 70 requests, {H} heads {kind}")
    rng = np.random.default_rng(H)
    lens = rng.integers(1, 6, 70).tolist()
    ctx = rng.integers(0, 200, 70).tolist()
    lens[3], ctx[3] = 5, 2500
    latent_run(Batch(H, lens, ctx, 4, 16, True), kind, H, L, 0.05)


def test_latent_attention_of_a_whole_tree_at_all_heads():
    say("latent attention, 65 rows of 128 heads")
    latent_run(Batch(5, [65, 1], [300, 900], 64, 64, True), "bf16", 128, 512, 0.05)


@pytest.mark.parametrize("kind,L,H,B,ctx", [("bf16", 512, 7, 3, 900), ("e4m3", 256, 40, 2, 2100),
                                            ("f16", 256, 3, 66, 70)])
def test_latent_attention_keeps_to_its_workspace(kind, L, H, B, ctx):
    say(f"latent attention workspace {kind}")
    b = Batch(B, [3] * B, [ctx] * B, 4, 16, False)
    cache, ql, qr = latent_setup(b, kind, H, L)
    o = dv.alloc_latent_attention_outputs(B, 4, b.rows, H, cache, lse=True)
    size = o.workspace.numel() * o.workspace.element_size()
    room = torch.full((size + 8192,), 0x5A, dtype=torch.uint8, device=DEV)
    o = o._replace(workspace=room[4096:4096 + size])
    o.out.fill_(-7)
    o.lse.fill_(-7)
    dv.dspark_latent_attention(B, 4, ql, qr, b.rows, *b.args(), cache, 0.05, o)
    torch.cuda.synchronize()
    latent_check(b, kind, H, L, 0.05, cache, ql, qr, o)
    assert bool((room[:4096] == 0x5A).all()) and bool((room[4096 + size:] == 0x5A).all())


@pytest.mark.parametrize("kind,n,H,lens", [("bf16", 128, 8, [130, 0, 31]), ("e4m3", 64, 3, [1, 300]),
                                           ("f16", 64, 16, [5] * 40)])
def test_latent_prefill_keeps_to_its_workspace(kind, n, H, lens):
    say(f"latent prefill workspace {kind}")
    b = Batch(7, lens, [40] * len(lens), 1, 16, False)
    cache, q, wk, wv, o, keys = prefill_run(b, kind, H, n, 256, 0.07, check=False)
    size = o.workspace.numel() * o.workspace.element_size()
    room = torch.full((size + 8192,), 0x5A, dtype=torch.uint8, device=DEV)
    o = o._replace(workspace=room[4096:4096 + size])
    o.out.fill_(-7)
    o.lse.fill_(-7)
    dv.dspark_latent_prefill(b.B, q, wk, wv, b.rows, keys, *b.args(), cache, 0.07, o)
    torch.cuda.synchronize()
    prefill_check(b, kind, H, n, 256, 0.07, cache, q, wk, wv, o)
    assert bool((room[:4096] == 0x5A).all()) and bool((room[4096 + size:] == 0x5A).all())


def test_latent_prefill_of_more_tiles_than_are_sorted():
    say("latent prefill of 1100 requests")
    rng = np.random.default_rng(8)
    lens, ctx = rng.integers(1, 4, 1100).tolist(), rng.integers(0, 20, 1100).tolist()
    lens[700] = 260
    prefill_run(Batch(4, lens, ctx, 1, 16, False), "bf16", 8, 64, 256, 0.07)


@pytest.mark.parametrize("kind,scale", [("bf16", 400.0), ("f16", -300.0), ("e4m3", 300.0)])
def test_latent_prefill_large_scores(kind, scale):
    """Scores of some thousands: a row's largest takes everything, its value comes out."""
    say(f"latent prefill scale {scale} {kind}")
    L, n, H, T = 256, 64, 2, 150
    b = Batch(3, [T], [0], 1, 16, False)
    dt = TYPES[kind][1]
    cache = make_latent(kind, b.nb, 16, L)
    rng = np.random.default_rng(1)
    lat = rng.integers(-3, 4, (T, L)).astype(np.float64)
    lat[:, 0] = rng.permutation(T) / 2  # key and score of a row, exact in every type
    rope = np.zeros((T, R))
    if kind == "e4m3":
        lat[:, 0] = np.clip(np.arange(T) // 10, 0, 15)
        lat[:, 0] += np.arange(T) / 10 % 1 >= 0.9
        rope[:, 0] = np.arange(T)
    lput(cache, b.slots(0, 0, T), lat, rope)
    q = torch.zeros(b.rows, H, n + R, dtype=dt, device=DEV)
    q[:, 0, 0], q[:, 1, 0] = 1.0, -1.0
    if kind == "e4m3":
        q[:, 0, 0] = q[:, 1, 0] = 0
        q[:, 0, n], q[:, 1, n] = 1.0, -1.0
    w = torch.zeros(H, 2 * n, L, dtype=dt, device=DEV)
    w[:, 0, 0] = 1.0
    for c in range(n):
        w[:, n + c, c] = 1.0
    o = dv.alloc_latent_prefill_outputs(1, b.rows, T, H, n, cache)
    dv.dspark_latent_prefill(1, q, w[:, :n], w[:, n:], b.rows, T, *b.args(), cache, scale, o)
    torch.cuda.synchronize()
    got = f64(o.out).reshape(b.rows, H, n)
    key = rope[:, 0] if kind == "e4m3" else lat[:, 0]
    for row in range(T):
        for h in range(H):
            s = scale * (1 if h == 0 else -1) * key[:row + 1]
            assert np.array_equal(got[row, h], lat[s.argmax(), :n]), (row, h)


def test_axes_rows_of_a_wave_and_of_a_workgroup_agree():
    """A call of many rows gives a wave to each, one of few a workgroup: the same bits."""
    say("append with axes, 1500 rows at once and in parts")
    hq, hkv, D, page, cut = 6, 3, 128, 16, 700
    rng = np.random.default_rng(2)
    dt = torch.bfloat16
    rows = 1500
    qkv = typed(rng, (rows, hq + 2 * hkv, D), dt).to(DEV)
    w = typed(rng, (2, D), dt).to(DEV)
    rope = up(turns(512, D))
    pos = i32(rng.integers(0, 512, (3, rows)))
    nb = -(-rows // page)
    table = i32(rng.permutation(nb)[None])
    axis = [i % 3 for i in range(D // 2)]
    for kind in ("bf16", "e4m3"):
        out = []
        for parts in ([(0, rows)], [(0, cut), (cut, rows)]):
            cache = make_cache(kind, nb, hkv, page, D)
            for p in (cache.k, cache.v):
                bits(p).zero_()
            got = []
            for lo, hi in parts:
                n = hi - lo
                x = qkv[lo:hi]
                o = dv.alloc_append_outputs(n, hq, cache)
                dv.dspark_kv_append_axes(1, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], n,
                                         i32([0, n]), i32([lo]), pos[:, lo:hi], axis, table, cache, o,
                                         rope, q_weight=w[0], k_weight=w[1])
                torch.cuda.synchronize()
                assert o.append_meta.tolist() == [n, 0]
                got.append(o.q_out.clone())
            out.append([bits(torch.cat(got)), bits(cache.k).clone(), bits(cache.v).clone()])
        for x, y in zip(*out):
            assert torch.equal(x, y)


@pytest.mark.parametrize("kind,L", [("bf16", 512), ("e4m3", 256)])
def test_layers_and_strided_rows(kind, L):
    """A layer of a pool of all layers' pages, queries and outputs that are parts of wider
    rows: the results of a cache and rows of their own, and nothing beside them."""
    say(f"latent layers and strides {kind}")
    H, n, layers = 6, 64, 3
    b = Batch(11, [4, 1, 5], [100, 0, 37], 4, 16, True)
    plain, ql, qr = latent_setup(b, kind, H, L)
    dt = ql.dtype
    pool = make_latent(kind, b.nb, 16, L, layers, joint=True)
    cache = pool.layer(1)
    for name in ("latent", "rope", "scale"):
        if getattr(plain, name) is not None:
            getattr(cache, name).copy_(getattr(plain, name))
    q = typed(np.random.default_rng(5), (b.rows, H, n + R), dt).to(DEV)
    w = typed(np.random.default_rng(6), (H, 2 * n, L), dt, L ** -0.5).to(DEV)
    keys = sum(b.ctx) + sum(b.lens)
    got = []
    for c, wide in ((plain, 0), (cache, 16)):
        a = dv.alloc_latent_attention_outputs(b.B, 4, b.rows, H, c, lse=True)
        p = dv.alloc_latent_prefill_outputs(b.B, b.rows, keys, H, n, c, lse=True)
        rows_of, rest = [], []
        for x in (ql, q):
            room = torch.full((b.rows, x.shape[1] * x.shape[2] + wide), 3.0, dtype=dt, device=DEV)
            room[:, :x.shape[1] * x.shape[2]] = x.flatten(1)
            rows_of.append(room[:, :x.shape[1] * x.shape[2]].unflatten(1, x.shape[1:]))
        for o, dim in ((a, L), (p, n)):
            room = torch.full((b.rows, H * dim + wide), -7.0, dtype=dt, device=DEV)
            rest.append(room)
        a = a._replace(out=rest[0][:, :H * L].unflatten(1, (H, L)))
        p = p._replace(out=rest[1][:, :H * n].unflatten(1, (H, n)))
        dv.dspark_latent_attention(b.B, 4, rows_of[0], qr, b.rows, *b.args(), c, 0.05, a,
                                   tree_parents=b.par())
        dv.dspark_latent_prefill(b.B, rows_of[1], w[:, :n], w[:, n:], b.rows, keys, *b.args(), c, 0.07, p)
        torch.cuda.synchronize()
        total = int(b.cu[-1])
        got.append([a.out[:total].clone(), a.lse[:total].clone(), p.out[:total].clone(),
                    p.lse[:total].clone()])
        for room, dim in zip(rest, (L, n)):
            assert bool((room[total:] == -7).all()) and bool((room[:, H * dim:] == -7).all())
    for x, y in zip(*got):
        assert torch.equal(x, y)


@pytest.mark.parametrize("kind", ["f16", "e4m3"])
def test_a_graph_of_a_step_takes_other_batches(kind):
    """Captured for the largest batch, replayed with other lengths, contexts, trees and
    paths in place: the eager results."""
    say(f"latent graph, other batches {kind}")
    H, n, L, gamma, B, page = 5, 64, 256, 5, 3, 16
    dt = TYPES[kind][1]
    batches = [Batch(s, lens, ctx, gamma, page, True, pad=30 - sum(lens)) for s, lens, ctx in (
        (1, [6, 6, 6], [700, 90, 15]), (2, [1, 1, 1], [0, 800, 63]), (3, [2, 6, 3], [64, 5, 330]))]
    nb, width = max(b.nb for b in batches), max(b.width for b in batches)
    cache = make_latent(kind, nb, page, L)
    rng = np.random.default_rng(7)
    for pg in range(nb):
        lput(cache, [(pg, i) for i in range(page)], rng.normal(0, 1, (page, L)), rng.normal(0, 1, (page, R)))
    keys = 900 + 3 * (gamma + 1)
    ql, qr = (typed(rng, (30, H, d), dt).to(DEV) for d in (L, R))
    q = typed(rng, (30, H, n + R), dt).to(DEV)
    w = typed(rng, (H, 2 * n, L), dt, L ** -0.5).to(DEV)
    cu, pre = torch.zeros(B + 1, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
    table = torch.zeros(B, width, dtype=torch.int32, device=DEV)
    par = torch.zeros(B, gamma, dtype=torch.int32, device=DEV)
    path, num = torch.zeros(B, gamma + 1, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
    meta = torch.empty(2, dtype=torch.int32, device=DEV)
    a = dv.alloc_latent_attention_outputs(B, gamma, 30, H, cache, lse=True)
    p = dv.alloc_latent_prefill_outputs(B, 30, keys, H, n, cache, lse=True)

    def fill(b):
        cu.copy_(i32(b.cu))
        pre.copy_(i32(b.ctx))
        table.fill_(-1)
        table[:, :b.width] = i32(b.table)
        par.copy_(i32(b.parents))
        r = np.random.default_rng(b.rows)
        steps = np.zeros((B, gamma + 1), np.int32)
        count = [int(r.integers(0, n)) for n in b.lens]
        for i, c in enumerate(count):
            steps[i, 1:c + 1] = np.sort(r.choice(np.arange(1, b.lens[i]), c, replace=False))
        path.copy_(i32(steps))
        num.copy_(i32(count))

    def step():
        dv.dspark_latent_attention(B, gamma, ql, qr, 30, cu, pre, table, cache, 0.05, a, tree_parents=par)
        dv.dspark_latent_prefill(B, q, w[:, :n], w[:, n:], 30, keys, cu, pre, table, cache, 0.07, p)
        dv.dspark_latent_commit(B, gamma, path, num, pre, table, cache, meta)

    pools = [bits(cache.latent), cache.rope] + ([cache.scale] if kind == "e4m3" else [])
    metas = [a.attention_meta, p.attention_meta, meta]
    outs = [a.out, a.lse, p.out, p.lse] + pools + metas
    start = [t.clone() for t in pools]

    def reset():
        for t in outs[:4]:
            t.fill_(-7)
        for t, y in zip(pools, start):
            t.copy_(y)

    fill(batches[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for turn in range(6):
        b = batches[turn % 3]
        fill(b)
        reset()
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in outs]
        assert all(t[1].item() == 0 for t in metas)
        reset()
        graph.replay()
        torch.cuda.synchronize()
        for k, (t, y) in enumerate(zip(outs, want)):
            assert torch.equal(t.view(torch.uint8), y.view(torch.uint8)), (turn, k)
        torch.randn(1 << 18, device=DEV).sum().item()


def test_expanded_attention_on_two_streams():
    say("latent prefill two streams")
    one = prefill_run(Batch(3, [300, 20], [100, 7], 1, 16, False), "bf16", 8, 128, 512, 0.07, 1)
    two = prefill_run(Batch(4, [40, 260], [900, 3], 1, 64, False), "bf16", 8, 128, 512, 0.07, 2)
    sets = []
    for (cache, q, wk, wv, o, keys), b in ((one, Batch(3, [300, 20], [100, 7], 1, 16, False)),
                                           (two, Batch(4, [40, 260], [900, 3], 1, 64, False))):
        sets.append((b, b.args(), cache, q, wk, wv, keys, o.out.clone(),
                     dv.alloc_latent_prefill_outputs(b.B, b.rows, keys, 8, 128, cache)))
        sets[-1][-1].out.fill_(-7)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (b, args, cache, q, wk, wv, keys, want, o) in zip(streams, sets):
            dv.dspark_latent_prefill(b.B, q, wk, wv, b.rows, keys, *args, cache, 0.07, o, stream=s)
    torch.cuda.synchronize()
    for b, args, cache, q, wk, wv, keys, want, o in sets:
        assert torch.equal(o.out, want)
