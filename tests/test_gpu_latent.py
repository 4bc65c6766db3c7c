"""GPU tests of the target pass over a latent cache (append, read, commit, both
forms of attention) and of the append with positions on several axes, through
the C ABI, against the float64 oracle.

Tolerances, with u the half step of the output type (2^-8 bfloat16, 2^-11
float16, relative to the value) and w = 2^-24 that of float32, as in
test_gpu_target.py:

* Whole numbers, moved bytes, values that no arithmetic precedes: equal.
* Rows with norm and rotation: u |y|, and for float32 (n + 16) w (|a| + |b|) with
  n the elements of the norm and a, b the pair's. In 8 bits half a step of the
  value, 2^-4 |y| or 2^-10 of the group's power of two, instead of u |y|.
* Absorbed attention over n keys: scores of m = latent_dim + 64 terms err by t =
  (m + 16) w scale sum |q||k|, weights round to the query type (u relative, 2^-25
  absolute in float16 against a sum of at least 1), float32 sums of n terms by n w,
  the output rounds once: u |out| + (u + 2 t + (n + 32) w) sum w_k |v_k| + n 2^-25
  max |v| (float16).
* Expanded attention: a key's element rounds once (u) after a float32 sum of L
  terms ((L + 16) w of the magnitudes), and so does a value's. t grows by scale
  (u sum |q||k| + (L + 16) w sum |q| sum |W||c|), and the output's bound by u sum w_k
  |v_k| + (L + 16) w sum w_k sum |W||c|. A float16 below 2^-14 rounds by up to 2^-25.
"""

import numpy as np
import pytest
import torch

import dspark_verify_scheduling_amd as dv
import oracle
from _gpu import DEV, say, up
from test_gpu_target import TYPES, W, Batch, bits, f64, get, i32, make_cache, within

pytestmark = pytest.mark.gpu
R = 64


@pytest.fixture(scope="module", autouse=True)
def _need_gpu(hip):
    return hip


def make_latent(kind, nb, page, L, layers=0, joint=False):
    """A cache whose every slot holds NaN; `joint`: latents and rotated parts of a
    page side by side in one pool."""
    code, dt, _ = TYPES[kind]
    e8 = kind == "e4m3"
    if joint:
        lead = (layers,) if layers else ()
        row = L // 2 if e8 else L
        pool = torch.empty(lead + (nb, page * (row + R)), dtype=dt, device=DEV)
        lat = pool[..., :page * row]
        lat = (lat.view(torch.float8_e4m3fn) if e8 else lat).unflatten(-1, (page, L))
        sc = torch.empty(lead + (nb, 2, page, L // 128), dtype=torch.uint8, device=DEV) if e8 else None
        c = dv.LatentCache(lat, pool[..., page * row:].unflatten(-1, (page, R)),
                           sc[..., 0, :, :] if e8 else None)
    else:
        c = dv.alloc_latent_cache(nb, page, L, code, DEV, layers)
    c.rope.fill_(float("nan"))
    if e8:
        c.latent.view(torch.uint8).fill_(0x7F)
        c.scale.fill_(120)
    else:
        c.latent.fill_(float("nan"))
    return c


def at(slots):
    return (torch.tensor([s[0] for s in slots], device=DEV),
            torch.tensor([s[1] for s in slots], device=DEV))


def lput(cache, slots, lat, rope, layer=None):
    """Host rows lat [n, L], rope [n, 64] into (page, offset) slots."""
    pg, of = at(slots)
    pools = [cache.latent, cache.rope, cache.scale]
    if layer is not None:
        pools = [None if p is None else p[layer] for p in pools]
    if cache.scale is not None:
        y = np.asarray(lat, np.float64).reshape(len(slots), -1, 128)
        e = oracle.e4m3_exponent(y)
        codes = np.ldexp(oracle.e4m3_round(y, e), -e[..., None]).reshape(lat.shape)
        codes = torch.from_numpy(codes).to(torch.float8_e4m3fn).view(torch.uint8).to(DEV)
        pools[0].view(torch.uint8)[pg, of] = codes
        pools[2][pg, of] = torch.from_numpy((e + 127).astype(np.uint8)).to(DEV)
    else:
        pools[0][pg, of] = torch.from_numpy(np.asarray(lat, np.float32)).to(DEV).to(pools[0].dtype)
    pools[1][pg, of] = torch.from_numpy(np.asarray(rope, np.float32)).to(DEV).to(pools[1].dtype)


def lget(cache, slots, layer=None):
    """Rows [n, L] and [n, 64] of the cache as float64."""
    pg, of = at(slots)
    pools = [cache.latent, cache.rope, cache.scale]
    if layer is not None:
        pools = [None if p is None else p[layer] for p in pools]
    rope = f64(pools[1][pg, of])
    if cache.scale is None:
        return f64(pools[0][pg, of]), rope
    v = oracle.e4m3_values()[pools[0].view(torch.uint8)[pg, of].cpu().numpy()]
    e = pools[2][pg, of].cpu().numpy().astype(np.int64) - 127
    return np.ldexp(v.reshape(len(slots), -1, 128), e[..., None]).reshape(v.shape), rope


def turns(n, rot):
    a = np.arange(n)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def turned_bound(x, w, eps, rot, inter, n):
    """The float32 part of the tolerance of a normed and rotated row x."""
    plain = np.abs(oracle.norm_rope(x, w, eps, None, rot, inter))
    size = plain.copy()
    if rot:
        p = np.arange(rot).reshape(-1, 2) if inter else np.arange(rot).reshape(2, -1).T
        size[p] = plain[p].sum(1, keepdims=True)
    return (n + 16) * W * size


def typed(rng, shape, dt, spread=1.0):
    return torch.from_numpy(rng.normal(0, spread, shape).astype(np.float32)).to(dt)


# ------------------------------------------------------------------ positions on several axes

AXES = [
    # kind, lens, ctx, hq, hkv, D, page, axes, cycle, norm, rot, interleaved, joint
    ("bf16", [1], [0], 1, 1, 64, 16, 1, False, True, 64, False, False),
    ("bf16", [3, 0, 70], [15, 16, 0], 6, 2, 128, 16, 3, False, True, 128, False, True),
    ("f16", [5, 2, 9, 1], [31, 100, 7, 255], 8, 8, 64, 32, 3, True, False, 32, True, False),
    ("f16", [0, 33, 0], [60, 3, 9], 10, 2, 256, 64, 4, True, True, 256, False, False),
    ("e4m3", [2, 9, 1, 130], [14, 250, 0, 33], 12, 3, 128, 16, 3, True, True, 96, False, True),
    ("e4m3", [17, 1], [500, 7], 4, 4, 64, 256, 2, False, False, 16, True, False),
]


@pytest.mark.parametrize("case", range(len(AXES)))
def test_append_axes(case):
    kind, lens, ctx, hq, hkv, D, page, n_axes, cycle, norm, rot, inter, joint = AXES[case]
    say(f"append axes case {case}: {kind} lens={lens} D={D} axes={n_axes}")
    code, dt, u = TYPES[kind]
    b = Batch(case, lens, ctx, 1, page, False)
    rng = b.rng
    cache = make_cache(kind, b.nb, hkv, page, D, joint=joint)
    before = [bits(t).clone() for t in (cache.k, cache.v)]
    qkv = typed(rng, (b.rows, hq + 2 * hkv, D), dt, 2)
    host = qkv.double().numpy()
    qkv = qkv.to(DEV)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    qw = kw = None
    if norm:
        qw, kw = (typed(rng, D, dt, 0.2) + 1 for _ in range(2))
    half = rot // 2
    axis = [i % n_axes for i in range(half)] if cycle else sorted(rng.integers(0, n_axes, half).tolist())
    table_h = turns(97, rot)
    pos = rng.integers(0, 97, (n_axes, b.rows + 5)).astype(np.int32)
    pos[:, int(b.cu[-1]):] = -9  # padding's positions do not count
    out = dv.alloc_append_outputs(b.rows, hq, cache)
    out.q_out.fill_(-7)
    cu, pre, table = b.args()
    dv.dspark_kv_append_axes(b.B, q, k, v, b.rows, cu, pre, i32(pos)[:, :b.rows], axis, table, cache,
                             out, up(table_h), q_weight=None if qw is None else qw.to(DEV),
                             k_weight=None if kw is None else kw.to(DEV), eps=1e-5,
                             rope_interleaved=inter)
    torch.cuda.synchronize()
    assert out.append_meta.tolist() == [int(b.cu[-1]), 0]
    got_q, written = f64(out.q_out), []
    for r in range(b.B):
        if not lens[r]:
            continue
        slots = b.slots(r, ctx[r], ctx[r] + lens[r])
        written += slots
        gk, gv = get(cache, slots, "k"), get(cache, slots, "v")
        for j in range(lens[r]):
            n = b.cu[r] + j
            x = host[n]
            for h in range(hq + hkv):
                w = None if not norm else f64(qw if h < hq else kw)
                y = oracle.axes_turn(x[h], w, 1e-5, table_h, pos[:, n], axis, inter)
                f32 = turned_bound(x[h], w, 1e-5, rot, inter, D)
                if h < hq or kind != "e4m3":
                    got = got_q[n, h] if h < hq else gk[j, h - hq]
                    within(got, y, u * np.abs(y) + 1.01 * f32 + (2.0 ** -25 if kind == "f16" else 1e-30),
                           (r, j, h))
                else:
                    e = oracle.e4m3_exponent(y[None])[0]
                    half_step = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** (e - 10))
                    within(gk[j, h - hq], y, half_step + 1.07 * f32, (r, j, h))
            xv = x[hq + hkv:]
            if kind == "e4m3":
                xv = oracle.e4m3_round(xv, oracle.e4m3_exponent(xv))
            assert np.array_equal(gv[j], xv), (r, j)
    assert bool((out.q_out[int(b.cu[-1]):] == -7).all())
    for name, old in zip("kv", before):  # every other slot is as it was
        now = bits(getattr(cache, name)).clone()
        pg, of = torch.tensor(written, device=DEV).T
        now[pg, :, of] = old[pg, :, of]
        assert torch.equal(now.view(torch.uint8), old.view(torch.uint8))


@pytest.mark.parametrize("kind", ["bf16", "f16", "e4m3"])
def test_axes_of_text_are_the_append(kind):
    """Equal positions on all axes give what dspark_kv_append gives, bit for bit; q_out
    may be q."""
    say(f"axes of text {kind}")
    b = Batch(5, [4, 1, 6], [30, 0, 77], 5, 32, False)
    hq, hkv, D = 6, 3, 128
    code, dt, _ = TYPES[kind]
    x = typed(b.rng, (b.rows, hq + 2 * hkv, D), dt).to(DEV)
    w = (typed(b.rng, D, dt, 0.2) + 1).to(DEV)
    rope = up(turns(100, D))
    cu, pre, table = b.args()
    one, two = (make_cache(kind, b.nb, hkv, 32, D) for _ in range(2))
    args = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    a = dv.alloc_append_outputs(b.rows, hq, one)
    dv.dspark_kv_append(b.B, 5, *args, b.rows, cu, pre, table, one, a, q_weight=w, k_weight=w,
                        rope=rope)
    pos = np.concatenate([np.arange(c, c + n) for c, n in zip(b.ctx, b.lens)] + [[0] * 3])
    q = args[0].contiguous()
    o = dv.AppendOutputs(q, torch.empty(2, dtype=torch.int32, device=DEV))
    dv.dspark_kv_append_axes(b.B, q, *args[1:], b.rows, cu, pre, i32([pos] * 3),
                             [i % 3 for i in range(64)], table, two, o, rope, q_weight=w, k_weight=w)
    torch.cuda.synchronize()
    n = int(b.cu[-1])
    assert torch.equal(a.q_out[:n], q[:n])
    for r in range(b.B):
        slots = b.slots(r, b.ctx[r], b.ctx[r] + b.lens[r])
        for name in "kv":
            assert np.array_equal(get(one, slots, name), get(two, slots, name))


def test_axes_data_errors():
    """Rows with a position or a page that is none are left out alone, requests that
    do not fit as a whole; the others come as if alone."""
    say("axes data errors")
    D, page = 64, 16
    b = Batch(3, [20, 5, 40, 3], [4, 0, 9, 1], 1, page, False)
    cache = make_cache("bf16", b.nb, 1, page, D)
    x = typed(b.rng, (b.rows, 1, D), torch.bfloat16).to(DEV)
    pos = np.zeros((3, b.rows), np.int32)
    pos[1, 2], pos[0, 21], pos[2, 66] = 10, -1, 9  # 10 is beyond the table, 9 its last row
    table = b.table.copy()
    table[2, 1] = b.nb  # indices 16..31 of request 2
    out = dv.alloc_append_outputs(b.rows, 1, cache)
    out.q_out.fill_(-7)
    cu, pre, _ = b.args()
    rope = torch.zeros(10, 64, device=DEV)
    rope[:, :32] = 1  # no turn
    dv.dspark_kv_append_axes(b.B, x, x, x, b.rows, cu, pre, i32(pos), [0, 1, 2, 0] * 8, i32(table),
                             cache, out, rope)
    torch.cuda.synchronize()
    assert out.append_meta.tolist() == [68, dv.DATA_BAD_POS | dv.DATA_BAD_PAGE]
    lost = {2, 21} | {25 + j for j in range(40) if 16 <= 9 + j < 32}
    for n in range(68):
        assert bool((out.q_out[n] == -7).all()) == (n in lost), n
    for r in range(4):
        for j in range(b.lens[r]):
            n = int(b.cu[r]) + j
            if n in lost and 25 <= n < 65:
                continue
            got = get(cache, b.slots(r, b.ctx[r] + j, b.ctx[r] + j + 1), "k")
            assert np.isnan(got).all() if n in lost else np.array_equal(got[0], f64(x[n])), n
    for bad, bit in ((dict(prefix=-1), dv.DATA_BAD_LENS), (dict(prefix=10 ** 6), dv.DATA_BAD_PAGE),
                     (dict(cu=70), dv.DATA_BAD_LENS)):
        p, c = b.ctx[:], b.cu.copy()
        if "prefix" in bad:
            p[2] = bad["prefix"]
        else:
            c[2] = 66  # request 1 takes rows of request 2, whose words are out of order
        out.q_out.fill_(-7)
        dv.dspark_kv_append_axes(b.B, x, x, x, b.rows, i32(c), i32(p), i32(0 * pos), [0] * 32,
                                 i32(b.table), cache, out, rope)
        torch.cuda.synchronize()
        assert out.append_meta[0].item() == 68
        assert out.append_meta[1].item() & bit, bad
        assert torch.equal(out.q_out[:20], x[:20])
        assert torch.equal(out.q_out[65:68], x[65:68]) or "cu" in bad
        if "prefix" in bad:
            assert bool((out.q_out[25:65] == -7).all())


# ------------------------------------------------------------------ latent append, read, commit

LAPPEND = [
    # kind, lens, ctx, gamma, H, L, page, tree, norm, rope, interleaved, joint
    ("bf16", [1], [0], 0, 1, 512, 16, False, True, True, False, False),
    ("bf16", [3, 0, 200], [15, 16, 0], 0, 20, 512, 16, False, True, True, True, True),
    ("f16", [5, 2, 9, 1], [31, 100, 7, 255], 8, 33, 256, 32, True, False, True, False, False),
    ("f16", [4, 0, 4], [60, 9, 3], 7, 0, 512, 64, False, True, False, False, False),
    ("e4m3", [2, 9, 1, 6], [14, 250, 0, 33], 8, 128, 512, 16, True, True, True, True, True),
    ("e4m3", [1, 65, 17], [1000, 7, 500], 64, 4, 256, 256, True, True, True, False, False),
    ("e4m3", [300], [129], 0, 7, 256, 128, False, False, True, True, False),
    ("bf16", [1200, 1300], [1, 40], 0, 9, 256, 64, False, True, True, False, False),
]


@pytest.mark.parametrize("case", range(len(LAPPEND)))
def test_latent_append(case):
    kind, lens, ctx, gamma, H, L, page, tree, norm, rot, inter, joint = LAPPEND[case]
    say(f"latent append case {case}: {kind} lens={lens} H={H} L={L}")
    code, dt, u = TYPES[kind]
    b = Batch(case, [max(n, 1) for n in lens] if tree else lens, ctx, max(gamma, 1), page, tree)
    rng = b.rng
    cache = make_latent(kind, b.nb, page, L, joint=joint)
    before = [bits(cache.latent).clone(), cache.rope.clone()]
    x = typed(rng, (b.rows, L + R + 8), dt, 2)[:, :L + R]
    x[0, :L] = 0
    q = typed(rng, (b.rows, H, R + 24), dt, 2)[..., 16:16 + R] if H else None
    wt = (typed(rng, L, dt, 0.2) + 1) if norm else None
    n_pos = max(c + n for c, n in zip(ctx, lens))
    table_h = turns(n_pos, R)
    out = dv.alloc_latent_append_outputs(b.rows, H, cache)
    if H:
        out.q_rope.fill_(-7)
    cu, pre, table = b.args()
    xd = x.to(DEV)
    qd = None
    if H:  # heads with a stride of their own
        qd = torch.zeros(b.rows, H, R + 24, dtype=dt, device=DEV)[..., 16:16 + R]
        qd.copy_(q)
    dv.dspark_latent_append(b.B, xd, b.rows, cu, pre, table, cache, out, q_rope=qd,
                            weight=None if wt is None else wt.to(DEV), eps=1e-5,
                            rope=up(table_h) if rot else None, rope_interleaved=inter, gamma=gamma,
                            tree_parents=b.par())
    torch.cuda.synchronize()
    assert out.append_meta.tolist() == [int(b.cu[-1]), 0]
    host, hq = x.double().numpy(), None if q is None else q.double().numpy()
    got_q = f64(out.q_rope) if H else None
    small = 2.0 ** -25 if kind == "f16" else 1e-30
    written = []
    for r in range(b.B):
        if not b.lens[r]:
            continue
        slots = b.slots(r, ctx[r], ctx[r] + b.lens[r])
        written += slots
        lat, rope = lget(cache, slots)
        paths = oracle.tree_paths(b.tree(r), b.lens[r]) if tree else None
        for j in range(b.lens[r]):
            n = b.cu[r] + j
            row = table_h[ctx[r] + (len(paths[j]) - 1 if tree else j)] if rot else None
            y = oracle.norm_rope(host[n, :L], None if wt is None else f64(wt), 1e-5, None, 0, False)
            f32 = (L + 16) * W * np.abs(y)
            if kind == "e4m3":
                e = np.repeat(oracle.e4m3_exponent(y.reshape(-1, 128)), 128)
                bound = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** (e - 10)) + 1.07 * f32
            else:
                bound = u * np.abs(y) + 1.01 * f32 + small
            within(lat[j], y, bound if norm else np.where(kind == "e4m3", bound, 0.0), (r, j, "latent"))
            for h in range(-1, H):
                z = host[n, L:] if h < 0 else hq[n, h]
                t = oracle.norm_rope(z, None, 0, row, R, inter)
                b32 = turned_bound(z, None, 0, R if rot else 0, inter, 0)
                within(rope[j] if h < 0 else got_q[n, h], t, u * np.abs(t) + 1.01 * b32 + small if rot
                       else 0.0, (r, j, h))
    if H:
        assert bool((out.q_rope[int(b.cu[-1]):] == -7).all())
    pg, of = torch.tensor(written, device=DEV).T
    for pool, old in zip((cache.latent, cache.rope), before):  # every other slot is as it was
        now = bits(pool).clone()
        now[pg, of] = old[pg, of]
        assert torch.equal(now.view(torch.uint8), old.view(torch.uint8))

    say(f"latent read case {case}")
    rd = dv.alloc_latent_read_outputs(b.rows, cache)
    rd.latent_out.fill_(-7)
    rd.rope_out.fill_(-7)
    dv.dspark_latent_read(b.B, b.rows, cu, pre, table, cache, rd)
    torch.cuda.synchronize()
    assert rd.read_meta.tolist() == [int(b.cu[-1]), 0]
    lat, rope = lget(cache, written)
    n = int(b.cu[-1])
    assert np.array_equal(f64(rd.latent_out[:n]), lat) and np.array_equal(f64(rd.rope_out[:n]), rope)
    assert bool((rd.latent_out[n:] == -7).all()) and bool((rd.rope_out[n:] == -7).all())


def test_latent_append_in_place_and_nonfinite():
    """q_rope_out may be q_rope, a part of wider heads; NaN and infinite elements become
    NaN in 8 bits, and a group's exponent comes from its finite ones."""
    say("latent append in place, non-finite")
    L, H, page = 512, 9, 16
    b = Batch(7, [4], [3], 1, page, False, pad=0)
    cache = make_latent("e4m3", b.nb, page, L)
    x = np.random.default_rng(0).normal(0, 1, (4, L + R)).astype(np.float32)
    x[0, 5], x[0, 200], x[1, 128:256], x[2, 300], x[3, :128] = np.nan, np.inf, -np.inf, 3.3e38, 1e-38
    x[1, L + 3] = np.inf
    t = torch.from_numpy(x).to(torch.bfloat16)
    x = t.double().numpy()
    q = typed(b.rng, (4, H, 128 + R), torch.bfloat16).to(DEV)
    part, keep = q[..., 128:], q.clone()
    o = dv.LatentAppendOutputs(part, torch.empty(2, dtype=torch.int32, device=DEV))
    cu, pre, table = b.args()
    rope = up(turns(10, R))
    dv.dspark_latent_append(1, t.to(DEV), 4, cu, pre, table, cache, o, q_rope=part, rope=rope)
    two = dv.alloc_latent_append_outputs(4, H, cache)
    dv.dspark_latent_append(1, t.to(DEV), 4, cu, pre, table, cache, two, q_rope=keep[..., 128:],
                            rope=rope)
    torch.cuda.synchronize()
    assert torch.equal(part, two.q_rope) and torch.equal(q[..., :128], keep[..., :128])
    lat, _ = lget(cache, b.slots(0, 3, 7))
    assert np.array_equal(lat, oracle.latent_e4m3(x[:, :L]), equal_nan=True)


@pytest.mark.parametrize("gamma", [0, 6])
def test_latent_append_data_errors(gamma):
    say(f"latent append data errors gamma={gamma}")
    L, page = 256, 16
    b = Batch(4, [5, 7, 4, 6], [14, 3, 20, 0], max(gamma, 1), page, False)
    x = typed(b.rng, (b.rows, L + R), torch.bfloat16).to(DEV)
    q = x[:, None, L:]
    par = np.tile(np.arange(max(gamma, 1)), (4, 1)).astype(np.int32)
    rope = up(turns(20, R))  # request 2 begins at its end
    rope[:, 32:] = 0
    rope[:, :32] = 1

    def call(want, lost, cu=b.cu, pre=b.ctx, table=b.table, parents=None, rope_rows=40):
        cache = make_latent("bf16", b.nb, page, L)
        o = dv.alloc_latent_append_outputs(b.rows, 1, cache)
        o.q_rope.fill_(-7)
        tab = torch.cat([rope, rope])[:rope_rows]
        dv.dspark_latent_append(b.B, x, b.rows, i32(cu), i32(pre), i32(table), cache, o, q_rope=q,
                                rope=tab, gamma=gamma, tree_parents=None if parents is None else
                                i32(parents))
        torch.cuda.synchronize()
        assert o.append_meta.tolist() == [int(b.cu[-1]), want]
        for n in range(int(b.cu[-1])):
            assert torch.equal(o.q_rope[n], q[n]) != (n in lost), n
        for r in range(4):
            for j in range(b.lens[r]):
                n = int(b.cu[r]) + j
                if n not in lost:
                    assert np.array_equal(lget(cache, b.slots(r, b.ctx[r] + j, b.ctx[r] + j + 1))[0][0],
                                          f64(x[n, :L]))

    rows = [set(range(int(b.cu[r]), int(b.cu[r + 1]))) for r in range(4)]
    call(0, set())
    call(dv.DATA_BAD_LENS, rows[1], pre=[14, -1, 20, 0])
    call(dv.DATA_BAD_PAGE, rows[1], pre=[14, 10 ** 6, 20, 0])
    call(dv.DATA_BAD_POS, rows[2], rope_rows=20)
    call(dv.DATA_BAD_POS, {int(b.cu[2]) + 3}, rope_rows=23)
    bad = b.table.copy()
    bad[0, 1] = -1
    call(dv.DATA_BAD_PAGE, {2, 3, 4}, table=bad)
    if gamma:
        p = par.copy()
        p[3, 2] = 3
        call(dv.DATA_BAD_TREE, rows[3], parents=p)
        flat = 0 * par  # every draft a child of the root: depth 1
        call(0, set(), parents=flat, rope_rows=22)
        call(dv.DATA_BAD_POS, rows[2] - {int(b.cu[2])}, parents=flat, rope_rows=21)


@pytest.mark.parametrize("kind,L", [("bf16", 512), ("f16", 256), ("e4m3", 512), ("e4m3", 256)])
def test_latent_read_spans(kind, L):
    """Spans of any length, none among them, a batch longer than one search, and words
    out of order."""
    say(f"latent read spans {kind} L={L}")
    rng = np.random.default_rng(L)
    n = [0, 1, 40, 0, 17, 300] + rng.integers(0, 9, 90).tolist()
    st = [0, 15, 3, 9, 0, 77] + rng.integers(0, 40, 90).tolist()
    b = Batch(1, [max(1, x) for x in n], st, 4, 16, False)
    b.cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    cache = make_latent(kind, b.nb, 16, L)
    rows = int(b.cu[-1])
    for r in range(b.B):
        if n[r]:
            lput(cache, b.slots(r, st[r], st[r] + n[r]), rng.normal(0, 1, (n[r], L)),
                 rng.normal(0, 1, (n[r], R)))
    for broken in (False, True):
        cu = b.cu.copy()
        if broken:
            cu[50] = 10 ** 6
        rd = dv.alloc_latent_read_outputs(rows, cache)
        rd.latent_out.fill_(-7)
        dv.dspark_latent_read(b.B, rows, i32(cu), i32(st), i32(b.table), cache, rd)
        torch.cuda.synchronize()
        assert rd.read_meta.tolist() == [rows, dv.DATA_BAD_LENS if broken else 0]
        for r in range(b.B):
            if n[r] and not (broken and r in (49, 50)):
                lat, rope = lget(cache, b.slots(r, st[r], st[r] + n[r]))
                assert np.array_equal(f64(rd.latent_out[b.cu[r]:b.cu[r + 1]]), lat), r
                assert np.array_equal(f64(rd.rope_out[b.cu[r]:b.cu[r + 1]]), rope), r


@pytest.mark.parametrize("kind,L,layers,gamma,joint", [
    ("bf16", 512, 3, 5, False), ("e4m3", 512, 5, 16, True), ("f16", 256, 1, 64, False),
    ("e4m3", 256, 9, 7, False), ("bf16", 256, 2, 33, True)])
def test_latent_commit(kind, L, layers, gamma, joint):
    say(f"latent commit {kind} L={L} layers={layers} gamma={gamma}")
    rng = np.random.default_rng(gamma)
    B, page = 7, 16
    ctx = rng.integers(0, 50, B).tolist()
    b = Batch(2, [gamma + 1] * B, ctx, gamma, page, False)
    cache = make_latent(kind, b.nb, page, L, layers, joint)
    for r in range(B):
        for layer in range(layers):
            n = ctx[r] + gamma + 1
            lput(cache, b.slots(r, 0, n), rng.normal(0, 1, (n, L)), rng.normal(0, 1, (n, R)), layer)
    num = [0, gamma] + rng.integers(0, gamma + 1, B - 2).tolist()
    paths = np.full((B, gamma + 1), -1, np.int32)
    for r in range(B):
        paths[r, :num[r] + 1] = [0] + sorted(rng.choice(np.arange(1, gamma + 1), num[r], False).tolist())
    paths[4, 0] = 2  # no path
    bad = [4]
    want, moved = {}, 0
    for r in range(B):
        moves = oracle.commit_moves(paths[r], num[r], ctx[r], gamma) if r not in bad else None
        n = ctx[r] + gamma + 1
        for layer in range(layers):
            lat, rope = lget(cache, b.slots(r, 0, n), layer)
            if moves:
                src, dst = [m[0] for m in moves], [m[1] for m in moves]
                lat[dst], rope[dst] = lat[src].copy(), rope[src].copy()
            want[r, layer] = lat, rope
        moved += len(moves or [])
    meta = torch.empty(2, dtype=torch.int32, device=DEV)
    dv.dspark_latent_commit(B, gamma, i32(paths), i32(num), i32(ctx), i32(b.table), cache, meta)
    torch.cuda.synchronize()
    assert meta.tolist() == [moved, dv.DATA_BAD_TREE]
    for (r, layer), (lat, rope) in want.items():
        got = lget(cache, b.slots(r, 0, ctx[r] + gamma + 1), layer)
        assert np.array_equal(got[0], lat) and np.array_equal(got[1], rope), (r, layer)


# ------------------------------------------------------------------ absorbed attention

def latent_setup(b, kind, H, L, seed=0, joint=False, spread=1.0):
    dt = TYPES[kind][1]
    rng = np.random.default_rng(seed)
    cache = make_latent(kind, b.nb, b.page, L, joint=joint)
    for r in range(b.B):
        T = b.ctx[r] + b.lens[r]
        if T:
            lput(cache, b.slots(r, 0, T), rng.normal(0, spread, (T, L)), rng.normal(0, spread, (T, R)))
    ql = typed(rng, (b.rows, H, L), dt).to(DEV)
    qr = torch.zeros(b.rows, H, 40 + R, dtype=dt, device=DEV)[..., 40:]
    qr.copy_(typed(rng, (b.rows, H, R), dt))
    for t in (ql, qr):
        t[int(b.cu[-1]):] = float("nan")
    return cache, ql, qr


def attention_bound(ref, lse_ref, mean_abs, t, top_v, n, u, kind):
    tail = n * 2.0 ** -25 * top_v if kind == "f16" else 0.0
    bound = u * np.abs(ref) + (u + 2 * t[..., None] + (n + 32) * W) * mean_abs + tail
    # log2, its product with ln 2, and the maximum's: steps of float32 of the parts
    lse_bound = t + (n + 32) * W + 4 * W * np.abs(lse_ref) + 1e-6
    return bound, lse_bound


def latent_check(b, kind, H, L, scale, cache, ql, qr, o, rows=None):
    u = TYPES[kind][2]
    got, got_lse = f64(o.out), f64(o.lse)
    for r in range(b.B):
        T, s = b.ctx[r] + b.lens[r], slice(int(b.cu[r]), int(b.cu[r + 1]))
        lat, rope = lget(cache, b.slots(r, 0, T))
        ref, lse, mean_abs, top = oracle.latent_attention(
            f64(ql[s]), f64(qr[s]), lat, rope, b.ctx[r], None if b.parents is None else b.parents[r],
            scale)
        t = (L + R + 16) * W * top
        bound, lse_bound = attention_bound(ref, lse, mean_abs, t, np.abs(lat).max(), T, u, kind)
        within(got[s], ref, bound, (r, "out"))
        within(got_lse[s], lse, lse_bound, (r, "lse"))
    assert bool((o.out[int(b.cu[-1]):] == -7).all()) and bool((o.lse[int(b.cu[-1]):] == -7).all())


def latent_run(b, kind, H, L, scale, seed=0, joint=False, spread=1.0):
    cache, ql, qr = latent_setup(b, kind, H, L, seed, joint, spread)
    o = dv.alloc_latent_attention_outputs(b.B, b.gamma, b.rows, H, cache, lse=True)
    o.workspace.fill_(0xFF)
    o.out.fill_(-7)
    o.lse.fill_(-7)
    dv.dspark_latent_attention(b.B, b.gamma, ql, qr, b.rows, *b.args(), cache, scale, o,
                               tree_parents=b.par())
    torch.cuda.synchronize()
    assert o.attention_meta.tolist() == [int(b.cu[-1]), 0]
    latent_check(b, kind, H, L, scale, cache, ql, qr, o)
    return cache, ql, qr, o


LATTN = [
    # kind, lens, ctx, gamma, H, L, page, tree, scale, joint
    ("bf16", [1], [0], 1, 1, 512, 16, False, 0.07, False),
    ("bf16", [1], [63], 1, 1, 512, 16, False, 0.07, False),
    ("bf16", [1, 1], [64, 700], 1, 32, 512, 64, False, 0.07, True),
    ("bf16", [3, 1, 5], [15, 200, 0], 4, 20, 512, 16, True, 0.05, False),
    ("bf16", [4, 2], [130, 61], 3, 128, 512, 128, False, 0.06, False),
    ("f16", [5, 2, 9, 1], [31, 100, 7, 255], 8, 33, 256, 32, True, 0.05, True),
    ("f16", [9], [1500], 8, 20, 512, 64, True, -0.05, False),
    ("e4m3", [2, 9, 1, 6], [14, 250, 0, 330], 8, 12, 512, 16, True, 0.05, True),
    ("e4m3", [1, 65, 17], [1000, 7, 500], 64, 3, 256, 256, True, 0.05, False),
    ("e4m3", [1, 3], [127, 128], 2, 128, 256, 16, False, 0.05, False),
    ("bf16", [65], [90], 64, 5, 256, 32, True, 0.05, False),
    ("bf16", [2], [4000], 1, 7, 256, 64, False, 0.05, False),
]


@pytest.mark.parametrize("case", range(len(LATTN)))
def test_latent_attention(case):
    kind, lens, ctx, gamma, H, L, page, tree, scale, joint = LATTN[case]
    say(f"latent attention case {case}: {kind} lens={lens} ctx={ctx} H={H} L={L}")
    latent_run(Batch(case, lens, ctx, gamma, page, tree), kind, H, L, scale, case, joint)


@pytest.mark.parametrize("kind,L", [("bf16", 512), ("f16", 256), ("e4m3", 512)])
@pytest.mark.parametrize("B", [64, 65, 200])
def test_latent_attention_of_large_batches(kind, L, B):
    say(f"latent attention batch of {B} {kind}")
    rng = np.random.default_rng(B)
    lens = rng.integers(1, 4, B).tolist()
    ctx = rng.integers(0, 150, B).tolist()
    latent_run(Batch(B, lens, ctx, 3, 16, True), kind, 3, L, 0.05)


@pytest.mark.parametrize("kind,L,ctx", [("bf16", 512, 20000), ("f16", 256, 33333), ("e4m3", 512, 12345)])
def test_latent_attention_over_a_long_context(kind, L, ctx):
    say(f"latent attention over {ctx}")
    latent_run(Batch(3, [2, 1], [ctx, 100], 2, 128, False), kind, 2, L, 0.05)


@pytest.mark.parametrize("scale", [0.0, -0.3, 1e30, 3.4e38, 1e-40])
@pytest.mark.parametrize("kind,L", [("bf16", 512), ("f16", 256)])
def test_latent_attention_scales(kind, L, scale):
    """A scale of zero gives the mean, its sign and size are the scores'."""
    say(f"latent attention scale {scale} {kind}")
    b = Batch(9, [3, 2], [70, 5], 3, 16, False)
    if abs(scale) < 1:
        latent_run(b, kind, 4, L, scale)
        return
    # the largest score takes everything: its latent comes out
    cache, ql, qr = latent_setup(b, kind, 4, L)
    o = dv.alloc_latent_attention_outputs(b.B, b.gamma, b.rows, 4, cache)
    dv.dspark_latent_attention(b.B, b.gamma, ql, qr, b.rows, *b.args(), cache, scale, o)
    torch.cuda.synchronize()
    got = f64(o.out)
    for r in range(b.B):
        lat, rope = lget(cache, b.slots(r, 0, b.ctx[r] + b.lens[r]))
        for j in range(b.lens[r]):
            n, T = int(b.cu[r]) + j, b.ctx[r] + j + 1
            s = f64(ql[n]) @ lat[:T].T + f64(qr[n]) @ rope[:T].T
            if scale > 1e38:
                # (scores past float32 are infinite: nothing to compare but that it ends)
                continue
            assert np.array_equal(got[n], lat[s.argmax(-1)]), (r, j)


@pytest.mark.parametrize("kind,L", [("bf16", 512), ("bf16", 256), ("f16", 512), ("e4m3", 512),
                                    ("e4m3", 256)])
def test_latent_attention_ignores_what_a_row_does_not_see(kind, L):
    """NaN, infinities and any exponent byte in a draft's row leave the rows that do
    not see it as they were, bit for bit; rows that see it have no meaning."""
    say(f"latent attention unseen rows {kind} L={L}")
    H, gamma = 7, 20
    b = Batch(6, [21, 9], [50, 61], gamma, 16, True)
    cache, ql, qr, o = latent_run(b, kind, H, L, 0.05)
    plain = o.out.clone()
    for what in ("latent", "rope", "byte"):
        if what == "byte" and kind != "e4m3":
            continue
        slot = b.slots(0, b.ctx[0] + 4, b.ctx[0] + 5)[0]
        pools = [p.clone() for p in (bits(cache.latent), cache.rope)] + \
            ([cache.scale.clone()] if kind == "e4m3" else [])
        if what == "latent":
            if kind == "e4m3":
                cache.latent.view(torch.uint8)[slot[0], slot[1], 77] = 0xFF
            else:
                cache.latent[slot[0], slot[1], 77:79] = torch.tensor([float("inf"), float("nan")],
                                                                     device=DEV)
        elif what == "rope":
            cache.rope[slot[0], slot[1], 63] = float("-inf")
        else:
            cache.scale[slot[0], slot[1], 1] = 255
        dv.dspark_latent_attention(b.B, gamma, ql, qr, b.rows, *b.args(), cache, 0.05, o,
                                   tree_parents=b.par())
        torch.cuda.synchronize()
        paths = oracle.tree_paths(b.parents[0], 21)
        for n in range(int(b.cu[-1])):
            sees = n < 21 and 4 in paths[n]
            same = torch.equal(o.out[n], plain[n])
            assert not same if sees else same, (what, n)
        for pool, old in zip((bits(cache.latent), cache.rope, cache.scale), pools):
            pool.copy_(old)


@pytest.mark.parametrize("kind,L", [("bf16", 512), ("e4m3", 256)])
def test_latent_attention_data_errors(kind, L):
    say(f"latent attention data errors {kind}")
    H, gamma, page = 5, 6, 16
    b = Batch(8, [5, 7, 4, 6], [40, 3, 90, 0], gamma, page, True)
    cache, ql, qr, o = latent_run(b, kind, H, L, 0.05)
    plain, plain_lse = o.out.clone(), o.lse.clone()
    rows = [slice(int(b.cu[r]), int(b.cu[r + 1])) for r in range(4)]

    def call(bit, lost, cu=b.cu, pre=b.ctx, table=b.table, par=b.parents):
        o.out.fill_(-7)
        o.lse.fill_(-7)
        dv.dspark_latent_attention(4, gamma, ql, qr, b.rows, i32(cu), i32(pre), i32(table), cache,
                                   0.05, o, tree_parents=i32(par))
        torch.cuda.synchronize()
        assert o.attention_meta.tolist() == [int(b.cu[-1]), bit]
        for r in range(4):
            if r == lost:
                assert bool((o.out[rows[r]] == -7).all()) and bool((o.lse[rows[r]] == -7).all())
            else:
                assert torch.equal(o.out[rows[r]], plain[rows[r]]), r
                assert torch.equal(o.lse[rows[r]], plain_lse[rows[r]]), r

    call(0, None)
    call(dv.DATA_BAD_LENS, 1, pre=[40, -3, 90, 0])
    call(dv.DATA_BAD_PAGE, 1, pre=[40, 10 ** 6, 90, 0])
    p = b.parents.copy()
    p[3, 4] = 5
    call(dv.DATA_BAD_TREE, 3, par=p)
    # indices on a page that is none count as not seen
    t = b.table.copy()
    t[2, 1], t[2, 3] = -1, b.nb
    o.out.fill_(-7)
    dv.dspark_latent_attention(4, gamma, ql, qr, b.rows, i32(b.cu), i32(b.ctx), i32(t), cache, 0.05,
                               o, tree_parents=i32(b.parents))
    torch.cuda.synchronize()
    assert o.attention_meta.tolist() == [int(b.cu[-1]), dv.DATA_BAD_PAGE]
    for r in (0, 1, 3):
        assert torch.equal(o.out[rows[r]], plain[rows[r]])
    keep = [i for i in range(94) if i // 16 not in (1, 3)]
    lat, rope = lget(cache, b.slots(2, 0, 94))
    ref, lse, mean_abs, top = oracle.latent_attention(
        f64(ql[rows[2]]), f64(qr[rows[2]]), lat[keep], rope[keep], 90 - 32, b.parents[2], 0.05)
    bound, _ = attention_bound(ref, lse, mean_abs, (L + R + 16) * W * top, np.abs(lat).max(), 94,
                               TYPES[kind][2], kind)
    within(f64(o.out[rows[2]]), ref, bound, "rest of the pages")
    # a request that sees nothing at all
    t[3, :] = -1
    dv.dspark_latent_attention(4, gamma, ql, qr, b.rows, i32(b.cu), i32(b.ctx), i32(t), cache, 0.05,
                               o, tree_parents=i32(b.parents))
    torch.cuda.synchronize()
    assert bool((o.out[rows[3]] == 0).all()) and bool((o.lse[rows[3]] == -float("inf")).all())


@pytest.mark.parametrize("kind,L,size", [("bf16", 512, 2.0 ** 60), ("f16", 256, 2.0 ** 7),
                                         ("e4m3", 512, 2.0 ** 60)])
def test_latent_equal_scores_of_any_size_give_the_mean(kind, L, size):
    """Equal scores of 2^30 and more keep a largest weight of 1: the plain mean of the
    latents comes out."""
    say(f"latent equal scores {kind}")
    b = Batch(2, [1], [40], 1, 16, False)
    dt, u = TYPES[kind][1:]
    cache = make_latent(kind, b.nb, 16, L)
    T = 41
    lat = np.zeros((T, L))
    lat[:, 0] = size
    lat[:, 1:] = np.random.default_rng(1).integers(-4, 5, (T, L - 1))
    if kind == "e4m3":
        lat[:, 1:128] = 0
    lput(cache, b.slots(0, 0, T), lat, np.zeros((T, R)))
    ql = torch.zeros(b.rows, 2, L, dtype=dt, device=DEV)
    ql[:, 0, 0], ql[:, 1, 0] = 1.0, -1.0
    qr = torch.zeros(b.rows, 2, R, dtype=dt, device=DEV)
    o = dv.alloc_latent_attention_outputs(1, 1, b.rows, 2, cache)
    dv.dspark_latent_attention(1, 1, ql, qr, b.rows, *b.args(), cache, 1.0 if kind != "f16" else 2.0 ** 24, o)
    torch.cuda.synchronize()
    got, _ = lget(cache, b.slots(0, 0, T))
    ref = np.tile(got.mean(0), (2, 1))
    # equal weights are exact in the product; the sum and the quotient in float32
    within(f64(o.out[0]), ref, u * np.abs(ref) + (T + 32) * W * np.abs(got).mean(0) +
           (2.0 ** -25 if kind == "f16" else 0), "mean")


# ------------------------------------------------------------------ expanded attention

def prefill_check(b, kind, H, n, L, scale, cache, q, wk, wv, o, lost=()):
    u = TYPES[kind][2]
    got, got_lse = f64(o.out), f64(o.lse)
    small = 2.0 ** -25 if kind == "f16" else 0.0
    for r in range(b.B):
        T, s = b.ctx[r] + b.lens[r], slice(int(b.cu[r]), int(b.cu[r + 1]))
        if r in lost:
            assert np.all(got[s] == -7) and np.all(got_lse[s] == -7)
            continue
        if not b.lens[r]:
            continue
        lat, rope = lget(cache, b.slots(r, 0, T))
        ref, lse, mean_abs, top, rounded, spread, deep = oracle.latent_prefill(
            f64(q[s]), f64(wk), f64(wv), lat, rope, b.ctx[r], scale)
        qsum = abs(scale) * np.abs(f64(q[s]))[..., :n].sum(-1)
        t = (n + R + 16) * W * top + 1.01 * (u * rounded + (L + 16) * W * spread + small * qsum)
        v = np.abs(lat @ np.swapaxes(f64(wv), 1, 2)).max()
        bound, lse_bound = attention_bound(ref, lse, mean_abs, t, v, T, u, kind)
        bound = bound + 1.01 * (u * mean_abs + (L + 16) * W * deep + small)
        # (the terms above are of first order in t)
        assert t.max() < 0.25
        within(got[s], ref, bound * np.exp(2 * t[..., None]), (r, "out"))
        within(got_lse[s], lse, lse_bound, (r, "lse"))
    assert np.all(got[int(b.cu[-1]):] == -7)


def prefill_run(b, kind, H, n, L, scale, seed=0, joint=False, spare=0, check=True):
    dt = TYPES[kind][1]
    cache, _, _ = latent_setup(b, kind, 1, L, seed, joint)
    rng = np.random.default_rng(seed + 100)
    q = typed(rng, (b.rows, H, n + R), dt).to(DEV)
    q[int(b.cu[-1]):] = float("nan")
    w = typed(rng, (H, 2 * n + 8, L), dt, L ** -0.5).to(DEV)
    wk, wv = w[:, :n], w[:, n:2 * n]
    keys = sum(b.ctx[r] + b.lens[r] for r in range(b.B) if b.lens[r])
    o = dv.alloc_latent_prefill_outputs(b.B, b.rows, keys + spare, H, n, cache, lse=True)
    o.workspace.fill_(0xFF)
    o.out.fill_(-7)
    o.lse.fill_(-7)
    dv.dspark_latent_prefill(b.B, q, wk, wv, b.rows, keys + spare, *b.args(), cache, scale, o)
    torch.cuda.synchronize()
    assert o.attention_meta.tolist() == [int(b.cu[-1]), 0]
    if check:
        prefill_check(b, kind, H, n, L, scale, cache, q, wk, wv, o)
    return cache, q, wk, wv, o, keys


PREFILL = [
    # kind, lens, ctx, H, nope, L, page, scale, joint
    ("bf16", [1], [0], 1, 128, 512, 16, 0.07, False),
    ("bf16", [1, 0, 2], [63, 7, 64], 3, 128, 512, 16, 0.07, False),
    ("bf16", [257], [0], 2, 128, 512, 64, 0.07, True),
    ("bf16", [64, 128, 31], [0, 0, 0], 8, 128, 256, 16, 0.07, False),
    ("f16", [100, 300], [77, 5], 4, 64, 256, 32, -0.06, False),
    ("f16", [33, 0, 0, 65], [500, 9, 0, 127], 5, 128, 512, 64, 0.07, False),
    ("e4m3", [90, 200], [300, 0], 9, 128, 512, 16, 0.07, True),
    ("e4m3", [256, 1, 256], [1, 255, 256], 2, 64, 256, 256, 0.0, False),
    ("bf16", [520], [700], 1, 64, 512, 128, 0.1, False),
]


@pytest.mark.parametrize("case", range(len(PREFILL)))
def test_latent_prefill(case):
    kind, lens, ctx, H, n, L, page, scale, joint = PREFILL[case]
    say(f"latent prefill case {case}: {kind} lens={lens} ctx={ctx} H={H} n={n} L={L}")
    prefill_run(Batch(case, lens, ctx, 1, page, False), kind, H, n, L, scale, case, joint,
                spare=37 * (case % 3))


def test_latent_prefill_of_a_large_batch():
    say("latent prefill batch of 300")
    rng = np.random.default_rng(4)
    lens = [int(x) if x > 2 else 0 for x in rng.integers(0, 9, 300)]
    ctx = rng.integers(0, 60, 300).tolist()
    prefill_run(Batch(4, lens, ctx, 1, 16, False), "bf16", 2, 64, 256, 0.07)


@pytest.mark.parametrize("kind,n", [("bf16", 128), ("f16", 64), ("e4m3", 128)])
def test_latent_prefill_ignores_the_future(kind, n):
    """A cached row with NaN or infinity leaves the rows before it as they were, bit for
    bit; rows from it on have no meaning."""
    say(f"latent prefill future {kind}")
    L = 256
    b = Batch(6, [200, 90], [30, 0], 1, 16, False)
    cache, q, wk, wv, o, keys = prefill_run(b, kind, 3, n, L, 0.07)
    plain = o.out.clone()
    for what in ("latent", "rope"):
        slot = b.slots(0, 30 + 77, 30 + 78)[0]
        pools = [bits(cache.latent).clone(), cache.rope.clone()]
        if what == "rope":
            cache.rope[slot[0], slot[1], 5] = float("inf")
        elif kind == "e4m3":
            cache.latent.view(torch.uint8)[slot[0], slot[1], 7] = 0x7F
        else:
            cache.latent[slot[0], slot[1], 7] = float("-inf")
        dv.dspark_latent_prefill(2, q, wk, wv, b.rows, keys, *b.args(), cache, 0.07, o)
        torch.cuda.synchronize()
        for row in range(290):
            sees = 77 <= row < 200
            same = torch.equal(o.out[row], plain[row])
            assert not same if sees else same, (what, row)
        bits(cache.latent).copy_(pools[0])
        cache.rope.copy_(pools[1])


def test_latent_prefill_data_errors():
    say("latent prefill data errors")
    kind, H, n, L, page = "bf16", 3, 64, 256, 16
    b = Batch(8, [50, 70, 40, 0, 60], [40, 3, 90, 8, 0], 1, page, False)
    cache, q, wk, wv, o, keys = prefill_run(b, kind, H, n, L, 0.07)

    def call(bit, lost, pre=b.ctx, table=b.table, max_keys=keys, cu=b.cu, rows=None):
        o.out.fill_(-7)
        o.lse.fill_(-7)
        dv.dspark_latent_prefill(b.B, q, wk, wv, b.rows if rows is None else rows, max_keys, i32(cu),
                                 i32(pre), i32(table), cache, 0.07, o)
        torch.cuda.synchronize()
        assert o.attention_meta.tolist() == [int(b.cu[-1]), bit]
        prefill_check(b, kind, H, n, L, 0.07, cache, q, wk, wv, o, lost)

    call(0, ())
    call(dv.DATA_BAD_LENS, (1,), pre=[40, -1, 90, 8, 0])
    call(dv.DATA_BAD_PAGE, (1,), pre=[40, 10 ** 6, 90, 8, 0])
    t = b.table.copy()
    t[2, 3] = b.nb
    call(dv.DATA_BAD_PAGE, (2,), table=t)
    call(dv.DATA_BAD_LENS, (4,), max_keys=keys - 1)
    call(dv.DATA_BAD_LENS, (2, 4), max_keys=90 + 73 + 10)
    call(dv.DATA_BAD_LENS, (0, 1, 2, 4), max_keys=0)
    call(dv.DATA_BAD_LENS, (4,), rows=int(b.cu[-1]) - 1)


def test_latent_prefill_is_the_absorbed_form():
    """The two forms of attention agree within their bounds, through the weights."""
    say("latent prefill against absorbed")
    H, n, L, scale = 4, 128, 512, 0.07
    b = Batch(12, [6, 9], [70, 200], 8, 32, False)
    cache, q, wk, wv, o, keys = prefill_run(b, "bf16", H, n, L, scale)
    rows = int(b.cu[-1])
    ql = torch.einsum("nha,hal->nhl", q[:rows, :, :n].double(), wk.double()).to(torch.bfloat16)
    pad = torch.zeros(b.rows - rows, H, L, dtype=torch.bfloat16, device=DEV)
    a = dv.alloc_latent_attention_outputs(b.B, 8, b.rows, H, cache, lse=True)
    a.lse.fill_(-7)
    dv.dspark_latent_attention(b.B, 8, torch.cat([ql, pad]), q[..., n:], b.rows, *b.args(), cache,
                               scale, a)
    torch.cuda.synchronize()
    # both lse err by the rounding of one operand of the scores: u of sum |q||k| each
    u = 2.0 ** -8
    for r in range(b.B):
        s = slice(int(b.cu[r]), int(b.cu[r + 1]))
        lat, rope = lget(cache, b.slots(r, 0, b.ctx[r] + b.lens[r]))
        size = oracle.latent_prefill(f64(q[s]), f64(wk), f64(wv), lat, rope, b.ctx[r], scale)[4]
        deep = oracle.latent_attention(f64(ql[s]), 0 * f64(q[s, :, n:]), lat, 0 * rope, b.ctx[r], None,
                                       scale)[3]
        within(f64(a.lse[s]), f64(o.lse[s]), 1.05 * u * (size + deep) + 1e-4, (r, "lse"))


# ------------------------------------------------------------------ together, captured, side by side

def test_latent_serving_loop():
    """A prompt in two chunks, then verify steps of trees: append, attention, accept and
    commit, each against what the cache holds."""
    say("latent serving loop")
    kind, H, n, L, gamma, V, page = "bf16", 4, 64, 256, 6, 500, 16
    rng = np.random.default_rng(21)
    B, u = 3, TYPES["bf16"][2]
    limit = [90, 70, 110]
    b = Batch(1, [gamma + 1] * B, limit, gamma, page, True, extra_pages=1)
    cache = make_latent(kind, b.nb, page, L)
    w = typed(rng, (H, 2 * n, L), torch.bfloat16, L ** -0.5).to(DEV)
    norm = (typed(rng, L, torch.bfloat16, 0.1) + 1).to(DEV)
    rope = up(turns(256, R))
    done = [0] * B
    table = i32(b.table)
    for chunk in ([40, 0, 33], [21, 52, 1]):
        cu = np.concatenate([[0], np.cumsum(chunk)])
        rows = int(cu[-1]) + 2
        x = typed(rng, (rows, L + R), torch.bfloat16).to(DEV)
        q = typed(rng, (rows, H, n + R), torch.bfloat16).to(DEV)
        ap = dv.LatentAppendOutputs(q[..., n:], torch.empty(2, dtype=torch.int32, device=DEV))
        dv.dspark_latent_append(B, x, rows, i32(cu), i32(done), table, cache, ap, q_rope=q[..., n:],
                                weight=norm, rope=rope)
        keys = sum(d + c for d, c in zip(done, chunk))
        o = dv.alloc_latent_prefill_outputs(B, rows, keys, H, n, cache, lse=True)
        o.out.fill_(-7)
        o.lse.fill_(-7)
        dv.dspark_latent_prefill(B, q, w[:, :n], w[:, n:], rows, keys, i32(cu), i32(done), table,
                                 cache, 0.08, o)
        torch.cuda.synchronize()
        b.lens, b.ctx, b.cu, par = list(chunk), list(done), cu, b.parents
        b.parents = None
        prefill_check(b, kind, H, n, L, 0.08, cache, q, w[:, :n], w[:, n:], o)
        b.parents = par
        done = [d + c for d, c in zip(done, chunk)]
    meta = torch.empty(2, dtype=torch.int32, device=DEV)
    for step in range(4):
        b.lens = rng.integers(1, gamma + 2, B).tolist()
        b.ctx, b.cu = list(done), np.concatenate([[0], np.cumsum(b.lens)]).astype(np.int32)
        b.rows = int(b.cu[-1]) + 1
        for r in range(B):
            for j in range(1, gamma + 1):
                b.parents[r, j - 1] = rng.integers(0, j)
        cu, pre, table = b.args()
        x = typed(rng, (b.rows, L + R), torch.bfloat16).to(DEV)
        qr = typed(rng, (b.rows, H, R), torch.bfloat16).to(DEV)
        ql = typed(rng, (b.rows, H, L), torch.bfloat16).to(DEV)
        ap = dv.alloc_latent_append_outputs(b.rows, H, cache)
        dv.dspark_latent_append(B, x, b.rows, cu, pre, table, cache, ap, q_rope=qr, weight=norm,
                                rope=rope, gamma=gamma, tree_parents=b.par())
        o = dv.alloc_latent_attention_outputs(B, gamma, b.rows, H, cache, lse=True)
        o.out.fill_(-7)
        o.lse.fill_(-7)
        dv.dspark_latent_attention(B, gamma, ql, ap.q_rope, b.rows, cu, pre, table, cache, 0.05, o,
                                   tree_parents=b.par())
        logits = torch.randn(b.rows, V, device=DEV)
        drafts = torch.stack([logits[(cu[:-1].long()[:, None] + i32(b.parents).long())
                                     .clamp(max=b.rows - 1).flatten()].argmax(-1).view(B, gamma)])[0]
        drafts = drafts.int()
        drafts[:, 1::3] = 1
        ac = dv.alloc_tree_accept_outputs(B, gamma, b.rows, V, dv.F32, DEV)
        dv.dspark_tree_accept(B, gamma, V, dv.F32, logits, V, b.rows, cu, drafts, b.par(), pre, ac)
        torch.cuda.synchronize()
        latent_check(b, kind, H, L, 0.05, cache, ql, ap.q_rope, o)
        num, paths = ac.num_correct.tolist(), ac.path_rows.tolist()
        want = [lget(cache, b.slots(r, 0, done[r]) + [b.slots(r, done[r] + p, done[r] + p + 1)[0]
                                                    for p in paths[r][:num[r] + 1]]) for r in range(B)]
        dv.dspark_latent_commit(B, gamma, ac.path_rows, ac.num_correct, pre, table, cache, meta)
        torch.cuda.synchronize()
        assert meta[1].item() == 0
        done = ac.new_seq_lens.tolist()
        for r in range(B):
            got = lget(cache, b.slots(r, 0, done[r]))
            assert np.array_equal(got[0], want[r][0]) and np.array_equal(got[1], want[r][1])
            done[r] = min(done[r], limit[r] - gamma)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_latent_calls_in_a_graph(kind):
    """Captured once and replayed with new inputs in place, with eager work between: the
    eager results every time."""
    say(f"latent graph {kind}")
    H, n, L, gamma, dt = 6, 64, 512, 4, torch.bfloat16
    b = Batch(5, [5, 2, 4], [60, 200, 3], gamma, 16, True)
    cache, ql, qr = latent_setup(b, kind, H, L)
    kv = make_cache(kind, b.nb, 2, 16, 64)
    for t in (ql, qr):
        t[int(b.cu[-1]):] = 0
    cu, pre, table = b.args()
    par = b.par()
    x = typed(b.rng, (b.rows, L + R), dt).to(DEV)
    q = typed(b.rng, (b.rows, H, n + R), dt).to(DEV)
    w = typed(b.rng, (H, 2 * n, L), dt, L ** -0.5).to(DEV)
    qkv = typed(b.rng, (b.rows, 8, 64), dt).to(DEV)
    pos = i32(b.rng.integers(0, 300, (3, b.rows)))
    rope = up(turns(300, R))
    keys = sum(b.ctx) + sum(b.lens)
    ap = dv.alloc_latent_append_outputs(b.rows, H, cache)
    at_ = dv.alloc_latent_attention_outputs(b.B, gamma, b.rows, H, cache)
    pf = dv.alloc_latent_prefill_outputs(b.B, b.rows, keys, H, n, cache)
    rd = dv.alloc_latent_read_outputs(b.rows, cache)
    ka, kr = dv.alloc_append_outputs(b.rows, 4, kv), dv.alloc_kv_read_outputs(b.rows, kv)
    outs = [ap.q_rope, at_.out, pf.out, rd.latent_out, rd.rope_out, ka.q_out, kr.k_out, kr.v_out]

    def step():
        dv.dspark_latent_append(b.B, x, b.rows, cu, pre, table, cache, ap, q_rope=qr, rope=rope,
                                gamma=gamma, tree_parents=par)
        dv.dspark_latent_attention(b.B, gamma, ql, ap.q_rope, b.rows, cu, pre, table, cache, 0.05,
                                   at_, tree_parents=par)
        dv.dspark_latent_prefill(b.B, q, w[:, :n], w[:, n:], b.rows, keys, cu, pre, table, cache,
                                 0.07, pf)
        dv.dspark_latent_read(b.B, b.rows, cu, pre, table, cache, rd)
        dv.dspark_kv_append_axes(b.B, qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], b.rows, cu, pre, pos,
                                 [i % 3 for i in range(32)], table, kv, ka, rope)
        dv.dspark_kv_read(b.B, b.rows, cu, pre, table, kv, kr)

    for t in outs:
        t.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        for t in (x, q, ql, qr, qkv):
            t.copy_(typed(np.random.default_rng(50 + i), tuple(t.shape), dt))
        pos.copy_(i32(np.random.default_rng(i).integers(0, 300, (3, b.rows))))
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in outs]
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for k, (t, y) in enumerate(zip(outs, want)):
            assert torch.equal(t, y), (i, k)
        torch.randn(1 << 20, device=DEV).sum().item()


def test_latent_calls_on_two_streams():
    """Two steps at once, each with its own workspace, and a stream of the caller's."""
    say("latent two streams")
    H, L, gamma = 16, 512, 4
    b = Batch(5, [5, 2, 4], [1600, 200, 3], gamma, 16, True)
    one = latent_setup(b, "bf16", H, L, 1)
    two = latent_setup(b, "bf16", H, L, 2)
    want = []
    for c, ql, qr in (one, two):
        o = dv.alloc_latent_attention_outputs(b.B, gamma, b.rows, H, c)
        dv.dspark_latent_attention(b.B, gamma, ql, qr, b.rows, *b.args(), c, 0.05, o, tree_parents=b.par())
        torch.cuda.synchronize()
        want.append(o.out[:int(b.cu[-1])].clone())
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [dv.alloc_latent_attention_outputs(b.B, gamma, b.rows, H, c[0]) for c in (one, two)]
    args, par = b.args(), b.par()
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (c, ql, qr), o in zip(streams, (one, two), outs):
            dv.dspark_latent_attention(b.B, gamma, ql, qr, b.rows, *args, c, 0.05, o, tree_parents=par,
                                       stream=s)
    torch.cuda.synchronize()
    for o, y in zip(outs, want):
        assert torch.equal(o.out[:int(b.cu[-1])], y)


@pytest.mark.parametrize("kind,L", [("bf16", 512), ("e4m3", 512)])
def test_pages_beyond_four_gigabytes(kind, L):
    """Page offsets past 2^32 bytes."""
    say(f"pages beyond 4 GB {kind}")
    page = 256
    per = page * L * (1 if kind == "e4m3" else 2)
    nb = (1 << 32) // per + 40
    b = Batch(3, [3, 2], [300, 40], 2, page, False)
    shift = nb - b.nb
    cache = make_latent(kind, nb, page, L)
    b.table = np.where(b.table >= 0, b.table + shift, b.table)
    rng = np.random.default_rng(0)
    for r in range(b.B):
        T = b.ctx[r] + b.lens[r]
        lput(cache, b.slots(r, 0, T), rng.normal(0, 1, (T, L)), rng.normal(0, 1, (T, R)))
    dt = TYPES[kind][1]
    x = typed(rng, (b.rows, L + R), dt).to(DEV)
    cu, pre, table = b.args()
    ap = dv.alloc_latent_append_outputs(b.rows, 0, cache)
    dv.dspark_latent_append(b.B, x, b.rows, cu, pre, table, cache, ap)
    rd = dv.alloc_latent_read_outputs(b.rows, cache)
    dv.dspark_latent_read(b.B, b.rows, cu, pre, table, cache, rd)
    n = int(b.cu[-1])
    want = f64(x[:n, :L])
    torch.cuda.synchronize()
    assert np.array_equal(f64(rd.latent_out[:n]), oracle.latent_e4m3(want) if kind == "e4m3" else want)
    H = 3
    ql, qr = typed(rng, (b.rows, H, L), dt).to(DEV), typed(rng, (b.rows, H, R), dt).to(DEV)
    o = dv.alloc_latent_attention_outputs(b.B, 2, b.rows, H, cache, lse=True)
    o.out.fill_(-7)
    o.lse.fill_(-7)
    dv.dspark_latent_attention(b.B, 2, ql, qr, b.rows, cu, pre, table, cache, 0.05, o)
    torch.cuda.synchronize()
    latent_check(b, kind, H, L, 0.05, cache, ql, qr, o)
    keys = sum(b.ctx) + sum(b.lens)
    q = typed(rng, (b.rows, H, 64 + R), dt).to(DEV)
    w = typed(rng, (H, 128, L), dt, L ** -0.5).to(DEV)
    p = dv.alloc_latent_prefill_outputs(b.B, b.rows, keys, H, 64, cache, lse=True)
    p.out.fill_(-7)
    p.lse.fill_(-7)
    dv.dspark_latent_prefill(b.B, q, w[:, :64], w[:, 64:], b.rows, keys, cu, pre, table, cache, 0.08, p)
    torch.cuda.synchronize()
    prefill_check(b, kind, H, 64, L, 0.08, cache, q, w[:, :64], w[:, 64:], p)


def test_latent_calls_without_requests_or_rows():
    say("latent calls without requests")
    c = make_latent("bf16", 2, 16, 256)
    kv = make_cache("bf16", 2, 1, 16, 64)
    for B, rows in ((0, 0), (0, 4), (2, 0)):
        cu, pre, table = i32([0] * (B + 1)), i32([0] * max(B, 1)), i32([[0]] * max(B, 1))
        x = torch.zeros(max(rows, 1), 256 + R, dtype=torch.bfloat16, device=DEV)
        q = torch.zeros(max(rows, 1), 2, 128, dtype=torch.bfloat16, device=DEV)
        a = dv.alloc_latent_append_outputs(max(rows, 1), 2, c)
        dv.dspark_latent_append(B, x, rows, cu, pre, table, c, a, q_rope=q[..., 64:])
        rd = dv.alloc_latent_read_outputs(max(rows, 1), c)
        dv.dspark_latent_read(B, rows, cu, pre, table, c, rd)
        p = dv.alloc_latent_prefill_outputs(B, rows, 8, 2, 64, c)
        w = torch.zeros(2, 64, 256, dtype=torch.bfloat16, device=DEV)
        if rows == 0:
            p = p._replace(out=torch.zeros(1, 2, 64, dtype=torch.bfloat16, device=DEV))
        dv.dspark_latent_prefill(B, q, w, w, rows, 8, cu, pre, table, c, 0.1, p)
        ql = torch.zeros(max(rows, 1), 2, 256, dtype=torch.bfloat16, device=DEV)
        o = dv.alloc_latent_attention_outputs(B, 1, max(rows, 1), 2, c)
        dv.dspark_latent_attention(B, 1, ql, q[..., 64:], rows, cu, pre, table, c, 0.1, o)
        ka = dv.alloc_append_outputs(max(rows, 1), 2, kv)
        z = torch.zeros(max(rows, 1), 4, 64, dtype=torch.bfloat16, device=DEV)
        dv.dspark_kv_append_axes(B, z[:, :2], z[:, 2:3], z[:, 3:], rows, cu, pre,
                                 i32([[0] * max(rows, 1)]), [0] * 16, table, kv, ka,
                                 torch.zeros(3, 32, device=DEV))
        torch.cuda.synchronize()
        want = [0, dv.DATA_BAD_LENS if B else 0]  # a request of the verify step has a row
        assert o.attention_meta.tolist() == want
        for m in (a.append_meta, rd.read_meta, p.attention_meta, ka.append_meta):
            assert m.tolist() == [0, 0]
