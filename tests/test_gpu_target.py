"""GPU tests of the target pass (cache append and read, tree attention, tree
accept, commit) through the C ABI, against the float64 oracle.

Tolerances, with u the half step of the output type (2^-8 bfloat16, 2^-11
float16, relative to the value) and w = 2^-24 that of float32:

* Whole numbers, moved bytes, values and exponents of 8-bit rows that no
  arithmetic precedes: equal.
* Rows with norm and rotation: u |y| for the one rounding, and for float32
  (D + 16) w (|a| + |b|) with a, b the pair's elements: the sum of squares
  errs by at most its number of terms, each further operation by w. Below 2^-14
  a float16 has steps of 2^-24, so there the rounding errs by up to 2^-25.
  In 8 bits: half a step of the value, 2^-4 |y| or 2^-10 of the row's power of
  two, and the float32 part.
* Attention: out = sum w_k v_k. The weights round to the query type (u relative,
  and 2^-25 absolute where float16 goes subnormal, against a sum of at least
  1), their scores err by (D + 16) w times scale * sum |q||k|, float32 sums of
  n terms by n w, the output rounds once:
  u |out| + (u + 2 t + (n + 32) w) sum w_k |v_k| + n 2^-25 max |v| (float16).
"""

import numpy as np
import pytest
import torch

import dspark_verify_scheduling_amd as dv
import oracle
from _gpu import DEV, say, up

pytestmark = pytest.mark.gpu

TYPES = {"bf16": (dv.BF16, torch.bfloat16, 2.0 ** -8), "f16": (dv.F16, torch.float16, 2.0 ** -11),
         "e4m3": (dv.E4M3, torch.bfloat16, 2.0 ** -8)}
W = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _need_gpu(hip):
    return hip


def i32(a):
    return up(np.asarray(a, np.int32))


def f64(t):
    return t.detach().double().cpu().numpy()


def make_cache(kind, nb, hkv, page, D, layers=0, joint=False):
    """A cache whose every slot holds NaN."""
    code, dt, _ = TYPES[kind]
    lead = (layers,) if layers else ()
    if joint:  # keys and values interleaved page by page in one pool
        el = torch.float8_e4m3fn if kind == "e4m3" else dt
        pool = torch.empty(lead + (nb, 2, hkv, page, D), dtype=el, device=DEV)
        sc = torch.full(lead + (nb, 2, hkv, page), 120, dtype=torch.uint8, device=DEV)
        e8 = kind == "e4m3"
        c = dv.KvCache(pool[..., 0, :, :, :], pool[..., 1, :, :, :],
                       sc[..., 0, :, :] if e8 else None, sc[..., 1, :, :] if e8 else None)
    else:
        c = dv.alloc_kv_cache(nb, hkv, page, D, code, DEV, layers)
        pool = None
    for t in ((pool,) if joint else (c.k, c.v)):
        t.view(torch.uint8).fill_(0x7F) if kind == "e4m3" else t.fill_(float("nan"))
    if kind == "e4m3" and not joint:
        c.k_scale.fill_(120)
        c.v_scale.fill_(120)
    return c


def within(got, ref, bound, what):
    """|got - ref| <= bound, naming the worst element."""
    err = np.abs(np.asarray(got) - ref)
    if not np.all(err <= bound):
        i = np.unravel_index(np.nanargmax(np.where(np.isnan(err), np.inf, err - bound)), err.shape)
        pytest.fail(f"{what} at {i}: got {np.asarray(got)[i]!r}, want {ref[i]!r}, off by {err[i]:.4g}, "
                    f"bound {np.broadcast_to(bound, err.shape)[i]:.4g}")


def bits(t):
    return t.contiguous().view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def put(cache, slots, k, v, layer=None):
    """Host float32 rows k, v [n, hkv, D] into (page, offset) slots."""
    pg = torch.tensor([s[0] for s in slots], device=DEV)
    of = torch.tensor([s[1] for s in slots], device=DEV)
    for name, x in (("k", k), ("v", v)):
        pool, sc = getattr(cache, name), getattr(cache, name + "_scale")
        if layer is not None:
            pool, sc = pool[layer], None if sc is None else sc[layer]
        if sc is not None:
            e = oracle.e4m3_exponent(np.asarray(x, np.float64))
            y = np.ldexp(oracle.e4m3_round(np.asarray(x, np.float64), e), -e[..., None])
            codes = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).to(DEV)
            pool.view(torch.uint8)[pg, :, of] = codes
            sc[pg, :, of] = torch.from_numpy((e + 127).astype(np.uint8)).to(DEV)
        else:
            pool[pg, :, of] = torch.from_numpy(np.asarray(x, np.float32)).to(DEV).to(pool.dtype)


def get(cache, slots, name, layer=None):
    """Rows [n, hkv, D] of the cache as float64."""
    pg = torch.tensor([s[0] for s in slots], device=DEV)
    of = torch.tensor([s[1] for s in slots], device=DEV)
    pool, sc = getattr(cache, name), getattr(cache, name + "_scale")
    if layer is not None:
        pool, sc = pool[layer], None if sc is None else sc[layer]
    if sc is None:
        return f64(pool[pg, :, of])
    codes = pool.view(torch.uint8)[pg, :, of].cpu().numpy()
    e = sc[pg, :, of].cpu().numpy().astype(np.int64) - 127
    return np.ldexp(oracle.e4m3_values()[codes], e[..., None])


class Batch:
    """Requests with their rows, trees and scattered pages."""

    def __init__(self, seed, lens, ctx, gamma, page, tree, pad=3, extra_pages=2):
        rng = self.rng = np.random.default_rng(seed)
        self.B, self.gamma, self.page = len(lens), gamma, page
        self.lens, self.ctx = list(lens), list(ctx)
        self.cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        self.rows = int(self.cu[-1]) + pad
        need = [-(-(c + n) // page) for c, n in zip(ctx, lens)]
        ids = rng.permutation(sum(need) + extra_pages)
        self.nb = len(ids)
        self.width = max(need) + 1
        self.table = np.full((self.B, self.width), -1, np.int32)  # unused entries are no page ids
        at = 0
        for r, n in enumerate(need):
            self.table[r, :n] = ids[at:at + n]
            at += n
        self.parents = None
        if tree:
            self.parents = np.full((self.B, gamma), -9, np.int32)  # entries past the rows do not count
            for r, n in enumerate(lens):
                for j in range(1, n):
                    self.parents[r, j - 1] = j - 1 if rng.random() < 0.4 else rng.integers(0, j)

    def slots(self, r, lo, hi):
        return [(int(self.table[r, i // self.page]), i % self.page) for i in range(lo, hi)]

    def args(self):
        return i32(self.cu), i32(self.ctx), i32(self.table)

    def par(self):
        return None if self.parents is None else i32(self.parents)

    def tree(self, r):
        return list(range(self.gamma)) if self.parents is None else self.parents[r]


# ------------------------------------------------------------------ append and read

APPEND = [
    # kind, lens, ctx, gamma, hq, hkv, D, page, tree, norm, rot, interleaved, joint
    ("bf16", [1], [0], 1, 1, 1, 64, 16, False, True, 64, False, False),
    ("bf16", [3, 1, 5], [15, 16, 0], 4, 6, 2, 128, 16, True, True, 128, False, True),
    ("f16", [5, 2, 9, 1], [31, 100, 7, 255], 8, 8, 8, 64, 32, True, False, 32, True, False),
    ("f16", [4, 4], [60, 3], 7, 10, 2, 256, 64, False, True, 0, False, False),
    ("e4m3", [2, 9, 1, 6], [14, 250, 0, 33], 8, 12, 3, 128, 16, True, True, 128, False, True),
    ("e4m3", [1, 65, 17], [1000, 7, 500], 64, 4, 4, 64, 256, True, True, 16, True, False),
    ("e4m3", [7], [129], 6, 16, 2, 256, 128, False, False, 64, False, False),
    ("bf16", [65], [1], 64, 5, 5, 128, 128, True, False, 0, False, False),
]


@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append(case):
    kind, lens, ctx, gamma, hq, hkv, D, page, tree, norm, rot, inter, joint = APPEND[case]
    say(f"append case {case}: {kind} lens={lens} ctx={ctx} D={D}")
    code, dt, u = TYPES[kind]
    b = Batch(case, lens, ctx, gamma, page, tree)
    rng = b.rng
    cache = make_cache(kind, b.nb, hkv, page, D, joint=joint)
    before = [bits(t).clone() for t in (cache.k, cache.v)]
    qkv = torch.from_numpy(rng.normal(0, 2, (b.rows, hq + 2 * hkv, D)).astype(np.float32)).to(dt)
    qkv[0, hq:] = 0  # a row of zeros
    host = qkv.double().numpy()
    qkv = qkv.to(DEV)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    qw = kw = None
    if norm:
        qw = torch.from_numpy(rng.normal(1, 0.2, D).astype(np.float32)).to(dt).to(DEV)
        kw = torch.from_numpy(rng.normal(1, 0.2, D).astype(np.float32)).to(dt).to(DEV)
    rope = None
    if rot:
        n_pos = max(c + n for c, n in zip(ctx, lens))
        ang = np.arange(n_pos)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
        rope = up(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32))
    out = dv.alloc_append_outputs(b.rows, hq, cache)
    out.q_out.fill_(-7)
    cu, pre, table = b.args()
    dv.dspark_kv_append(b.B, gamma, q, k, v, b.rows, cu, pre, table, cache, out, q_weight=qw,
                        k_weight=kw, eps=1e-5, rope=rope, rope_interleaved=inter,
                        tree_parents=b.par())
    torch.cuda.synchronize()
    assert out.append_meta.tolist() == [int(b.cu[-1]), 0]
    got_q = f64(out.q_out)
    table_h = None if rope is None else rope.cpu().numpy()
    written = []
    for r in range(b.B):
        slots = b.slots(r, ctx[r], ctx[r] + lens[r])
        written += slots
        gk, gv = get(cache, slots, "k"), get(cache, slots, "v")
        paths = oracle.tree_paths(b.tree(r), lens[r])
        for j in range(lens[r]):
            x = host[b.cu[r] + j]
            row = None if rope is None else table_h[ctx[r] + len(paths[j]) - 1]
            for h in range(hq + hkv):
                w = (qw if h < hq else kw) if norm else None
                w = None if w is None else f64(w)
                y = oracle.norm_rope(x[h], w, 1e-5, row, rot, inter)
                plain = np.abs(oracle.norm_rope(x[h], w, 1e-5, None, rot, inter))
                size = plain.copy()
                if rot:
                    p = np.arange(rot).reshape(-1, 2) if inter else np.arange(rot).reshape(2, -1).T
                    size[p] = plain[p].sum(1, keepdims=True)
                f32 = (D + 16) * W * size
                if h < hq or kind != "e4m3":
                    got = got_q[b.cu[r] + j, h] if h < hq else gk[j, h - hq]
                    within(got, y, u * np.abs(y) + 1.01 * f32 + (2.0 ** -25 if kind == "f16" else 1e-30),
                               (r, j, h))
                else:
                    e = oracle.e4m3_exponent(y[None])[0]
                    half = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** (e - 10))
                    within(gk[j, h - hq], y, half + 1.07 * f32, (r, j, h))
            xv = x[hq + hkv:]
            if kind == "e4m3":
                xv = oracle.e4m3_round(xv, oracle.e4m3_exponent(xv))
            assert np.array_equal(gv[j], xv), (r, j)
    assert bool((out.q_out[int(b.cu[-1]):] == -7).all())
    # every other slot is as it was
    for name, old in zip("kv", before):
        now = bits(getattr(cache, name)).clone()
        pg, of = torch.tensor(written, device=DEV).T
        now[pg, :, of] = old[pg, :, of]
        assert torch.equal(now.view(torch.uint8), old.view(torch.uint8))

    # read back, the rows and then other spans
    say(f"read case {case}")
    rd = dv.alloc_kv_read_outputs(b.rows, cache)
    for t in rd[:2]:
        t.fill_(-7)
    dv.dspark_kv_read(b.B, b.rows, cu, pre, table, cache, rd)
    torch.cuda.synchronize()
    assert rd.read_meta.tolist() == [int(b.cu[-1]), 0]
    for r in range(b.B):
        slots = b.slots(r, ctx[r], ctx[r] + lens[r])
        assert np.array_equal(f64(rd.k_out[b.cu[r]:b.cu[r + 1]]), get(cache, slots, "k"))
        assert np.array_equal(f64(rd.v_out[b.cu[r]:b.cu[r + 1]]), get(cache, slots, "v"))
    assert bool((rd.k_out[int(b.cu[-1]):] == -7).all())


def test_append_in_place_and_nonfinite():
    """q_out may be q; NaN and infinite elements become NaN in 8 bits, and the
    exponent comes from the finite ones; values beyond the range saturate."""
    say("append in place, non-finite")
    D, hq, hkv, page = 64, 2, 2, 16
    b = Batch(7, [4], [3], 4, page, False, pad=0)
    cache = make_cache("e4m3", b.nb, hkv, page, D)
    x = np.random.default_rng(0).normal(0, 1, (4, hq + 2 * hkv, D)).astype(np.float32)
    x[0, hq, 5] = np.nan
    x[0, hq + hkv, 7] = np.inf
    x[1, hq + hkv, :] = -np.inf
    x[2, hq + hkv + 1, 3] = 3.3e38
    x[3, hq + hkv, :] = 1e-38
    t = torch.from_numpy(x).to(torch.bfloat16)
    x = t.double().numpy()
    t = t.to(DEV)
    q = t[:, :hq].contiguous()
    keep = q.clone()
    out = dv.AppendOutputs(q, torch.empty(2, dtype=torch.int32, device=DEV))
    cu, pre, table = b.args()
    dv.dspark_kv_append(1, 4, q, t[:, hq:hq + hkv], t[:, hq + hkv:], 4, cu, pre, table, cache, out)
    torch.cuda.synchronize()
    assert torch.equal(q, keep)  # neither norm nor rotation
    slots = b.slots(0, 3, 7)
    for name, y in (("k", x[:, hq:hq + hkv]), ("v", x[:, hq + hkv:])):
        ref = oracle.e4m3_round(y, oracle.e4m3_exponent(y))
        assert np.array_equal(get(cache, slots, name), ref, equal_nan=True), name


@pytest.mark.parametrize("kind,hkv,D,page", [("bf16", 1, 64, 16), ("f16", 3, 256, 32),
                                             ("e4m3", 8, 128, 64), ("e4m3", 5, 64, 256)])
def test_read_spans(kind, hkv, D, page):
    """Spans of any length, none among them, and a batch longer than one
    workgroup's search."""
    say(f"read spans {kind} D={D} page={page}")
    rng = np.random.default_rng(D + page)
    n = [0, 1, 40, 0, 17, 300] + rng.integers(0, 9, 90).tolist()
    st = [0, 15, 3, 9, 0, 77] + rng.integers(0, 40, 90).tolist()
    b = Batch(1, [max(1, x) for x in n], st, 4, page, False)
    b.cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    cache = make_cache(kind, b.nb, hkv, page, D)
    rows = int(b.cu[-1])
    for r in range(b.B):
        if n[r]:
            put(cache, b.slots(r, st[r], st[r] + n[r]), *rng.normal(0, 1, (2, n[r], hkv, D)))
    rd = dv.alloc_kv_read_outputs(rows, cache)
    dv.dspark_kv_read(b.B, rows, i32(b.cu), i32(st), i32(b.table), cache, rd)
    torch.cuda.synchronize()
    assert rd.read_meta.tolist() == [rows, 0]
    for name, t in (("k", rd.k_out), ("v", rd.v_out)):
        t = f64(t)
        assert not np.isnan(t).any()
        for r in range(b.B):
            if n[r]:
                want = get(cache, b.slots(r, st[r], st[r] + n[r]), name)
                assert np.array_equal(t[b.cu[r]:b.cu[r + 1]], want)


# ------------------------------------------------------------------ attention

def attention_check(b, kind, hq, hkv, D, scale, seed=0, joint=False, spread=1.0, repeat=1):
    code, dt, u = TYPES[kind]
    rng = np.random.default_rng(seed)
    cache = make_cache(kind, b.nb, hkv, b.page, D, joint=joint)
    for r in range(b.B):
        T = b.ctx[r] + b.lens[r]
        put(cache, b.slots(r, 0, T), *rng.normal(0, spread, (2, T, hkv, D)).astype(np.float32))
    q = torch.from_numpy(rng.normal(0, 1, (b.rows, hq, D)).astype(np.float32)).to(dt).to(DEV)
    q[int(b.cu[-1]):] = float("nan")
    outs = []
    o = dv.alloc_attention_outputs(b.B, b.gamma, b.rows, hq, cache, lse=True)
    cu, pre, table = b.args()
    par = b.par()
    for _ in range(repeat):
        o.out.fill_(-7)
        o.lse.fill_(-7)
        o.workspace.fill_(0xFF)  # its contents do not matter
        dv.dspark_tree_attention(b.B, b.gamma, q, b.rows, cu, pre, table, cache, scale, o,
                                 tree_parents=par)
        torch.cuda.synchronize()
        outs.append(o.out.clone())
    for x in outs[1:]:
        assert torch.equal(x, outs[0])
    assert o.attention_meta.tolist() == [int(b.cu[-1]), 0]
    got, lse, qh = f64(o.out), f64(o.lse), f64(q)
    for r in range(b.B):
        T = b.ctx[r] + b.lens[r]
        k, v = (get(cache, b.slots(r, 0, T), n).transpose(1, 0, 2) for n in "kv")
        c0, c1 = b.cu[r], b.cu[r + 1]
        ref, rl, mean_abs, top = oracle.tree_attention(qh[c0:c1], k, v, b.ctx[r],
                                                       None if b.parents is None else b.parents[r],
                                                       scale)
        t = (D + 16) * W * top[..., None] + 2 * W
        bound = u * np.abs(ref) + (u + 2 * t + (T + 32) * W) * mean_abs
        if kind == "f16":
            bound += T * 2.0 ** -25 * np.abs(v).max()
        within(got[c0:c1], ref, bound, f"request {r}")
        lb = t[..., 0] + (T + 32) * W + 4 * W * np.abs(rl)
        within(lse[c0:c1], rl, lb, f"lse of request {r}")
    assert bool((o.out[int(b.cu[-1]):] == -7).all()) and bool((o.lse[int(b.cu[-1]):] == -7).all())


ATTN = [
    # kind, lens, ctx, gamma, hq, hkv, D, page, tree, joint
    ("bf16", [1], [0], 1, 1, 1, 64, 16, False, False),  # one token, no context
    ("bf16", [1, 1, 1], [15, 16, 17], 1, 2, 1, 128, 16, False, False),
    ("f16", [1], [127], 1, 4, 4, 256, 32, False, False),
    ("bf16", [9, 1, 4], [700, 31, 0], 8, 8, 2, 128, 64, False, True),  # chains
    ("f16", [9, 5, 2, 7], [33, 250, 96, 511], 8, 7, 1, 64, 16, True, False),  # odd groups
    ("e4m3", [9, 3, 1], [127, 128, 1000], 8, 16, 2, 128, 32, True, True),
    ("e4m3", [17, 2, 17], [63, 5, 400], 16, 10, 2, 64, 128, True, False),
    ("e4m3", [4, 6], [257, 64], 6, 8, 1, 256, 16, True, False),
    ("bf16", [65, 1, 33], [100, 2000, 0], 64, 16, 2, 128, 16, True, False),  # the largest trees
    ("f16", [65], [1500], 64, 40, 5, 64, 256, True, False),
    ("bf16", [65, 64], [40, 300], 64, 6, 3, 256, 64, False, False),  # the longest chains
    ("bf16", [13], [5000], 12, 64, 1, 64, 32, True, False),  # a group of 64
    ("bf16", [2] * 150, list(range(150)), 2, 4, 2, 64, 16, True, False),  # many short ones
    ("e4m3", [1, 9, 2], [9001, 4100, 7000], 8, 8, 2, 128, 64, True, False),  # long, split keys
    ("f16", [3], [20011], 4, 8, 1, 128, 16, True, False),
]


@pytest.mark.parametrize("case", range(len(ATTN)))
def test_attention(case):
    kind, lens, ctx, gamma, hq, hkv, D, page, tree, joint = ATTN[case]
    say(f"attention case {case}: {kind} lens={lens[:6]} ctx={ctx[:6]} hq={hq} hkv={hkv} D={D}")
    b = Batch(case, lens, ctx, gamma, page, tree)
    attention_check(b, kind, hq, hkv, D, D ** -0.5, seed=case, joint=joint, repeat=2)


@pytest.mark.parametrize("scale,spread", [(4.0, 2.0), (-0.2, 1.0), (0.0, 1.0), (1e-3, 100.0)])
def test_attention_scales(scale, spread):
    """Weights that all sit on one key, a negative and a zero scale, large values."""
    say(f"attention scale={scale} spread={spread}")
    b = Batch(5, [9, 4], [300, 77], 8, 32, True)
    attention_check(b, "bf16", 8, 2, 64, scale, seed=9, spread=spread)


@pytest.mark.parametrize("kind", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_ignores_what_a_row_does_not_see(kind, D):
    """NaN and infinities in the keys and values of a sibling's row reach the
    rows that see it and no other."""
    say(f"attention masked non-finite {kind} D={D}")
    _, dt, u = TYPES[kind]
    b = Batch(3, [5, 1], [61, 30], 6, 16, True)
    b.parents[0, :4] = [0, 0, 1, 2]  # 0-1-3, 0-2-4
    hq, hkv = 4, 2
    rng = np.random.default_rng(1)
    cache = make_cache(kind, b.nb, hkv, 16, D)
    for r in range(2):
        T = b.ctx[r] + b.lens[r]
        k, v = rng.normal(0, 1, (2, T, hkv, D)).astype(np.float32)
        if r == 0:
            k[61 + 1, :, 3] = np.nan  # row 1: seen by rows 1 and 3
            v[61 + 1, :, D - 1] = np.inf if kind != "e4m3" else np.nan
        put(cache, b.slots(r, 0, T), k, v)
    q = torch.from_numpy(rng.normal(0, 1, (b.rows, hq, D)).astype(np.float32)).to(dt).to(DEV)
    o = dv.alloc_attention_outputs(2, 6, b.rows, hq, cache)
    cu, pre, table = b.args()
    dv.dspark_tree_attention(2, 6, q, b.rows, cu, pre, table, cache, 0.1, o, tree_parents=b.par())
    torch.cuda.synchronize()
    bad = torch.isnan(o.out[:6].float()).flatten(1)
    assert bad.any(1).tolist() == [False, True, False, True, False, False]
    # values alone: the key is finite, one value is not
    put(cache, b.slots(0, 62, 63), *np.ones((2, 1, hkv, D), np.float32))
    v = np.ones((1, hkv, D), np.float32)
    v[0, :, 5] = np.nan
    v[0, :, 6] = np.inf
    put(cache, b.slots(0, 62, 63), np.ones((1, hkv, D), np.float32), v)
    dv.dspark_tree_attention(2, 6, q, b.rows, cu, pre, table, cache, 0.1, o, tree_parents=b.par())
    torch.cuda.synchronize()
    x = o.out[:6].float()
    assert torch.isnan(x[1, :, 5]).all() and torch.isnan(x[3, :, 5]).all()
    if kind != "e4m3":
        assert torch.isinf(x[1, :, 6]).all() and torch.isinf(x[3, :, 6]).all()
    ok = torch.ones(D, dtype=torch.bool)
    ok[5:7] = False
    assert torch.isfinite(x[:, :, ok.to(DEV)]).all()
    assert torch.isfinite(x[[0, 2, 4, 5]]).all()


def test_attention_all_scores_minus_infinity_or_pages_missing():
    say("attention empty rows")
    D, page = 64, 16
    b = Batch(2, [2, 3], [20, 3], 4, page, False)
    cache = make_cache("bf16", b.nb, 1, page, D)
    rng = np.random.default_rng(0)
    for r in range(2):
        T = b.ctx[r] + b.lens[r]
        put(cache, b.slots(r, 0, T), *rng.normal(0, 1, (2, T, 1, D)).astype(np.float32))
    q = torch.ones(b.rows, 2, D, dtype=torch.bfloat16, device=DEV)
    o = dv.alloc_attention_outputs(2, 4, b.rows, 2, cache, lse=True)
    table = b.table.copy()
    table[1, 0] = b.nb  # request 1's only page does not exist
    table[0, 1] = -1  # of request 0's two pages the second
    dv.dspark_tree_attention(2, 4, q, b.rows, i32(b.cu), i32(b.ctx), i32(table), cache, 0.125, o)
    torch.cuda.synchronize()
    assert o.attention_meta.tolist() == [5, oracle.DATA_BAD_PAGE]
    assert bool((o.out[2:5] == 0).all()) and bool((o.lse[2:5] == -float("inf")).all())
    k, v = (get(cache, b.slots(0, 0, 16), n).transpose(1, 0, 2) for n in "kv")
    ref, *_ = oracle.tree_attention(f64(q[:1]), k, v, 15, None, 0.125)  # what is left of the context
    assert np.allclose(f64(o.out[0]), ref[0], atol=2e-2) and np.allclose(f64(o.out[1]), ref[0], atol=2e-2)
    # every score -infinity: nothing is left of the row
    put(cache, b.slots(1, 0, 6), np.full((6, 1, D), -np.inf, np.float32), np.ones((6, 1, D), np.float32))
    dv.dspark_tree_attention(2, 4, q, b.rows, *b.args(), cache, 0.125, o)
    torch.cuda.synchronize()
    assert bool((o.out[2:5] == 0).all()) and bool((o.lse[2:5] == -float("inf")).all())


# ------------------------------------------------------------------ data errors

def test_malformed_requests_are_left_out():
    say("malformed requests")
    D, page, gamma = 64, 16, 4
    b = Batch(4, [2, 3, 1, 4, 2, 1], [5, 40, 9, 20, 3, 8], gamma, page, True)
    cache = make_cache("bf16", b.nb, 1, page, D)
    rng = np.random.default_rng(0)
    for r in range(b.B):
        T = b.ctx[r] + b.lens[r]
        put(cache, b.slots(r, 0, T), *rng.normal(0, 1, (2, T, 1, D)).astype(np.float32))
    q = torch.from_numpy(rng.normal(0, 1, (b.rows, 2, D)).astype(np.float32)).bfloat16().to(DEV)
    k = q[:, :1].contiguous()
    o = dv.alloc_attention_outputs(b.B, gamma, b.rows, 2, cache)
    ap = dv.alloc_append_outputs(b.rows, 2, cache)
    parents, ctx, table = b.parents.copy(), list(b.ctx), b.table.copy()
    parents[1, 1] = 2  # row 2 its own parent
    ctx[2] = -1
    ctx[3] = b.width * page - 2  # ends beyond the table row
    L, T, P = oracle.DATA_BAD_LENS, oracle.DATA_BAD_TREE, oracle.DATA_BAD_PAGE
    good = [r for r in range(b.B) if r not in (1, 2, 3)]
    was = bits(cache.k).clone()
    for name in ("append", "attention"):
        if name == "append":
            ap.q_out.fill_(-7)
            dv.dspark_kv_append(b.B, gamma, q, k, k, b.rows, i32(b.cu), i32(ctx), i32(table), cache,
                                ap, tree_parents=i32(parents))
            got, meta = ap.q_out, ap.append_meta
        else:
            o.out.fill_(-7)
            dv.dspark_tree_attention(b.B, gamma, q, b.rows, i32(b.cu), i32(ctx), i32(table), cache,
                                     0.1, o, tree_parents=i32(parents))
            got, meta = o.out, o.attention_meta
        torch.cuda.synchronize()
        assert meta.tolist() == [int(b.cu[-1]), L | T | P], name
        for r in range(b.B):
            same = bool((got[int(b.cu[r]):int(b.cu[r + 1])] == -7).all())
            assert same == (r not in good), (name, r)
    for r in (1, 2, 3):
        for pg, of in b.slots(r, 0, b.ctx[r] + b.lens[r]):
            assert torch.equal(bits(cache.k)[pg, :, of], was[pg, :, of])
    # a total beyond the buffer: the requests inside it still run
    o.out.fill_(-7)
    rows = int(b.cu[2])
    dv.dspark_tree_attention(b.B, gamma, q, rows, i32(b.cu), i32(b.ctx), i32(b.table), cache, 0.1, o,
                             tree_parents=b.par())
    torch.cuda.synchronize()
    assert o.attention_meta.tolist() == [int(b.cu[-1]), L]
    assert not bool((o.out[:rows] == -7).all(-1).any()) and bool((o.out[rows:] == -7).all())
    # lengths out of order, or longer than gamma + 1
    cu = b.cu.copy()
    cu[2], cu[5] = 1, cu[5] - 2
    o.out.fill_(-7)
    dv.dspark_tree_attention(b.B, gamma, q, b.rows, i32(cu), i32(b.ctx), i32(b.table), cache, 0.1, o)
    rd = dv.alloc_kv_read_outputs(b.rows, cache)
    dv.dspark_kv_read(b.B, b.rows, i32(cu), i32(b.ctx), i32(b.table), cache, rd)
    torch.cuda.synchronize()
    assert o.attention_meta.tolist()[1] & L and rd.read_meta.tolist()[1] & L


def test_positions_beyond_the_rotation_table_and_bad_append_pages():
    say("append beyond the table")
    D, page, gamma = 64, 16, 4
    b = Batch(6, [5, 3], [14, 2], gamma, page, True)
    b.parents[0, :4] = [0, 1, 0, 2]  # depths 0 1 2 1 3
    cache = make_cache("bf16", b.nb, 1, page, D)
    q = torch.ones(b.rows, 1, D, dtype=torch.bfloat16, device=DEV)
    ap = dv.alloc_append_outputs(b.rows, 1, cache)
    ap.q_out.fill_(-7)
    rope = torch.ones(16, 32, device=DEV)  # positions 0..15: rows of depth > 1 of request 0 lie beyond
    cu, pre, table = b.args()
    dv.dspark_kv_append(2, gamma, q, q, q, b.rows, cu, pre, table, cache, ap, rope=rope,
                        tree_parents=b.par())
    torch.cuda.synchronize()
    assert ap.append_meta.tolist() == [8, oracle.DATA_BAD_POS]
    left = (ap.q_out[:5, 0] == -7).all(-1).tolist()
    assert left == [False, False, True, False, True]
    got = [bool(torch.isnan(cache.k[pg, 0, of]).all()) for pg, of in b.slots(0, 14, 19)]
    assert got == left
    bad = b.table.copy()
    bad[0, 1] = 10 ** 6
    ap.q_out.fill_(-7)
    dv.dspark_kv_append(2, gamma, q, q, q, b.rows, cu, pre, i32(bad), cache, ap)
    rd = dv.alloc_kv_read_outputs(b.rows, cache)
    rd.k_out.fill_(-7)
    dv.dspark_kv_read(2, b.rows, cu, pre, i32(bad), cache, rd)
    torch.cuda.synchronize()
    assert ap.append_meta.tolist() == [8, oracle.DATA_BAD_PAGE] == rd.read_meta.tolist()
    assert (ap.q_out[:5, 0] == -7).all(-1).tolist() == [False, False, True, True, True]
    assert (rd.k_out[:5, 0] == -7).all(-1).tolist() == [False, False, True, True, True]


def test_empty_batches():
    say("empty batches")
    cache = make_cache("bf16", 2, 1, 16, 64)
    cu = i32([0])
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    tab = torch.empty(0, 1, dtype=torch.int32, device=DEV)
    q = torch.empty(1, 1, 64, dtype=torch.bfloat16, device=DEV)
    ap = dv.alloc_append_outputs(1, 1, cache)
    dv.dspark_kv_append(0, 3, q, q, q, 1, cu, none, tab, cache, ap)
    o = dv.alloc_attention_outputs(0, 3, 1, 1, cache)
    dv.dspark_tree_attention(0, 3, q, 1, cu, none, tab, cache, 1.0, o)
    rd = dv.alloc_kv_read_outputs(1, cache)
    dv.dspark_kv_read(0, 1, cu, none, tab, cache, rd)
    cm = torch.empty(2, dtype=torch.int32, device=DEV)
    dv.dspark_kv_commit(0, 3, none, none, none, tab, cache, cm)
    torch.cuda.synchronize()
    for m in (ap.append_meta, o.attention_meta, rd.read_meta, cm):
        assert m.tolist() == [0, 0]


def test_binding_refuses_on_the_gpu():
    cache = make_cache("bf16", 2, 2, 16, 64, layers=3)
    cm = torch.empty(2, dtype=torch.int32, device=DEV)
    one = i32([0])
    tab = i32([[0]])
    o = dv.alloc_attention_outputs(1, 1, 2, 2, cache)
    q = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="one layer"):
        dv.dspark_tree_attention(1, 1, q, 2, i32([0, 1]), one, tab, cache, 1.0, o)
    lay = cache.layer(1)
    assert lay.num_layers == 1 and cache.num_layers == 3
    with pytest.raises(TypeError):
        dv.dspark_tree_attention(1, 1, q.float(), 2, i32([0, 1]), one, tab, lay, 1.0, o)
    with pytest.raises(ValueError, match="dense"):
        dv.dspark_tree_attention(1, 1, torch.zeros(2, 2, 128, dtype=torch.bfloat16, device=DEV)[..., ::2],
                                 2, i32([0, 1]), one, tab, lay, 1.0, o)
    with pytest.raises(ValueError, match="current device"):
        dv.dspark_tree_attention(1, 1, q, 2, i32([0, 1]).cpu(), one, tab, lay, 1.0, o)
    with pytest.raises(ValueError):
        dv.dspark_kv_commit(1, 3, i32([0, 1]), one, one, tab, cache, cm)  # path_rows too short
    with pytest.raises(dv.DsparkError):
        dv.dspark_tree_attention(1, 65, q, 2, i32([0, 1]), one, tab, lay, 1.0, o)


# ------------------------------------------------------------------ tree accept

def tree_logits(rng, b, V, ld, dt, hit=0.7):
    x = rng.normal(0, 2, (b.rows, ld)).astype(np.float32)
    if dt == dv.BF16:
        bf = (x.view(np.uint32) >> 16).astype(np.uint16)
        am = oracle.row_argmax((bf.astype(np.uint32) << 16).view(np.float32)[:, :V])
        x = bf
    else:
        am = oracle.row_argmax(x[:, :V])
    drafts = rng.integers(0, V, (b.B, b.gamma)).astype(np.int32)
    for r in range(b.B):
        for j in range(1, b.lens[r]):
            if rng.random() < hit:
                drafts[r, j - 1] = am[b.cu[r] + int(b.tree(r)[j - 1])]
    return x, drafts


def run_tree_accept(b, V, ld, dt, x, drafts, prefix, max_rows=None):
    rows = b.rows if max_rows is None else max_rows
    t = torch.from_numpy(x.view(np.int16)).to(DEV).view(torch.bfloat16) if dt == dv.BF16 else up(x)
    o = dv.alloc_tree_accept_outputs(b.B, b.gamma, rows, V, dt, DEV)
    o.row_argmax.fill_(-7)
    dv.dspark_tree_accept(b.B, b.gamma, V, dt, t, ld, rows, i32(b.cu), i32(drafts), b.par(),
                          i32(prefix), o)
    torch.cuda.synchronize()
    ref = oracle.tree_accept(b.B, b.gamma, x[:, :V], "bf16" if dt == dv.BF16 else "f32", b.cu,
                             drafts, b.parents, prefix, max_rows=rows)
    n = len(ref["row_argmax"])
    assert np.array_equal(o.row_argmax[:n].cpu().numpy(), ref["row_argmax"])
    assert bool((o.row_argmax[n:] == -7).all())
    for name, got in (("num_correct", o.num_correct), ("bonus", o.bonus), ("commit", o.commit_lens),
                      ("out_tokens", o.out_tokens), ("path_rows", o.path_rows),
                      ("new_seq", o.new_seq_lens), ("meta", o.accept_meta)):
        assert np.array_equal(got.cpu().numpy(), ref[name]), name
    return ref


@pytest.mark.parametrize("B,gamma,V,ld,dt", [
    (1, 1, 1, 8, dv.F32), (7, 5, 1001, 1008, dv.BF16), (40, 8, 32000, 32000, dv.F32),
    (5, 64, 700, 704, dv.BF16), (3, 64, 129280, 129280, dv.BF16), (200, 3, 257, 260, dv.F32)])
def test_tree_accept(B, gamma, V, ld, dt):
    say(f"tree accept B={B} gamma={gamma} V={V} dt={dt}")
    rng = np.random.default_rng(B * 100 + gamma)
    lens = rng.integers(1, gamma + 2, B).tolist()
    lens[-1] = gamma + 1
    b = Batch(B, lens, [4] * B, gamma, 16, True)
    x, drafts = tree_logits(rng, b, V, ld, dt)
    ref = run_tree_accept(b, V, ld, dt, x, drafts, rng.integers(0, 99, B))
    say(f"accepted {int(ref['num_correct'].sum())} of {sum(lens) - B}")


def test_tree_accept_chain_siblings_and_bad_trees():
    say("tree accept: chain, equal siblings, malformed")
    rng = np.random.default_rng(8)
    b = Batch(8, [5, 9, 1, 9, 4, 6], [4] * 6, 8, 16, False)
    x, drafts = tree_logits(rng, b, 300, 304, dv.F32, hit=0.9)
    ref = run_tree_accept(b, 300, 304, dv.F32, x, drafts, [1, 2, 3, 4, 5, 6])
    # the chain accept of the framework agrees
    a = dv.alloc_accept_outputs(6, 8, b.rows, 300, dv.F32, DEV)
    dv.dspark_accept(6, 8, 300, dv.F32, up(x), 304, b.rows, i32(b.cu), i32(drafts), i32([1, 2, 3, 4, 5, 6]), a)
    torch.cuda.synchronize()
    assert np.array_equal(a.num_correct.cpu().numpy(), ref["num_correct"])
    assert np.array_equal(a.bonus.cpu().numpy(), ref["bonus"])
    b = Batch(9, [5, 9, 1, 9, 4, 6], [4] * 6, 8, 16, True)
    x, drafts = tree_logits(rng, b, 300, 304, dv.F32, hit=0.9)
    b.parents[0, :4] = 0
    am = oracle.row_argmax(x[:, :300])
    drafts[0, :4] = am[0]  # four equal children of the root
    b.parents[1, 3] = 4
    b.parents[4, 0] = -1
    ref = run_tree_accept(b, 300, 304, dv.F32, x, drafts, [1] * 6)
    assert ref["path_rows"][0, 1] == 1 and ref["meta"][1] == oracle.DATA_BAD_TREE
    b.cu[3] = b.cu[2]  # an empty request
    run_tree_accept(b, 300, 304, dv.F32, x, drafts, [1] * 6, max_rows=int(b.cu[5]))


# ------------------------------------------------------------------ commit

@pytest.mark.parametrize("kind,layers,hkv,D,page,gamma,joint", [
    ("bf16", 0, 1, 64, 16, 1, False), ("f16", 3, 2, 128, 16, 8, True),
    ("e4m3", 2, 8, 128, 32, 16, False), ("e4m3", 4, 3, 64, 16, 64, True),
    ("bf16", 2, 5, 256, 256, 64, False)])
def test_commit(kind, layers, hkv, D, page, gamma, joint):
    say(f"commit {kind} layers={layers} D={D} gamma={gamma}")
    rng = np.random.default_rng(gamma + D)
    B = 9
    b = Batch(2, [gamma + 1] * B, rng.integers(0, 60, B).tolist(), gamma, page, False)
    cache = make_cache(kind, b.nb, hkv, page, D, layers=layers, joint=joint)
    for t in (cache.k, cache.v):
        raw = torch.randint(0, 100, t.shape, device=DEV, dtype=torch.uint8)
        bits_t = t.view(torch.uint8) if kind == "e4m3" else t
        bits_t.copy_(raw if kind == "e4m3" else raw.to(t.dtype))
    if kind == "e4m3":
        for t in (cache.k_scale, cache.v_scale):
            t.copy_(torch.randint(90, 140, t.shape, device=DEV, dtype=torch.uint8))
    num = rng.integers(0, gamma + 1, B)
    num[0], num[1] = gamma, 0
    path = np.full((B, gamma + 1), -1, np.int32)
    for r in range(B):
        path[r, :num[r] + 1] = [0] + sorted(rng.choice(np.arange(1, gamma + 1), num[r], replace=False))
    ctx, table = np.array(b.ctx), b.table.copy()
    status = 0
    if gamma >= 8:
        path[2, 0] = 1
        num[3] = gamma + 1
        num[4], path[4, :4] = 3, [0, 5, 5, 6]
        num[5], path[5, :3] = 2, [0, 4, gamma]
        table[5, (ctx[5] + gamma) // page] = b.nb + 3
        ctx[6] = -4
        status = oracle.DATA_BAD_LENS | oracle.DATA_BAD_TREE | oracle.DATA_BAD_PAGE
    pools = [cache.k, cache.v] + ([cache.k_scale, cache.v_scale] if kind == "e4m3" else [])
    want = [bits(t).clone() for t in pools]
    moved = 0
    for r in range(B):
        mv = oracle.commit_moves(path[r], num[r], int(ctx[r]), gamma)
        if not mv or any(not 0 <= table[r, i // page] < b.nb for m in mv for i in m):
            continue
        moved += len(mv)
        for w in want:
            for s, d in mv:
                src = (Ellipsis,) if not layers else (slice(None),)
                a = src[:0] + ((slice(None),) if layers else ()) + (int(table[r, s // page]), slice(None), s % page)
                z = ((slice(None),) if layers else ()) + (int(table[r, d // page]), slice(None), d % page)
                w[z] = w[a]
    cm = torch.empty(2, dtype=torch.int32, device=DEV)
    dv.dspark_kv_commit(B, gamma, i32(path), i32(num), i32(ctx), i32(table), cache, cm)
    torch.cuda.synchronize()
    assert cm.tolist() == [moved, status]
    for t, w in zip(pools, want):
        assert torch.equal(bits(t), w)


# ------------------------------------------------------------------ graphs and streams

def test_graph_replays_and_a_side_stream():
    """Append, attention, accept and commit captured together, replayed with
    eager work between: every replay gives the eager result."""
    say("graph replays")
    D, hq, hkv, page, gamma, V = 128, 8, 2, 16, 8, 512
    b = Batch(11, [9, 4, 6], [100, 33, 700], gamma, page, True)
    rng = np.random.default_rng(3)
    cache = make_cache("e4m3", b.nb, hkv, page, D, layers=2)
    lay = cache.layer(1)
    for L in range(2):
        for r in range(b.B):
            put(cache, b.slots(r, 0, b.ctx[r] + b.lens[r]),
                *rng.normal(0, 1, (2, b.ctx[r] + b.lens[r], hkv, D)).astype(np.float32), layer=L)
    keep = [t.clone() for t in (cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale,
                                cache.v_scale)]
    x = torch.from_numpy(rng.normal(0, 1, (b.rows, hq + 2 * hkv, D)).astype(np.float32)).bfloat16().to(DEV)
    b.parents[0, :3] = [0, 0, 2]  # row 1 is wrong, rows 2 and 3 are right: they move
    logits, drafts = tree_logits(rng, b, V, V, dv.F32, hit=1.0)
    drafts[0, 0] = (drafts[0, 0] + 1) % V
    logits, drafts = up(logits), i32(drafts)
    ap = dv.alloc_append_outputs(b.rows, hq, lay)
    o = dv.alloc_attention_outputs(b.B, gamma, b.rows, hq, lay, lse=True)
    ta = dv.alloc_tree_accept_outputs(b.B, gamma, b.rows, V, dv.F32, DEV)
    cm = torch.empty(2, dtype=torch.int32, device=DEV)
    cu, pre, table = b.args()
    par = b.par()
    outs = [ap.q_out, o.out, o.lse, ta.path_rows, ta.num_correct, cm, o.attention_meta, ap.append_meta]

    def step():
        dv.dspark_kv_append(b.B, gamma, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], b.rows, cu, pre,
                            table, lay, ap, tree_parents=par)
        dv.dspark_tree_attention(b.B, gamma, ap.q_out, b.rows, cu, pre, table, lay, 0.09, o,
                                 tree_parents=par)
        dv.dspark_tree_accept(b.B, gamma, V, dv.F32, logits, V, b.rows, cu, drafts, par, pre, ta)
        dv.dspark_kv_commit(b.B, gamma, ta.path_rows, ta.num_correct, pre, table, cache, cm)

    def reset():
        for t, k in zip((cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale,
                         cache.v_scale), keep):
            t.copy_(k)
        for t in outs:
            t.fill_(-7)

    def result():
        torch.cuda.synchronize()
        return [t.clone() for t in outs] + [cache.k.view(torch.uint8).clone(),
                                            cache.v.view(torch.uint8).clone(), cache.k_scale.clone()]

    reset()
    step()
    eager = result()
    assert int(eager[5][0]) > 0  # something moves
    side = torch.cuda.Stream()
    reset()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
    for a, e in zip(result(), eager):
        assert torch.equal(a, e)
    g = torch.cuda.CUDAGraph()
    reset()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step()
    for i in range(4):
        reset()
        torch.cuda.synchronize()
        g.replay()
        for n, (a, e) in enumerate(zip(result(), eager)):
            assert torch.equal(a, e), (i, n)
        step()  # eager work between the replays
        torch.cuda.synchronize()
