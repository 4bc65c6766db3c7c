"""Timed cases of the target-pass operators of a verify step.

The operators sit between the packing of a verify step's rows and its accept,
and after it: the norms, rotation and (quantising) write of the step's keys and
values into a paged cache, the read of cache rows, the attention of a tree or
chain of drafted rows over that cache, the greedy accept along a draft tree,
and the move of the accepted path's cache rows to consecutive slots.

With ``own`` false ``run`` computes a case in elementary torch operations in
float32, rounded once at the end; with ``own`` true it makes the calls that a
serving program makes of the framework. ``exact`` is the definition in float64.

Common layout: request r owns packed rows cu[r] .. cu[r+1]-1 (row 0 its root),
its context of prefix[r] tokens is in the cache, and its row j lives at cache
index prefix[r] + j. ``parents[r, j-1]`` is the parent row of row j.
"""

from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6
ROPE_BASE = 10000.0
_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one request decoding a single token over a short context: latency
        dict(name="attn_decode_b1", op="attn", B=1, gamma=1, rows_hi=1, ctx_lo=700, ctx_hi=700, hq=32, hkv=8,
             D=128, page=16, cache="bf16", tree=False),
        # a serving batch verifying chains of up to 8 drafts over mixed contexts
        dict(name="attn_chain_b32_bf16", op="attn", B=32, gamma=8, rows_hi=9, ctx_lo=1024, ctx_hi=8192, hq=32,
             hkv=8, D=128, page=64, cache="bf16", tree=False),
        # a larger batch verifying trees of 16 drafts over an 8-bit cache
        dict(name="attn_tree_b64_e4m3", op="attn", B=64, gamma=16, rows_hi=17, ctx_lo=500, ctx_hi=8000, hq=64,
             hkv=8, D=128, page=32, cache="e4m3", tree=True),
        # two long documents, trees of the largest size, narrow heads
        dict(name="attn_tree_b2_long_f16", op="attn", B=2, gamma=64, rows_hi=65, ctx_lo=70001, ctx_hi=131001,
             hq=16, hkv=2, D=64, page=256, cache="f16", tree=True),
        # a few requests, narrow heads, no norm: what a small draft model appends
        dict(name="append_b4_f16", op="append", B=4, gamma=4, rows_hi=5, ctx_lo=33, ctx_hi=900, hq=16, hkv=4, D=64,
             page=16, cache="f16", tree=False, norm=False, rot=64, interleaved=True),
        # the step's rows of a full batch into an 8-bit cache, norms and rotation
        dict(name="append_b256_e4m3", op="append", B=256, gamma=8, rows_hi=9, ctx_lo=100, ctx_hi=4000, hq=32, hkv=8,
             D=128, page=32, cache="e4m3", tree=True, norm=True, rot=128, interleaved=False),
        # a few short spans of a cache, as they come back after a rejected step
        dict(name="read_b8_bf16", op="read", B=8, n_lo=1, n_hi=64, hkv=8, D=128, page=16, cache="bf16"),
        # whole contexts read back from an 8-bit cache, to be moved to another worker
        dict(name="read_b16_e4m3", op="read", B=16, n_lo=700, n_hi=8192, hkv=8, D=128, page=64, cache="e4m3"),
        # a small batch of small trees over a 32000-word vocabulary
        dict(name="accept_b8_f32", op="accept", B=8, gamma=8, rows_hi=9, V=32000, dtype="f32"),
        # a full batch of trees over the largest vocabulary of the verify step
        dict(name="accept_b256_bf16", op="accept", B=256, gamma=8, rows_hi=9, V=129280, dtype="bf16"),
        # a few requests, few layers: latency
        dict(name="commit_b4_bf16", op="commit", B=4, gamma=8, layers=2, ctx_lo=20, ctx_hi=500, hkv=8, D=128, page=16,
             cache="bf16"),
        # a full batch over all layers of a model in one call
        dict(name="commit_b256_e4m3", op="commit", B=256, gamma=16, layers=32, ctx_lo=100, ctx_hi=4000, hkv=8, D=128,
             page=16, cache="e4m3"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "read", "accept", "commit"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "attn":
        cache = rng.choice(["bf16", "f16", "e4m3"])
        D = rng.choice([64, 128, 128, 256])
        hkv = rng.choice([1, 2, 3, 4, 8])
        group = rng.choice([1, 2, 4, 5, 7, 8])
        gamma = _log(rng, 1, 64)
        B = _log(rng, 1, 64)
        # keys in all, so that no case exceeds the largest listed one
        heads = B * hkv
        most = int(min(130000, 140e6 / (heads * D), 300e6 / (heads * group * (gamma + 1)),
                       30e9 / (heads * group * (gamma + 1) * D)))
        hi = _log(rng, 1, max(1, most))
        return dict(op=op, B=B, gamma=gamma, rows_hi=rng.randint(1, gamma + 1), ctx_lo=rng.randint(0, hi), ctx_hi=hi,
                    hq=hkv * group, hkv=hkv, D=D, page=page, cache=cache, tree=rng.random() < 0.6)
    if op == "append":
        D = rng.choice([64, 128, 128, 256])
        hkv = rng.choice([1, 2, 4, 5, 8])
        group = rng.choice([1, 3, 4])
        gamma = _log(rng, 1, 32)
        B = _log(rng, 1, max(1, min(256, 14_000_000 // (D * hkv * (group + 2) * (gamma + 1)))))
        hi = _log(rng, 1, 30000)
        return dict(op=op, B=B, gamma=gamma, rows_hi=rng.randint(1, gamma + 1), ctx_lo=rng.randint(0, hi), ctx_hi=hi,
                    hq=hkv * group, hkv=hkv, D=D, page=page, cache=rng.choice(["bf16", "f16", "e4m3"]),
                    tree=rng.random() < 0.5, norm=rng.random() < 0.7, rot=rng.choice([0, 32, 64, D]),
                    interleaved=rng.random() < 0.5)
    if op == "read":
        hkv = rng.choice([1, 2, 4, 5, 8])
        D = rng.choice([64, 128, 256])
        B = _log(rng, 1, 128)
        hi = _log(rng, 1, max(1, int(50_000_000 / (B * hkv * D))))
        return dict(op=op, B=B, n_lo=rng.randint(0, hi), n_hi=hi, hkv=hkv, D=D, page=page,
                    cache=rng.choice(["bf16", "f16", "e4m3"]))
    if op == "accept":
        gamma = _log(rng, 1, 64)
        B = _log(rng, 1, max(1, min(256, 1300 // (gamma + 1))))
        dtype = rng.choice(["bf16", "f32"])
        V = _log(rng, 1000, 129280 if dtype == "bf16" else 64640)
        return dict(op=op, B=B, gamma=gamma, rows_hi=rng.randint(1, gamma + 1), V=V, dtype=dtype)
    gamma = _log(rng, 1, 32)
    B = _log(rng, 1, 128)
    hi = _log(rng, 1, 4000)
    return dict(op=op, B=B, gamma=gamma, layers=_log(rng, 1, 24), ctx_lo=rng.randint(0, hi), ctx_hi=hi,
                hkv=rng.choice([1, 2, 4, 5, 8]), D=rng.choice([64, 128, 256]), page=rng.choice([16, 32, 64]),
                cache=rng.choice(["bf16", "f16", "e4m3"]))


def _spread(n, lo, hi):
    """n whole numbers from lo to hi, evenly spread: the case alone fixes them."""
    if n == 1:
        return [hi]
    return [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _accepted(n, gamma):
    """Accepted drafts of n requests: short paths are the common ones."""
    return [min(gamma, int(gamma * ((i + 0.5) / n) ** 2 + 0.5)) for i in range(n)]


def work(case):
    c = case
    op = c["op"]
    cb = 1 if c.get("cache") == "e4m3" else 2
    if op in ("attn", "append"):
        lens = _spread(c["B"], 1, c["rows_hi"])
        ctx = _spread(c["B"], c["ctx_lo"], c["ctx_hi"])
    if op == "attn":
        # pairs of lengths are shuffled by the seed: the mean stands for all
        keys = sum(ctx) + sum(lens)
        pairs = sum(lens) * keys / c["B"]
        sc = 2 if cb == 1 else 0
        return dict(bytes=keys * c["hkv"] * (2 * c["D"] * cb + sc) + 2 * 2 * sum(lens) * c["hq"] * c["D"],
                    flops=4 * pairs * c["hq"] * c["D"])
    if op == "append":
        rows = sum(lens)
        heads = c["hq"] + 2 * c["hkv"]
        return dict(bytes=rows * c["D"] * (2 * heads + 2 * c["hq"] + 2 * c["hkv"] * (2 * cb + 2)) + rows * c["rot"] * 4,
                    flops=10 * rows * heads * c["D"])
    if op == "read":
        rows = sum(_spread(c["B"], c["n_lo"], c["n_hi"]))
        return dict(bytes=max(1, rows) * 2 * c["hkv"] * c["D"] * (cb + 2), flops=0)
    if op == "accept":
        rows = sum(_spread(c["B"], 1, c["rows_hi"]))
        return dict(bytes=rows * c["V"] * (2 if c["dtype"] == "bf16" else 4), flops=rows * c["V"])
    moved = sum(_accepted(c["B"], c["gamma"]))
    return dict(bytes=max(1, moved) * c["layers"] * 2 * 2 * c["hkv"] * c["D"] * cb, flops=0)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _i32(a):
    return torch.tensor(a, dtype=torch.int32, device=DEV)


def _make_parents(rng, B, gamma, tree):
    """Drafts in topological order: mostly a spine, with branches off it."""
    rows = []
    for _ in range(B):
        row = []
        for j in range(1, gamma + 1):
            row.append(j - 1 if not tree or rng.random() < 0.5 else rng.randint(max(0, j - 9), j - 1))
        rows.append(row)
    return rows


def _power(e):
    """2^e in float32, for whole e in [-126, 127]."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _e4m3(x):
    """[..., D] float32 -> codes and exponent bytes, one exponent for each row."""
    amax = x.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(amax / 448.0)  # amax / 448 = m 2^e, m in [0.5, 1)
    e = torch.where(m == 0.5, e - 1, e)
    e = torch.where(amax == 0, torch.zeros_like(e), e).clamp(-100, 119)
    codes = (x * _power(-e)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8).squeeze(-1)


def _pool(g, shape, cache):
    """A pool of cache rows with the spread that keys and values have."""
    if cache == "e4m3":
        out = torch.empty(shape, dtype=torch.float8_e4m3fn, device=DEV)
        scale = torch.empty(shape[:-1], dtype=torch.uint8, device=DEV)
        flat, fs = out.view(-1, shape[-1]), scale.view(-1)
        for i in range(0, flat.shape[0], 1 << 20):
            x = torch.randn(min(1 << 20, flat.shape[0] - i), shape[-1], generator=g, device=DEV)
            c, s = _e4m3(x)
            flat[i:i + x.shape[0]] = c
            fs[i:i + x.shape[0]] = s
        return out, scale
    return torch.randn(shape, generator=g, device=DEV, dtype=_DT[cache]), None


def _blocks(rng, needs, page):
    """A table of scattered pages for the given token counts, and the pool's size
    (its last page belongs to nobody)."""
    counts = [max(1, -(-n // page)) for n in needs]
    ids = list(range(sum(counts)))
    rng.shuffle(ids)
    table, at = [], 0
    width = max(counts)
    for n in counts:
        table.append(ids[at:at + n] + [0] * (width - n))
        at += n
    return table, sum(counts) + 1


def _cum(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def prepare(case, seed):
    c = case
    rng = random.Random(seed * 7919 + 13)
    g = _gen(seed)
    s = dict(c=dict(c))
    op, B = c["op"], c["B"]
    if op in ("attn", "append", "accept"):
        lens = _spread(B, 1, c["rows_hi"])
        rng.shuffle(lens)
        cu = _cum(lens)
        rows = -(-cu[-1] // 16) * 16  # the captured tier: rows past the total are padding
        parents = _make_parents(rng, B, c["gamma"], c.get("tree", True))
        s.update(cu=_i32(cu), rows=rows, parents=_i32(parents) if c.get("tree", True) else None)
    if op in ("attn", "append"):
        ctx = _spread(B, c["ctx_lo"], c["ctx_hi"])
        rng.shuffle(ctx)
        dt = torch.float16 if c["cache"] == "f16" else torch.bfloat16
        D, hq, hkv = c["D"], c["hq"], c["hkv"]
        s.update(prefix=_i32(ctx), dt=dt)
    if op == "attn":
        table, nb = _blocks(rng, [a + b for a, b in zip(ctx, lens)], c["page"])
        s["k"], s["ks"] = _pool(g, (nb, hkv, c["page"], D), c["cache"])
        s["v"], s["vs"] = _pool(g, (nb, hkv, c["page"], D), c["cache"])
        s["q"] = (1.5 * torch.randn(rows, hq, D, generator=g, device=DEV)).to(dt)
        s["table"] = _i32(table)
        s["scale"] = D ** -0.5
    elif op == "append":
        table, nb = _blocks(rng, [a + b for a, b in zip(ctx, lens)], c["page"])
        # one buffer of a fused projection: the three are views of its rows
        qkv = torch.randn(rows, (hq + 2 * hkv) * D, generator=g, device=DEV).to(dt)
        s["q"] = qkv[:, :hq * D].unflatten(1, (hq, D))
        s["kn"] = qkv[:, hq * D:(hq + hkv) * D].unflatten(1, (hkv, D))
        s["vn"] = qkv[:, (hq + hkv) * D:].unflatten(1, (hkv, D))
        kind = torch.float8_e4m3fn if c["cache"] == "e4m3" else dt
        s["k"] = torch.zeros(nb, hkv, c["page"], D, device=DEV).to(kind)
        s["v"] = torch.zeros(nb, hkv, c["page"], D, device=DEV).to(kind)
        sc = c["cache"] == "e4m3"
        s["ks"] = torch.full((nb, hkv, c["page"]), 127, dtype=torch.uint8, device=DEV) if sc else None
        s["vs"] = torch.full((nb, hkv, c["page"]), 127, dtype=torch.uint8, device=DEV) if sc else None
        s["table"] = _i32(table)
        s["qw"] = s["kw"] = s["rope"] = None
        if c["norm"]:
            s["qw"] = (1 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(dt)
            s["kw"] = (1 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(dt)
        if c["rot"]:
            at = torch.arange(c["ctx_hi"] + c["gamma"] + 1, device=DEV, dtype=torch.float64)
            f = ROPE_BASE ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"])
            a = at[:, None] * f
            s["rope"] = torch.cat([a.cos(), a.sin()], 1).float()
    elif op == "read":
        n = _spread(B, c["n_lo"], c["n_hi"])
        rng.shuffle(n)
        starts = [rng.randint(0, 3 * c["page"]) for _ in range(B)]
        table, nb = _blocks(rng, [a + b for a, b in zip(n, starts)], c["page"])
        s["k"], s["ks"] = _pool(g, (nb, c["hkv"], c["page"], c["D"]), c["cache"])
        s["v"], s["vs"] = _pool(g, (nb, c["hkv"], c["page"], c["D"]), c["cache"])
        cu = _cum(n)
        s.update(cu=_i32(cu), rows=max(1, cu[-1]), prefix=_i32(starts), table=_i32(table),
                 dt=torch.float16 if c["cache"] == "f16" else torch.bfloat16)
    elif op == "accept":
        V, gamma = c["V"], c["gamma"]
        ld = -(-V // 8) * 8
        dt = _DT[c["dtype"]]
        x = torch.empty(rows, ld, dtype=dt, device=DEV)
        for i in range(0, rows, 256):
            x[i:i + 256] = (3 * torch.randn(min(256, rows - i), ld, generator=g, device=DEV)).to(dt)
        # what the target predicts: a planted maximum, sometimes twice in a row
        top = torch.randint(0, V, (rows,), generator=g, device=DEV)
        twin = torch.randint(0, V, (rows,), generator=g, device=DEV)
        at = torch.arange(rows, device=DEV)
        x[at, top] = 24.0
        x[at[::10], twin[::10]] = 24.0
        first = top.clone()
        first[::10] = torch.minimum(top[::10], twin[::10])
        # drafts: what their parent's row predicts, three times in four
        par = _i32(parents).long()
        src = (s["cu"][:-1, None].long() + par).clamp(max=rows - 1)
        other = torch.randint(0, V, (B, gamma), generator=g, device=DEV)
        hit = torch.rand(B, gamma, generator=g, device=DEV) < 0.75
        s["drafts"] = torch.where(hit, first[src], other).int()
        s["x"], s["ld"] = x, ld
        s["prefix"] = _i32([rng.randint(1, 4000) for _ in range(B)])
    else:
        gamma, D, hkv, page = c["gamma"], c["D"], c["hkv"], c["page"]
        ctx = _spread(B, c["ctx_lo"], c["ctx_hi"])
        rng.shuffle(ctx)
        acc = _accepted(B, gamma)
        rng.shuffle(acc)
        paths = [[0] + sorted(rng.sample(range(1, gamma + 1), n)) + [-1] * (gamma - n) for n in acc]
        # a request's own pages hold its window; its context before it is a
        # common prompt, whose page 0 is shared and never moved
        need = [-(-(n + gamma + 1) // page) for n in ctx]
        own_pages = [b - n // page for n, b in zip(ctx, need)]
        ids = list(range(1, 1 + sum(own_pages)))
        rng.shuffle(ids)
        table, at, width = [], 0, max(need)
        for n, b, o in zip(ctx, need, own_pages):
            table.append([0] * (b - o) + ids[at:at + o] + [0] * (width - b))
            at += o
        nb = 2 + sum(own_pages)
        s["k"], s["ks"] = _pool(g, (c["layers"], nb, hkv, page, D), c["cache"])
        s["v"], s["vs"] = _pool(g, (c["layers"], nb, hkv, page, D), c["cache"])
        s.update(prefix=_i32(ctx), paths=_i32(paths), acc=_i32(acc), table=_i32(table))
    return s


# ------------------------------------------------------------------ plain form

def _row_of(s, rows):
    """For each packed row: its request, its index there, whether it is a real row."""
    cu = s["cu"].long()
    at = torch.arange(rows, device=DEV)
    r = torch.searchsorted(cu[1:], at, right=True)
    ok = at < cu[-1]
    r = torch.where(ok, r, torch.zeros_like(r))
    j = torch.where(ok, at - cu[r], torch.zeros_like(r))
    return r, j, ok


def _ancestors(s, c):
    """[B, gamma + 1, gamma + 1]: row j's own and its ancestors' columns."""
    n = c["gamma"] + 1
    if s["parents"] is None:
        return torch.ones(n, n, device=DEV).tril().bool().expand(c["B"], n, n)
    step = torch.eye(n, device=DEV).repeat(c["B"], 1, 1)
    step[:, 1:].scatter_(2, s["parents"].long()[..., None], 1.0, reduce="add")
    return torch.linalg.matrix_power(step, 64) > 0


def _values(pool, scale):
    x = pool.float()
    return x if scale is None else x * _power(scale.int()[..., None] - 127)


def _plain_attn(s):
    c = s["c"]
    B, hkv, D, rows = c["B"], c["hkv"], c["D"], s["rows"]
    G, L = c["hq"] // hkv, c["gamma"] + 1
    r, j, ok = _row_of(s, rows)
    table = s["table"].long()
    T = table.shape[1] * c["page"]

    def dense(pool, scale):
        x = _values(pool[table], None if scale is None else scale[table])
        return x.permute(0, 2, 1, 3, 4).reshape(B, hkv, T, D)

    q = torch.zeros(B, L + 1, c["hq"], D, device=DEV)
    q[r, torch.where(ok, j, L)] = s["q"].float()
    q = q[:, :L].view(B, L, hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, hkv, L * G, D)
    k = dense(s["k"], s["ks"])
    sc = torch.matmul(q, k.transpose(2, 3).contiguous()) * s["scale"]
    del k
    cu = s["cu"].long()
    lens, pre = cu[1:] - cu[:-1], s["prefix"].long()
    key = torch.arange(T, device=DEV)
    live = key < (pre + lens)[:, None]
    i = (key - pre[:, None]).clamp(0, L - 1)
    seen = torch.gather(_ancestors(s, c), 2, i[:, None, :].expand(B, L, T))
    seen = (seen | (key < pre[:, None])[:, None]) & live[:, None]
    sc = sc.view(B, hkv, L, G, T).masked_fill(~seen[:, None, :, None], -math.inf).view(B, hkv, L * G, T)
    sc = torch.exp(sc - sc.amax(-1, keepdim=True))
    total = sc.sum(-1, keepdim=True)
    v = dense(s["v"], s["vs"]).masked_fill(~live[:, None, :, None], 0.0)
    o = torch.matmul(sc, v) / total
    o = o.view(B, hkv, L, G, D).permute(0, 2, 1, 3, 4).reshape(B, L, c["hq"], D)
    return [torch.where(ok[:, None, None], o[r, j], 0.0).to(s["dt"])]


def _rotate(x, cs, c):
    """x [rows, heads, D] float32, cs [rows, rot]: cosines, then sines."""
    h = c["rot"] // 2
    co, si = cs[:, None, :h], cs[:, None, h:]
    if c["interleaved"]:
        a, b = x[..., 0:2 * h:2], x[..., 1:2 * h:2]
        turned = torch.stack([a * co - b * si, b * co + a * si], -1).flatten(-2)
    else:
        a, b = x[..., :h], x[..., h:2 * h]
        turned = torch.cat([a * co - b * si, b * co + a * si], -1)
    return torch.cat([turned, x[..., 2 * h:]], -1)


def _plain_append(s):
    c = s["c"]
    r, j, ok = _row_of(s, s["rows"])
    q, k, v = s["q"].float(), s["kn"].float(), s["vn"].float()
    if c["norm"]:
        q = q * torch.rsqrt((q * q).mean(-1, keepdim=True) + EPS) * s["qw"].float()
        k = k * torch.rsqrt((k * k).mean(-1, keepdim=True) + EPS) * s["kw"].float()
    if c["rot"]:
        depth = _ancestors(s, c).sum(-1) - 1
        cs = s["rope"][s["prefix"].long()[r] + depth[r, j]]
        q, k = _rotate(q, cs, c), _rotate(k, cs, c)
    slot = s["prefix"].long()[r] + j
    block = s["table"].long()[r, slot // c["page"]]
    block = torch.where(ok, block, s["k"].shape[0] - 1)  # the page of nobody
    off = slot % c["page"]
    back = []
    for name, x in (("k", k), ("v", v)):
        if c["cache"] == "e4m3":
            codes, e = _e4m3(x)
            s[name].view(torch.uint8)[block, :, off] = codes.view(torch.uint8)
            s[name + "s"][block, :, off] = e
            x = _values(s[name].view(torch.uint8)[block, :, off].view(torch.float8_e4m3fn),
                        s[name + "s"][block, :, off])
        else:
            s[name][block, :, off] = x.to(s["dt"])
            x = s[name][block, :, off]
        back.append(torch.where(ok[:, None, None], x, 0.0).to(s["dt"]))
    return [torch.where(ok[:, None, None], q, 0.0).to(s["dt"])] + back


def _plain_read(s):
    c = s["c"]
    r, j, ok = _row_of(s, s["rows"])
    slot = s["prefix"].long()[r] + j
    block, off = s["table"].long()[r, slot // c["page"]], slot % c["page"]
    outs = []
    for name in ("k", "v"):
        if c["cache"] == "e4m3":
            x = _values(s[name].view(torch.uint8)[block, :, off].view(torch.float8_e4m3fn),
                        s[name + "s"][block, :, off])
        else:
            x = s[name][block, :, off]
        outs.append(torch.where(ok[:, None, None], x, 0.0).to(s["dt"]))
    return outs


def _plain_accept(s):
    c = s["c"]
    B, gamma, V, rows = c["B"], c["gamma"], c["V"], s["rows"]
    x = s["x"][:, :V].float()
    word = torch.arange(V, device=DEV)
    am = torch.where(x == x.amax(-1, keepdim=True), word, V).amin(-1)
    _, _, ok = _row_of(s, rows)
    cu = s["cu"].long()
    lens = cu[1:] - cu[:-1]
    par, dr = s["parents"].long(), s["drafts"].long()
    k = torch.arange(1, gamma + 1, device=DEV)
    real = k < lens[:, None]
    hit = real & (am[(cu[:-1, None] + par).clamp(max=rows - 1)] == dr)
    # of equal siblings the first counts
    same = (par[:, :, None] == par[:, None, :]) & (dr[:, :, None] == dr[:, None, :])
    hit &= ~(same.tril(-1)).any(-1)
    missed = torch.cat([torch.zeros(B, 1, device=DEV), (~hit).float()], 1)
    path = torch.matmul(_ancestors(s, c).float(), missed[..., None])[..., 0] == 0  # [B, gamma + 1]
    n = path.sum(-1) - 1
    row = torch.where(path, torch.arange(gamma + 1, device=DEV), gamma + 1).sort(-1).values
    on = torch.arange(gamma + 1, device=DEV) <= n[:, None]
    last = torch.gather(row, 1, n[:, None])[:, 0]
    bonus = am[cu[:-1] + last]
    # column t holds the draft of the path's row t + 1, then the bonus
    nxt = torch.cat([row[:, 1:], torch.full((B, 1), gamma + 1, device=DEV)], 1)
    tok = torch.gather(dr, 1, (nxt - 1).clamp(0, gamma - 1))
    col = torch.arange(gamma + 1, device=DEV)
    out = torch.where(col < n[:, None], tok, torch.where(col == n[:, None], bonus[:, None], -1))
    return [torch.where(ok, am, -1).int(), n.int(), bonus.int(), (n + 1).int(), out.int(),
            torch.where(on, row, -1).int(), (s["prefix"].long() + n + 1).int()]


def _plain_commit(s):
    c = s["c"]
    gamma, page = c["gamma"], c["page"]
    k = torch.arange(1, gamma + 1, device=DEV)
    on = k <= s["acc"].long()[:, None]
    pre = s["prefix"].long()[:, None]
    src = torch.where(on, pre + s["paths"].long()[:, 1:], pre)
    dst = torch.where(on, pre + k, pre)
    table = s["table"].long()
    bs, bd = torch.gather(table, 1, src // page), torch.gather(table, 1, dst // page)
    spare = s["k"].shape[1] - 1
    bd = torch.where(on, bd, spare)
    outs = []
    for name in ("k", "v", "ks", "vs"):
        pool = s[name]
        if pool is not None:
            p = pool.view(torch.uint8) if pool.dtype == torch.float8_e4m3fn else pool
            p[:, bd, :, dst % page] = p[:, bs, :, src % page]
            outs.append(pool[:, :spare])
    return outs


# ------------------------------------------------------------------ the framework's calls

def _own(s):
    import dspark_verify_scheduling_amd as dv

    c = s["c"]
    op, B = c["op"], c["B"]
    new = "out" not in s
    if new and op != "accept":
        s["cache"] = dv.KvCache(s["k"], s["v"], s["ks"], s["vs"])
    if op == "attn":
        if new:
            s["out"] = dv.alloc_attention_outputs(B, c["gamma"], s["rows"], c["hq"], s["cache"])
            s["out"].out.zero_()
        dv.dspark_tree_attention(B, c["gamma"], s["q"], s["rows"], s["cu"], s["prefix"], s["table"], s["cache"],
                                 s["scale"], s["out"], tree_parents=s["parents"])
        return [s["out"].out]
    if op in ("append", "read"):
        if new:
            s["back"] = dv.alloc_kv_read_outputs(s["rows"], s["cache"])
            s["back"].k_out.zero_()
            s["back"].v_out.zero_()
            s["out"] = s["back"]
            if op == "append":
                s["out"] = dv.alloc_append_outputs(s["rows"], c["hq"], s["cache"])
                s["out"].q_out.zero_()
        if op == "append":
            dv.dspark_kv_append(B, c["gamma"], s["q"], s["kn"], s["vn"], s["rows"], s["cu"], s["prefix"], s["table"],
                                s["cache"], s["out"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS, rope=s["rope"],
                                rope_interleaved=c["interleaved"], tree_parents=s["parents"])
        dv.dspark_kv_read(B, s["rows"], s["cu"], s["prefix"], s["table"], s["cache"], s["back"])
        back = [s["back"].k_out, s["back"].v_out]
        return [s["out"].q_out] + back if op == "append" else back
    if op == "accept":
        dt = dv.BF16 if c["dtype"] == "bf16" else dv.F32
        if new:
            s["out"] = dv.alloc_tree_accept_outputs(B, c["gamma"], s["rows"], c["V"], dt, DEV)
            s["out"].row_argmax.fill_(-1)
        o = s["out"]
        dv.dspark_tree_accept(B, c["gamma"], c["V"], dt, s["x"], s["ld"], s["rows"], s["cu"], s["drafts"],
                              s["parents"], s["prefix"], o)
        return [o.row_argmax, o.num_correct, o.bonus, o.commit_lens, o.out_tokens, o.path_rows, o.new_seq_lens]
    if new:
        s["out"] = torch.empty(2, dtype=torch.int32, device=DEV)
    dv.dspark_kv_commit(B, c["gamma"], s["paths"], s["acc"], s["prefix"], s["table"], s["cache"], s["out"])
    spare = s["k"].shape[1] - 1
    return [s[n][:, :spare] for n in ("k", "v", "ks", "vs") if s[n] is not None]


def run(state):
    if own:
        return _own(state)
    return {"attn": _plain_attn, "append": _plain_append, "read": _plain_read, "accept": _plain_accept,
            "commit": _plain_commit}[state["c"]["op"]](state)


# ------------------------------------------------------------------ the definition in 64 bits

def _tree_of(parents, r, n):
    """Row j's path from the root, for the n rows of request r."""
    paths = [[0]]
    for j in range(1, n):
        paths.append(paths[j - 1 if parents is None else parents[r][j - 1]] + [j])
    return paths


def _span(s, name, r, lo, n, page):
    """n cache rows from index lo of request r, [hkv, n, D] float64."""
    at = torch.arange(lo, lo + n, device=DEV)
    b, o = s["table"][r].long()[at // page], at % page
    raw = s[name]
    raw = raw.view(torch.uint8) if raw.dtype == torch.float8_e4m3fn else raw
    x = raw[b, :, o]
    if s[name + "s"] is not None:
        e = s[name + "s"][b, :, o].double() - 127
        x = x.view(torch.float8_e4m3fn).double() * torch.exp2(e)[..., None]
    return x.double().transpose(0, 1)


def _to_e4m3(x):
    """The value that 8 bits keep of each row's elements: steps of 2^-3 of the leading power of two."""
    top = x.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.ceil(torch.log2(top / 448)), torch.zeros_like(top)).clamp(-100, 119)
    e = torch.where(top > 448 * torch.exp2(e), e + 1, e)
    y = x * torch.exp2(-e)
    lead = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(lead - 3)
    return torch.round(y / step) * step * torch.exp2(e)


def exact(case, seed):
    c = case
    op = c["op"]
    s = prepare(c, seed)
    if op == "accept":
        return _exact_accept(s, c)
    if op == "commit":
        return None  # bytes are moved: nothing is computed
    cu, pre = s["cu"].tolist(), s["prefix"].tolist()
    hkv, D, page = c["hkv"], c["D"], c["page"]
    if op == "read":
        out = [torch.zeros(s["rows"], hkv, D, dtype=torch.float64, device=DEV) for _ in range(2)]
        for r in range(c["B"]):
            n = cu[r + 1] - cu[r]
            if n:
                for o, name in zip(out, "kv"):
                    o[cu[r]:cu[r + 1]] = _span(s, name, r, pre[r], n, page).transpose(0, 1)
        return out
    parents = None if s["parents"] is None else s["parents"].tolist()
    G = c["hq"] // hkv
    if op == "attn":
        out = torch.zeros(s["rows"], c["hq"], D, dtype=torch.float64, device=DEV)
        for r in range(c["B"]):
            n = cu[r + 1] - cu[r]
            T = pre[r] + n
            k, v = (_span(s, name, r, 0, T, page) for name in "kv")
            see = torch.zeros(n, T, dtype=torch.bool, device=DEV)
            see[:, :pre[r]] = True
            pairs = [(j, pre[r] + i) for j, p in enumerate(_tree_of(parents, r, n)) for i in p]
            see[tuple(torch.tensor(pairs, device=DEV).T)] = True
            q = s["q"][cu[r]:cu[r + 1]].double().view(n, hkv, G, D)
            for h in range(hkv):
                a = (q[:, h].reshape(n * G, D) @ k[h].T).view(n, G, T) * s["scale"]
                a.masked_fill_(~see[:, None], -math.inf)
                a = torch.softmax(a, -1).view(n * G, T)
                out[cu[r]:cu[r + 1], h * G:(h + 1) * G] = (a @ v[h]).view(n, G, D)
        return [out]
    total = cu[-1]
    qkv = [s[n][:total].double() for n in ("q", "kn", "vn")]
    if c["norm"]:
        for i, w in ((0, s["qw"]), (1, s["kw"])):
            rms = torch.sqrt(qkv[i].square().sum(-1, keepdim=True) / D + EPS)
            qkv[i] = qkv[i] / rms * w.double()
    if c["rot"]:
        at = [pre[r] + len(p) - 1 for r in range(c["B"]) for p in _tree_of(parents, r, cu[r + 1] - cu[r])]
        cs = s["rope"][torch.tensor(at, device=DEV)].double()
        h = c["rot"] // 2
        turn = torch.complex(cs[:, :h], cs[:, h:])[:, None]
        for i in (0, 1):
            x = qkv[i]
            if c["interleaved"]:
                z = torch.view_as_complex(x[..., :2 * h].unflatten(-1, (h, 2)).contiguous()) * turn
                head = torch.view_as_real(z).flatten(-2)
            else:
                z = torch.complex(x[..., :h].contiguous(), x[..., h:2 * h].contiguous()) * turn
                head = torch.cat([z.real, z.imag], -1)
            qkv[i] = torch.cat([head, x[..., 2 * h:]], -1)
    out = []
    for i, x in enumerate(qkv):
        if i and c["cache"] == "e4m3":
            x = _to_e4m3(x)
        out.append(torch.cat([x, torch.zeros(s["rows"] - total, *x.shape[1:], dtype=torch.float64, device=DEV)]))
    return out


def _exact_accept(s, c):
    cu, pre = s["cu"].tolist(), s["prefix"].tolist()
    gamma, V = c["gamma"], c["V"]
    x = s["x"].cpu()[:cu[-1], :V].double().numpy()
    best = x.argmax(-1).tolist()  # numpy: the first of equal values
    am = best + [-1] * (s["rows"] - cu[-1])
    par, dr = s["parents"].tolist(), s["drafts"].tolist()
    num, bonus, toks, paths, seq = [], [], [], [], []
    for r in range(c["B"]):
        n, node, path = cu[r + 1] - cu[r], 0, [0]
        while True:
            said = best[cu[r] + node]
            step = [j for j in range(1, n) if par[r][j - 1] == node and dr[r][j - 1] == said]
            if not step:
                break
            node = step[0]
            path.append(node)
        num.append(len(path) - 1)
        bonus.append(said)
        toks.append([dr[r][j - 1] for j in path[1:]] + [said] + [-1] * (gamma + 1 - len(path)))
        paths.append(path + [-1] * (gamma + 1 - len(path)))
        seq.append(pre[r] + len(path))
    return [_i32(a) for a in (am, num, bonus, [n + 1 for n in num], toks, paths, seq)]
