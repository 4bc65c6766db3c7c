"""Timed cases of the target pass of models with a latent cache, and of the
cache append with positions on several axes.

The operators are: the append of packed rows to a paged key/value cache whose
rotation takes a position on several axes (time, height, width); the append to
a paged cache of one latent vector and one rotated part a token, and the read
of its rows; the attention of a tree or chain of drafted rows over the latents
themselves (absorbed form); and the attention of prompt rows over keys and
values expanded from the latents (expanded form).

With ``own`` false ``run`` computes a case in elementary torch operations in
float32, rounded once at the end; with ``own`` true it makes the calls that a
serving program makes of the framework. ``exact`` is the definition in float64.

Common layout: request r owns packed rows cu[r] .. cu[r+1]-1, its context of
prefix[r] tokens is in the cache, and its row j lives at cache index
prefix[r] + j. ``parents[r, j-1]`` is the parent row of row j of a tree.
"""

from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6
ROPE_BASE = 10000.0
PART = 128  # elements of a latent that share an exponent in an 8-bit cache
ROT = 64  # elements of the rotated part of a latent cache
_DT = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a few requests decoding a token of text after an image: latency
        dict(name="axes_step_b8", op="axes", B=8, lo=1, hi=1, ctx_lo=300, ctx_hi=2000, hq=28, hkv=4, D=128, page=16,
             cache="bf16", rot=128, cycle=False, norm=False, interleaved=False),
        # prompts with images and video entering an 8-bit cache
        dict(name="axes_video_b4_e4m3", op="axes", B=4, lo=500, hi=6001, ctx_lo=0, ctx_hi=1000, hq=32, hkv=8, D=128,
             page=64, cache="e4m3", rot=128, cycle=True, norm=True, interleaved=False),
        # chains of a few requests: latency
        dict(name="lappend_step_b4", op="lappend", B=4, lo=1, hi=5, ctx_lo=100, ctx_hi=3000, H=20, L=512, page=64,
             cache="bf16", tree=False, gamma=4, norm=True, interleaved=True),
        # prompts entering an 8-bit cache
        dict(name="lappend_prompt_b8_e4m3", op="lappend", B=8, lo=100, hi=4001, ctx_lo=0, ctx_hi=2000, H=64, L=512,
             page=64, cache="e4m3", tree=False, gamma=0, norm=True, interleaved=True),
        # one request decoding a single token over a short context: latency
        dict(name="lattn_decode_b1", op="lattn", B=1, gamma=1, lo=1, hi=1, ctx_lo=1500, ctx_hi=1500, H=32, L=512,
             page=64, cache="bf16", tree=False),
        # a serving batch verifying chains of up to 3 drafts over mixed contexts, all heads on the card
        dict(name="lattn_chain_b32_bf16", op="lattn", B=32, gamma=3, lo=1, hi=4, ctx_lo=1024, ctx_hi=8192, H=128, L=512,
             page=64, cache="bf16", tree=False),
        # trees of up to 16 drafts over an 8-bit cache, a share of the heads
        dict(name="lattn_tree_b16_e4m3", op="lattn", B=16, gamma=16, lo=1, hi=17, ctx_lo=500, ctx_hi=16000, H=32, L=512,
             page=32, cache="e4m3", tree=True),
        # two long contexts, a small model's heads and latent
        dict(name="lattn_long_b2_f16", op="lattn", B=2, gamma=8, lo=1, hi=9, ctx_lo=40000, ctx_hi=131000, H=20, L=256,
             page=128, cache="f16", tree=True),
        # short ragged prompts: latency
        dict(name="lprefill_short_b3", op="lprefill", B=3, lo=1, hi=190, ctx_lo=0, ctx_hi=0, H=8, L=512, n=128, page=64,
             cache="bf16"),
        # one whole prompt
        dict(name="lprefill_prompt_b1", op="lprefill", B=1, lo=4096, hi=4096, ctx_lo=0, ctx_hi=0, H=32, L=512, n=128,
             page=64, cache="bf16"),
        # chunks of prompts over what an 8-bit cache already holds of them
        dict(name="lprefill_chunk_b4_e4m3", op="lprefill", B=4, lo=300, hi=1100, ctx_lo=1000, ctx_hi=8000, H=64, L=512,
             n=128, page=64, cache="e4m3"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["axes", "lappend", "lattn", "lattn", "lprefill", "lprefill"])
    page = rng.choice([16, 32, 64, 128, 256])
    cache = rng.choice(["bf16", "f16", "e4m3"])
    L = rng.choice([256, 512, 512])
    if op == "axes":
        D = rng.choice([64, 128, 128, 256])
        hkv = rng.choice([1, 2, 4, 5, 8])
        group = rng.choice([1, 3, 4, 7])
        B = _log(rng, 1, 32)
        hi = _log(rng, 1, max(1, min(8000, 60_000_000 // (D * hkv * (group + 2) * B))))
        top = _log(rng, 1, 20000)
        return dict(op=op, B=B, lo=rng.randint(1, hi), hi=hi, ctx_lo=rng.randint(0, top), ctx_hi=top, hq=hkv * group,
                    hkv=hkv, D=D, page=page, cache=cache, rot=rng.choice([32, 64, D]), cycle=rng.random() < 0.5,
                    norm=rng.random() < 0.5, interleaved=rng.random() < 0.3)
    if op == "lappend":
        H = rng.choice([1, 4, 8, 20, 32, 64, 128])
        tree = rng.random() < 0.4
        gamma = _log(rng, 1, 32) if tree else 0
        B = _log(rng, 1, 64)
        hi = rng.randint(1, gamma + 1) if tree else _log(rng, 1, max(1, min(6000, int(300e6 / (B * (5000 + 4 * ROT * H))))))
        top = _log(rng, 1, 20000)
        return dict(op=op, B=B, lo=rng.randint(1, hi), hi=hi, ctx_lo=rng.randint(0, top), ctx_hi=top, H=H, L=L,
                    page=page, cache=cache, tree=tree, gamma=gamma, norm=rng.random() < 0.7,
                    interleaved=rng.random() < 0.6)
    if op == "lattn":
        H = rng.choice([1, 4, 8, 12, 20, 32, 64, 128])
        gamma = _log(rng, 1, 64)
        B = _log(rng, 1, 64)
        most = int(min(130000, 200e6 / (B * (L + ROT)), 60e6 / (B * H * (gamma + 1))))
        hi = _log(rng, 1, max(1, most))
        return dict(op=op, B=B, gamma=gamma, lo=1, hi=rng.randint(1, gamma + 1), ctx_lo=rng.randint(0, hi), ctx_hi=hi,
                    H=H, L=L, page=page, cache=cache, tree=rng.random() < 0.6)
    H = rng.choice([1, 4, 8, 20, 32, 64, 128])
    B = _log(rng, 1, 8)
    hi = _log(rng, 1, max(1, min(4096, int(math.sqrt(2e9 / (B * H))))))
    top = _log(rng, 1, max(1, min(8000, 1_200_000 // (B * H), int(6e8 / (B * H * hi)))))
    return dict(op=op, B=B, lo=rng.randint(1, hi), hi=hi, ctx_lo=0, ctx_hi=rng.choice([0, top]), H=H, L=L,
                n=rng.choice([64, 128, 128]), page=page, cache=cache)


def _spread(n, lo, hi):
    """n whole numbers from lo to hi, evenly spread: the case alone fixes them."""
    if n == 1:
        return [hi]
    return [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def work(case):
    c = case
    op = c["op"]
    e8 = c["cache"] == "e4m3"
    lens, ctx = _spread(c["B"], c["lo"], c["hi"]), _spread(c["B"], c["ctx_lo"], c["ctx_hi"])
    rows, keys = sum(lens), sum(ctx) + sum(lens)
    if op == "axes":
        heads, cb = c["hq"] + 2 * c["hkv"], 1 if e8 else 2
        # and the cache's rows once more on their way back
        return dict(bytes=rows * (c["D"] * (2 * heads + 2 * c["hq"] + 2 * c["hkv"] * (2 * cb + 2)) + 12 + 4 * c["rot"]),
                    flops=10 * rows * heads * c["D"])
    # a latent row of the cache
    row = c["L"] * (1 if e8 else 2) + 2 * ROT + (c["L"] // PART if e8 else 0)
    if op == "lappend":
        one = 2 * (c["L"] + ROT)
        return dict(bytes=rows * (2 * one + 2 * row + 4 * c["H"] * ROT + 4 * ROT), flops=10 * rows * (c["L"] + c["H"] * ROT))
    if op == "lattn":
        # pairs of lengths are shuffled by the seed: the mean stands for all
        pairs = rows * keys / c["B"]
        return dict(bytes=keys * row + rows * c["H"] * 2 * (2 * c["L"] + ROT),
                    flops=2 * pairs * c["H"] * (2 * c["L"] + ROT))
    pairs = rows * sum(ctx) / c["B"] + sum(n * (n + 1) // 2 for n in lens)
    return dict(bytes=keys * row + rows * c["H"] * 2 * (2 * c["n"] + ROT) + c["H"] * 2 * c["n"] * c["L"] * 2,
                flops=2 * keys * c["H"] * c["L"] * 2 * c["n"] + 2 * pairs * c["H"] * (2 * c["n"] + ROT))


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
    """[..., n] float32 -> codes and exponent bytes, one exponent for each n."""
    amax = x.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(amax / 448.0)  # amax / 448 = m 2^e, m in [0.5, 1)
    e = torch.where(m == 0.5, e - 1, e)
    e = torch.where(amax == 0, torch.zeros_like(e), e).clamp(-100, 119)
    codes = (x * _power(-e)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8).squeeze(-1)


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


def _latents(g, nb, c):
    """A filled latent cache: normed latents and rotated parts."""
    shape = (nb, c["page"], c["L"])
    dt = torch.float16 if c["cache"] == "f16" else torch.bfloat16
    rope = torch.randn(nb, c["page"], ROT, generator=g, device=DEV, dtype=dt)
    if c["cache"] != "e4m3":
        return torch.randn(shape, generator=g, device=DEV, dtype=dt), rope, None
    out = torch.empty(shape, dtype=torch.float8_e4m3fn, device=DEV)
    scale = torch.empty(nb, c["page"], c["L"] // PART, dtype=torch.uint8, device=DEV)
    flat, fs = out.view(-1, PART), scale.view(-1)
    for i in range(0, flat.shape[0], 1 << 20):
        x = torch.randn(min(1 << 20, flat.shape[0] - i), PART, generator=g, device=DEV)
        flat[i:i + x.shape[0]], fs[i:i + x.shape[0]] = _e4m3(x)
    return out, rope, scale


def _turns(n, rot):
    """Cosines, then sines, of positions 0 .. n - 1."""
    at = torch.arange(n, device=DEV, dtype=torch.float64)
    f = ROPE_BASE ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    a = at[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def _positions(rng, start, n):
    """Positions on three axes of n tokens: text, and pictures of a grid each."""
    out, at = [], start
    while len(out) < n:
        for _ in range(rng.randint(1, 40)):
            out.append((at, at, at))
            at += 1
        t, h, w = rng.randint(1, 4), rng.randint(2, 24), rng.randint(2, 24)
        out += [(at + i, at + j, at + k) for i in range(t) for j in range(h) for k in range(w)]
        at += max(t, h, w)
    return out[:n]


def prepare(case, seed):
    c = case
    rng = random.Random(seed * 7919 + 13)
    g = _gen(seed)
    op, B = c["op"], c["B"]
    lens, ctx = _spread(B, c["lo"], c["hi"]), _spread(B, c["ctx_lo"], c["ctx_hi"])
    rng.shuffle(lens)
    rng.shuffle(ctx)
    cu = _cum(lens)
    rows = -(-cu[-1] // 16) * 16  # the captured tier: rows past the total are padding
    table, nb = _blocks(rng, [a + b for a, b in zip(ctx, lens)], c["page"])
    dt = torch.float16 if c["cache"] == "f16" else torch.bfloat16
    e8 = c["cache"] == "e4m3"
    s = dict(c=dict(c), cu=_i32(cu), rows=rows, table=_i32(table), prefix=_i32(ctx), dt=dt, parents=None)
    if c.get("tree"):
        s["parents"] = _i32(_make_parents(rng, B, c["gamma"], True))
    if op == "axes":
        D, hq, hkv = c["D"], c["hq"], c["hkv"]
        # one buffer of a fused projection: the three are views of its rows
        qkv = torch.randn(rows, (hq + 2 * hkv) * D, generator=g, device=DEV, dtype=dt)
        s["q"] = qkv[:, :hq * D].unflatten(1, (hq, D))
        s["kn"] = qkv[:, hq * D:(hq + hkv) * D].unflatten(1, (hkv, D))
        s["vn"] = qkv[:, (hq + hkv) * D:].unflatten(1, (hkv, D))
        kind = torch.float8_e4m3fn if e8 else dt
        for x in "kv":
            s[x] = torch.zeros(nb, hkv, c["page"], D, device=DEV).to(kind)
            s[x + "s"] = torch.full((nb, hkv, c["page"]), 127, dtype=torch.uint8, device=DEV) if e8 else None
        s["qw"] = s["kw"] = None
        if c["norm"]:
            s["qw"] = (1 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(dt)
            s["kw"] = (1 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(dt)
        at = []
        for n, p in zip(lens, ctx):
            at += _positions(rng, p // 2, n)  # pictures before took fewer positions than tokens
        at += [(0, 0, 0)] * (rows - len(at))
        s["positions"] = _i32(list(zip(*at)))
        half = c["rot"] // 2
        s["axis"] = [i % 3 for i in range(half)] if c["cycle"] else \
            [0] * (half // 4) + [1] * (3 * half // 8) + [2] * (half - half // 4 - 3 * half // 8)
        s["rope"] = _turns(int(max(map(max, at))) + 1, c["rot"])
        return s
    L, H = c["L"], c["H"]
    if op == "lappend":
        # the projection's rows: latent, then the part that turns
        s["kvn"] = torch.randn(rows, L + ROT, generator=g, device=DEV, dtype=dt)
        s["q"] = torch.randn(rows, H, 128 + ROT, generator=g, device=DEV, dtype=dt)[..., 128:]
        s["w"] = (1 + 0.1 * torch.randn(L, generator=g, device=DEV)).to(dt) if c["norm"] else None
        s["latent"] = torch.zeros(nb, c["page"], L, device=DEV).to(torch.float8_e4m3fn if e8 else dt)
        s["lrope"] = torch.zeros(nb, c["page"], ROT, device=DEV, dtype=dt)
        s["lscale"] = torch.full((nb, c["page"], L // PART), 127, dtype=torch.uint8, device=DEV) if e8 else None
        s["rope"] = _turns(c["ctx_hi"] + c["hi"] + 1, ROT)
        return s
    s["latent"], s["lrope"], s["lscale"] = _latents(g, nb, c)
    if op == "lattn":
        s["ql"] = torch.randn(rows, H, L, generator=g, device=DEV, dtype=dt)
        s["qr"] = torch.randn(rows, H, 128 + ROT, generator=g, device=DEV, dtype=dt)[..., 128:]
        s["scale"] = (128 + ROT) ** -0.5 * (512 / L) ** 0.5
        return s
    n = c["n"]
    s["q"] = (1.5 * torch.randn(rows, H, n + ROT, generator=g, device=DEV)).to(dt)
    # one projection's weight: a head's keys, then its values
    w = (torch.randn(H, 2 * n, L, generator=g, device=DEV) * L ** -0.5).to(dt)
    s["wk"], s["wv"] = w[:, :n], w[:, n:]
    s["keys"] = sum(lens) + sum(ctx)
    s["scale"] = (n + ROT) ** -0.5
    return s


# ------------------------------------------------------------------ plain form

def _row_of(s):
    """For each packed row: its request, its index there, whether it is a real row."""
    cu = s["cu"].long()
    at = torch.arange(s["rows"], device=DEV)
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


def _values(codes, scale):
    x = codes.float()
    if scale is None:
        return x
    return (x.unflatten(-1, (scale.shape[-1], -1)) * _power(scale.int()[..., None] - 127)).flatten(-2)


def _norm(x, w):
    return x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()


def _rotate(x, co, si, interleaved):
    """x [..., n] float32, its first pairs turned by cosines and sines [..., h]."""
    h = co.shape[-1]
    if interleaved:
        a, b = x[..., 0:2 * h:2], x[..., 1:2 * h:2]
        turned = torch.stack([a * co - b * si, b * co + a * si], -1).flatten(-2)
    else:
        a, b = x[..., :h], x[..., h:2 * h]
        turned = torch.cat([a * co - b * si, b * co + a * si], -1)
    return torch.cat([turned, x[..., 2 * h:]], -1)


def _place(s, r, j, ok):
    """Page and offset of each packed row (padding goes to the page of nobody)."""
    page = s["c"]["page"]
    slot = s["prefix"].long()[r] + j
    block = s["table"].long()[r, slot // page]
    pool = s["k"] if "k" in s else s["latent"]
    return torch.where(ok, block, pool.shape[0] - 1), slot % page


def _plain_axes(s):
    c = s["c"]
    r, j, ok = _row_of(s)
    q, k, v = _norm(s["q"].float(), s["qw"]), _norm(s["kn"].float(), s["kw"]), s["vn"].float()
    half = c["rot"] // 2
    axis = torch.tensor(s["axis"], device=DEV)
    at = s["positions"].long()[axis].t()  # [rows, half]
    pair = torch.arange(half, device=DEV)
    co, si = s["rope"][at, pair][:, None], s["rope"][at, half + pair][:, None]
    q, k = _rotate(q, co, si, c["interleaved"]), _rotate(k, co, si, c["interleaved"])
    block, off = _place(s, r, j, ok)
    back = []
    for name, x in (("k", k), ("v", v)):
        if c["cache"] == "e4m3":
            codes, e = _e4m3(x)
            s[name].view(torch.uint8)[block, :, off] = codes.view(torch.uint8)
            s[name + "s"][block, :, off] = e
            x = s[name].view(torch.uint8)[block, :, off].view(torch.float8_e4m3fn).float()
            x = x * _power(s[name + "s"][block, :, off].int()[..., None] - 127)
        else:
            s[name][block, :, off] = x.to(s["dt"])
            x = s[name][block, :, off]
        back.append(torch.where(ok[:, None, None], x, 0.0).to(s["dt"]))
    return [torch.where(ok[:, None, None], q, 0.0).to(s["dt"])] + back


def _plain_lappend(s):
    c = s["c"]
    L = c["L"]
    r, j, ok = _row_of(s)
    depth = j
    if s["parents"] is not None:
        depth = (_ancestors(s, c).sum(-1) - 1)[r, j]
    cs = s["rope"][s["prefix"].long()[r] + depth]
    co, si = cs[:, :ROT // 2], cs[:, ROT // 2:]
    x = s["kvn"].float()
    lat = _norm(x[:, :L], s["w"])
    turned = _rotate(x[:, L:], co, si, c["interleaved"])
    q = _rotate(s["q"].float(), co[:, None], si[:, None], c["interleaved"])
    block, off = _place(s, r, j, ok)
    s["lrope"][block, off] = turned.to(s["dt"])
    if c["cache"] == "e4m3":
        codes, e = _e4m3(lat.unflatten(-1, (L // PART, PART)))
        s["latent"].view(torch.uint8)[block, off] = codes.flatten(-2).view(torch.uint8)
        s["lscale"][block, off] = e
        lat = _values(s["latent"].view(torch.uint8)[block, off].view(torch.float8_e4m3fn), s["lscale"][block, off])
    else:
        s["latent"][block, off] = lat.to(s["dt"])
        lat = s["latent"][block, off]
    return [torch.where(ok[:, None, None], q, 0.0).to(s["dt"]), torch.where(ok[:, None], lat, 0.0).to(s["dt"]),
            torch.where(ok[:, None], s["lrope"][block, off], 0.0).to(s["dt"])]


def _cached(s, table):
    """Latents and rotated parts of the tables' pages, [..., tokens, n] float32."""
    lat = s["latent"].view(torch.uint8)[table].view(torch.float8_e4m3fn) if s["lscale"] is not None else s["latent"][table]
    lat = _values(lat, None if s["lscale"] is None else s["lscale"][table])
    return lat.flatten(-3, -2), s["lrope"][table].float().flatten(-3, -2)


def _plain_lattn(s):
    c = s["c"]
    B, H, n, rows = c["B"], c["H"], c["gamma"] + 1, s["rows"]
    r, j, ok = _row_of(s)
    lat, rope = _cached(s, s["table"].long())
    T = lat.shape[1]
    q = torch.zeros(B, n + 1, H, c["L"] + ROT, device=DEV)
    q[r, torch.where(ok, j, n)] = torch.cat([s["ql"].float(), s["qr"].float()], -1)
    q = q[:, :n].reshape(B, n * H, c["L"] + ROT)
    sc = torch.matmul(q, torch.cat([lat, rope], -1).transpose(1, 2).contiguous()) * s["scale"]
    cu = s["cu"].long()
    lens, pre = cu[1:] - cu[:-1], s["prefix"].long()
    key = torch.arange(T, device=DEV)
    live = key < (pre + lens)[:, None]
    i = (key - pre[:, None]).clamp(0, n - 1)
    seen = torch.gather(_ancestors(s, c), 2, i[:, None, :].expand(B, n, T))
    seen = (seen | (key < pre[:, None])[:, None]) & live[:, None]
    sc = sc.view(B, n, H, T).masked_fill(~seen[:, :, None], -math.inf).view(B, n * H, T)
    sc = torch.exp(sc - sc.amax(-1, keepdim=True))
    total = sc.sum(-1, keepdim=True)
    o = torch.matmul(sc, lat.masked_fill(~live[..., None], 0.0)) / total
    o = o.view(B, n, H, c["L"])
    return [torch.where(ok[:, None, None], o[r, j], 0.0).to(s["dt"])]


def _plain_lprefill(s):
    c = s["c"]
    H, n = c["H"], c["n"]
    cu, pre = s["cu"].tolist(), s["prefix"].tolist()
    out = torch.zeros(s["rows"], H, n, device=DEV)
    wk, wv = s["wk"].float(), s["wv"].float()
    for r in range(c["B"]):
        rows, T = cu[r + 1] - cu[r], pre[r] + cu[r + 1] - cu[r]
        lat, rope = _cached(s, s["table"][r, :-(-T // c["page"])].long())
        lat, rope = lat[:T], rope[:T]
        q = s["q"][cu[r]:cu[r + 1]].float().transpose(0, 1)
        hidden = torch.arange(T, device=DEV) > torch.arange(pre[r], T, device=DEV)[:, None]
        at_once = max(1, int(2e9 / (4 * rows * T)))
        for h in range(0, H, at_once):
            k = torch.matmul(lat, wk[h:h + at_once].transpose(1, 2).contiguous())
            v = torch.matmul(lat, wv[h:h + at_once].transpose(1, 2).contiguous())
            a = torch.matmul(q[h:h + at_once, :, :n], k.transpose(1, 2).contiguous())
            a += torch.matmul(q[h:h + at_once, :, n:], rope.t().contiguous())
            a = (a * s["scale"]).masked_fill_(hidden, -math.inf)
            a = torch.exp(a - a.amax(-1, keepdim=True))
            out[cu[r]:cu[r + 1], h:h + at_once] = (torch.matmul(a, v) / a.sum(-1, keepdim=True)).transpose(0, 1)
    return [out.to(s["dt"])]


# ------------------------------------------------------------------ the framework's calls

def _own(s):
    import dspark_verify_scheduling_amd as dv

    c = s["c"]
    op, B, rows = c["op"], c["B"], s["rows"]
    new = "out" not in s
    if op == "axes":
        if new:
            s["cache"] = dv.KvCache(s["k"], s["v"], s["ks"], s["vs"])
            s["out"] = dv.alloc_append_outputs(rows, c["hq"], s["cache"])
            s["back"] = dv.alloc_kv_read_outputs(rows, s["cache"])
            for x in (s["out"].q_out, s["back"].k_out, s["back"].v_out):
                x.zero_()
        dv.dspark_kv_append_axes(B, s["q"], s["kn"], s["vn"], rows, s["cu"], s["prefix"], s["positions"], s["axis"],
                                 s["table"], s["cache"], s["out"], s["rope"], q_weight=s["qw"], k_weight=s["kw"],
                                 eps=EPS, rope_interleaved=c["interleaved"])
        dv.dspark_kv_read(B, rows, s["cu"], s["prefix"], s["table"], s["cache"], s["back"])
        return [s["out"].q_out, s["back"].k_out, s["back"].v_out]
    if new:
        s["cache"] = dv.LatentCache(s["latent"], s["lrope"], s["lscale"])
    if op == "lappend":
        if new:
            s["out"] = dv.alloc_latent_append_outputs(rows, c["H"], s["cache"])
            s["back"] = dv.alloc_latent_read_outputs(rows, s["cache"])
            for x in (s["out"].q_rope, s["back"].latent_out, s["back"].rope_out):
                x.zero_()
        dv.dspark_latent_append(B, s["kvn"], rows, s["cu"], s["prefix"], s["table"], s["cache"], s["out"],
                                q_rope=s["q"], weight=s["w"], eps=EPS, rope=s["rope"],
                                rope_interleaved=c["interleaved"], gamma=c["gamma"] if c["tree"] else 0,
                                tree_parents=s["parents"])
        dv.dspark_latent_read(B, rows, s["cu"], s["prefix"], s["table"], s["cache"], s["back"])
        return [s["out"].q_rope, s["back"].latent_out, s["back"].rope_out]
    if op == "lattn":
        if new:
            s["out"] = dv.alloc_latent_attention_outputs(B, c["gamma"], rows, c["H"], s["cache"])
            s["out"].out.zero_()
        dv.dspark_latent_attention(B, c["gamma"], s["ql"], s["qr"], rows, s["cu"], s["prefix"], s["table"], s["cache"],
                                   s["scale"], s["out"], tree_parents=s["parents"])
        return [s["out"].out]
    if new:
        s["out"] = dv.alloc_latent_prefill_outputs(B, rows, s["keys"], c["H"], c["n"], s["cache"])
        s["out"].out.zero_()
    dv.dspark_latent_prefill(B, s["q"], s["wk"], s["wv"], rows, s["keys"], s["cu"], s["prefix"], s["table"], s["cache"],
                             s["scale"], s["out"])
    return [s["out"].out]


def run(state):
    if own:
        return _own(state)
    return {"axes": _plain_axes, "lappend": _plain_lappend, "lattn": _plain_lattn,
            "lprefill": _plain_lprefill}[state["c"]["op"]](state)


# ------------------------------------------------------------------ the definition in 64 bits

def _tree_of(parents, r, n):
    """Row j's path from the root, for the n rows of request r."""
    paths = [[0]]
    for j in range(1, n):
        paths.append(paths[j - 1 if parents is None else parents[r][j - 1]] + [j])
    return paths


def _to_e4m3(x):
    """The value that 8 bits keep of each row's elements: steps of 2^-3 of the leading power of two."""
    top = x.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.ceil(torch.log2(top / 448)), torch.zeros_like(top)).clamp(-100, 119)
    e = torch.where(top > 448 * torch.exp2(e), e + 1, e)
    y = x * torch.exp2(-e)
    lead = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(lead - 3)
    return torch.round(y / step) * step * torch.exp2(e)


def _turn64(x, angle, interleaved):
    """x [rows, heads, n] float64, its pairs turned by `angle` (cosine and sine [rows, h])."""
    turn = torch.complex(*angle)[:, None]
    h = turn.shape[-1]
    if interleaved:
        z = torch.view_as_complex(x[..., :2 * h].unflatten(-1, (h, 2)).contiguous()) * turn
        head = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(x[..., :h].contiguous(), x[..., h:2 * h].contiguous()) * turn
        head = torch.cat([z.real, z.imag], -1)
    return torch.cat([head, x[..., 2 * h:]], -1)


def _norm64(x, w):
    return x if w is None else x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()


def _padded(x, rows):
    return torch.cat([x, torch.zeros(rows - x.shape[0], *x.shape[1:], dtype=torch.float64, device=DEV)])


def _span64(s, r, T):
    """The first T cached latents and rotated parts of request r, float64."""
    at = torch.arange(T, device=DEV)
    b, o = s["table"][r].long()[at // s["c"]["page"]], at % s["c"]["page"]
    if s["lscale"] is None:
        lat = s["latent"][b, o].double()
    else:
        lat = s["latent"].view(torch.uint8)[b, o].view(torch.float8_e4m3fn).double().view(T, -1, PART)
        lat = (lat * torch.exp2(s["lscale"][b, o].double() - 127)[..., None]).flatten(1)
    return lat, s["lrope"][b, o].double()


def exact(case, seed):
    c = case
    op = c["op"]
    s = prepare(c, seed)
    cu, pre = s["cu"].tolist(), s["prefix"].tolist()
    total, rows = cu[-1], s["rows"]
    parents = None if s["parents"] is None else s["parents"].tolist()
    if op == "axes":
        half = c["rot"] // 2
        at = s["positions"][:, :total].long()
        co, si = torch.empty(2, total, half, dtype=torch.float64, device=DEV)
        for i, ax in enumerate(s["axis"]):
            co[:, i], si[:, i] = s["rope"][at[ax], i].double(), s["rope"][at[ax], half + i].double()
        out = []
        for name, w, turns in (("q", s["qw"], True), ("kn", s["kw"], True), ("vn", None, False)):
            x = _norm64(s[name][:total].double(), w)
            x = _turn64(x, (co, si), c["interleaved"]) if turns else x
            out.append(_padded(_to_e4m3(x) if c["cache"] == "e4m3" and name != "q" else x, rows))
        return out
    if op == "lappend":
        L = c["L"]
        at = [pre[r] + len(p) - 1 for r in range(c["B"]) for p in _tree_of(parents, r, cu[r + 1] - cu[r])] \
            if parents is not None else [pre[r] + j for r in range(c["B"]) for j in range(cu[r + 1] - cu[r])]
        cs = s["rope"][torch.tensor(at, device=DEV)].double()
        angle = cs[:, :ROT // 2].contiguous(), cs[:, ROT // 2:].contiguous()
        x = s["kvn"][:total].double()
        lat = _norm64(x[:, :L], s["w"])
        if c["cache"] == "e4m3":
            lat = _to_e4m3(lat.view(total, -1, PART)).flatten(1)
        turned = _turn64(x[:, None, L:], angle, c["interleaved"])[:, 0]
        q = _turn64(s["q"][:total].double(), angle, c["interleaved"])
        return [_padded(y, rows) for y in (q, lat, turned)]
    H = c["H"]
    if op == "lattn":
        out = torch.zeros(rows, H, c["L"], dtype=torch.float64, device=DEV)
        for r in range(c["B"]):
            n = cu[r + 1] - cu[r]
            T = pre[r] + n
            lat, rope = _span64(s, r, T)
            see = torch.zeros(n, T, dtype=torch.bool, device=DEV)
            see[:, :pre[r]] = True
            pairs = [(j, pre[r] + i) for j, p in enumerate(_tree_of(parents, r, n)) for i in p]
            see[tuple(torch.tensor(pairs, device=DEV).T)] = True
            ql, qr = s["ql"][cu[r]:cu[r + 1]].double(), s["qr"][cu[r]:cu[r + 1]].double()
            for j in range(n):
                a = (ql[j] @ lat.T + qr[j] @ rope.T) * s["scale"]
                out[cu[r] + j] = torch.softmax(a.masked_fill(~see[j], -math.inf), -1) @ lat
        return [out]
    n = c["n"]
    out = torch.zeros(rows, H, n, dtype=torch.float64, device=DEV)
    for r in range(c["B"]):
        T = pre[r] + cu[r + 1] - cu[r]
        lat, rope = _span64(s, r, T)
        future = torch.ones(T - pre[r], T, dtype=torch.bool, device=DEV).triu(pre[r] + 1)
        for h in range(H):
            q = s["q"][cu[r]:cu[r + 1], h].double()
            k = torch.cat([lat @ s["wk"][h].double().T, rope], 1)
            a = (q @ k.T * s["scale"]).masked_fill(future, -math.inf)
            out[cu[r]:cu[r + 1], h] = torch.softmax(a, -1) @ (lat @ s["wv"][h].double().T)
    return [out]
