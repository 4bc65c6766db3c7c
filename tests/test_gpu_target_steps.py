"""GPU tests of the target pass as a serving loop runs it: plan and pack, append,
attention, accept and commit, step after step; and of calls at the edges of what
the entry points allow (large batches, long shares, strided rows, two at once).

The loop's last check: with the cache's own rows as keys and values, a query
that differs from the float64 one by its rounding (u relative) moves a score by
at most u * scale * sum |q||k|. That adds u to (D + 16) w in the attention
bound of test_gpu_target.py. A committed token's logit is then at least the
largest one less twice sum_i |W_i| times that bound, plus the float32 product's
hq D w sum |out||W|.
"""

import numpy as np
import pytest
import torch

import dspark_verify_scheduling_amd as dv
import oracle
from _gpu import DEV, say, up
from test_gpu_target import (TYPES, W, Batch, bits, f64, get, i32, make_cache, put, within)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu(hip):
    return hip


class Model:
    """One layer: rows of a token are looked up, logits are a product with the
    attention's output."""

    def __init__(self, rng, kind, V, hq, hkv, D, positions):
        self.dt, self.u = TYPES[kind][1], TYPES[kind][2]
        self.V, self.hq, self.hkv, self.D = V, hq, hkv, D
        x = rng.normal(0, 1, (V, hq + 2 * hkv, D)).astype(np.float32)
        self.rows = torch.from_numpy(x).to(self.dt).to(DEV)
        w = rng.uniform(0.5, 1.5, (2, D)).astype(np.float32)
        self.qw, self.kw = torch.from_numpy(w).to(self.dt).to(DEV)
        ang = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(D // 2) / (D // 2))
        self.rope = up(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32))
        self.out = up(rng.normal(0, 1, (hq * D, V)).astype(np.float32))
        self.scale = D ** -0.5

    def append(self, B, gamma, ids, n, cu, prefix, table, cache, parents=None):
        """The queries of packed rows whose ids are given, keys and values written."""
        x = self.rows[ids.long()]
        hq, hkv = self.hq, self.hkv
        o = dv.alloc_append_outputs(n, hq, cache)
        dv.dspark_kv_append(B, gamma, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], n, cu, prefix,
                            table, cache, o, self.qw, self.kw, 1e-6, self.rope,
                            tree_parents=parents)
        return o

    def fill(self, tokens, r, gamma, cache, table):
        """Tokens of request r into its pages, a chain of gamma + 1 at a time."""
        for lo in range(0, len(tokens), gamma + 1):
            part = tokens[lo:lo + gamma + 1]
            o = self.append(1, gamma, i32(part), len(part), i32([0, len(part)]), i32([lo]),
                            i32(table[r:r + 1]), cache)
            assert o.append_meta.tolist() == [len(part), 0]

    def heads64(self):
        f = [f64(t) for t in (self.rows, self.qw, self.kw, self.rope)]
        return f

    def greedy64(self, host, tokens, n):
        """The next n tokens in float64, nothing rounded."""
        rows, qw, kw, rope = host
        tokens, start = list(tokens), len(tokens)
        hq, hkv, D = self.hq, self.hkv, self.D
        while len(tokens) < start + n:
            T = len(tokens)
            k = np.stack([[oracle.norm_rope(rows[t, hq + h], kw, 1e-6, rope[p], D, False)
                           for h in range(hkv)] for p, t in enumerate(tokens)], 1)
            v = np.stack([rows[t, hq + hkv:] for t in tokens], 1)
            q = np.stack([oracle.norm_rope(rows[tokens[-1], h], qw, 1e-6, rope[T - 1], D, False)
                          for h in range(hq)])[None]
            o, *_ = oracle.tree_attention(q, k, v, T - 1, None, self.scale)
            tokens.append(int(np.argmax(o.reshape(-1) @ f64(self.out))))
        return tokens[start:]


@pytest.mark.parametrize("kind,tree", [("bf16", True), ("f16", False), ("e4m3", True)])
def test_serving_loop(kind, tree):
    """Steps of a small batch: what the loop commits is what decoding one token
    at a time would, the cache holds the committed tokens' rows bit for bit."""
    say(f"serving loop {kind} tree={tree}")
    rng = np.random.default_rng(17)
    B, gamma, hq, hkv, D, page, V, steps = 5, 6, 4, 2, 64, 16, 40, 6
    m = Model(rng, kind, V, hq, hkv, D, 160)
    host = m.heads64()
    prompts = [1, 15, 16, 31, 40]
    seqs = [rng.integers(0, V, n).tolist() for n in prompts]
    most = [n + steps * (gamma + 1) + gamma + 1 for n in prompts]
    b = Batch(1, [1] * B, most, gamma, page, False)
    cache = make_cache(kind, b.nb, hkv, page, D)
    for r in range(B):
        m.fill(seqs[r][:-1], r, gamma, cache, b.table)
    table = i32(b.table)
    cap = B * (gamma + 1)
    po = dv.alloc_plan_outputs(B, gamma, DEV)
    ko = dv.alloc_pack_outputs(B, cap, DEV)
    o = None
    ta = dv.alloc_tree_accept_outputs(B, gamma, cap, V, dv.F32, DEV)
    cm = torch.empty(2, dtype=torch.int32, device=DEV)
    alpha, theta = up(np.zeros(B + 1, np.float32)), up(np.linspace(0, 1, cap + 1).astype(np.float32))
    accepted = moved = 0
    for step in range(steps):
        # drafts: the right continuation down one path (cut short at random), others beside it
        drafts = rng.integers(0, V, (B, gamma)).astype(np.int32)
        parents = np.tile(np.arange(gamma, dtype=np.int32), (B, 1))
        for r in range(B):
            right = m.greedy64(host, seqs[r], 4)[:rng.integers(0, 5)]
            at = 0
            for j in range(1, gamma + 1):
                if tree and rng.random() < 0.4:
                    parents[r, j - 1] = rng.integers(0, j)  # some wrong row
                    continue
                if not tree and len(right) == 0:
                    break
                parents[r, j - 1] = at if tree else j - 1
                at = j
                if right:
                    drafts[r, j - 1] = right.pop(0)
        prefix = i32([len(s) - 1 for s in seqs])
        anchors, dr = i32([s[-1] for s in seqs]), i32(drafts)
        par = i32(parents) if tree else None
        conf = up(np.sort(rng.uniform(0.3, 1, (B, gamma)).astype(np.float32), 1)[:, ::-1].copy())
        dv.dspark_plan_pack(B, gamma, dv.IN_SURVIVAL, conf, None, 2, gamma + 1, 0.05, 0, -1, 1.0,
                            alpha, theta, po, anchors, dr, [cap], prefix, ko)
        cu = ko.cu_seqlens
        ids = torch.where(torch.arange(cap, device=DEV) < cu[B], ko.packed_ids, 0)
        ap = m.append(B, gamma, ids, cap, cu, prefix, table, cache, par)
        if o is None:
            o = dv.alloc_attention_outputs(B, gamma, cap, hq, cache)
        dv.dspark_tree_attention(B, gamma, ap.q_out, cap, cu, prefix, table, cache, m.scale, o,
                                 tree_parents=par)
        logits = o.out.float().flatten(1) @ m.out
        dv.dspark_tree_accept(B, gamma, V, dv.F32, logits, V, cap, cu, dr, par, prefix, ta)
        dv.dspark_kv_commit(B, gamma, ta.path_rows, ta.num_correct, prefix, table, cache, cm)
        torch.cuda.synchronize()
        rows = int(cu[B])
        assert ap.append_meta.tolist() == o.attention_meta.tolist() == [rows, 0]
        assert ta.accept_meta.tolist()[1] == 0 and cm.tolist()[1] == 0
        moved += cm.tolist()[0]
        n, tok = ta.commit_lens.tolist(), ta.out_tokens.tolist()
        assert ta.new_seq_lens.tolist() == [len(s) - 1 + k for s, k in zip(seqs, n)]
        for r in range(B):
            accepted += n[r] - 1
            seqs[r] += tok[r][:n[r]]
    say(f"accepted {accepted}, moved {moved}")
    assert accepted >= steps and (moved > 0 or not tree)

    again = make_cache(kind, b.nb, hkv, page, D)
    for r, s in enumerate(seqs):
        m.fill(s[:-1], r, gamma, again, b.table)
        for pg, of in b.slots(r, 0, len(s) - 1):
            assert torch.equal(bits(cache.k)[pg, :, of], bits(again.k)[pg, :, of])
            assert torch.equal(bits(cache.v)[pg, :, of], bits(again.v)[pg, :, of])
    rows64, qw, _, rope = host
    Wf = f64(m.out)
    for r, s in enumerate(seqs):
        T = len(s) - 1
        k, v = (get(again, b.slots(r, 0, T), x).transpose(1, 0, 2) for x in "kv")
        for p in range(prompts[r] - 1, T):
            q = np.stack([oracle.norm_rope(rows64[s[p], h], qw, 1e-6, rope[p], D, False)
                          for h in range(hq)])[None]
            ref, _, mean_abs, top = oracle.tree_attention(q, k[:, :p + 1], v[:, :p + 1], p, None,
                                                          m.scale)
            t = ((D + 16) * W + m.u) * top[..., None] + 2 * W
            bound = m.u * np.abs(ref) + (m.u + 2 * t + (p + 33) * W) * mean_abs
            if kind == "f16":
                bound = bound + (p + 1) * 2.0 ** -25 * np.abs(v).max()
            lg = ref.reshape(-1) @ Wf
            err = (bound.reshape(-1) @ np.abs(Wf) +
                   hq * D * W * ((np.abs(ref) + bound).reshape(-1) @ np.abs(Wf)))
            assert lg[s[p + 1]] + err[s[p + 1]] >= (lg - err).max(), (r, p)


def ref_long(q, k, v, prefix, scale):
    """Chain rows q [n, H, D] over k, v [H, keys, D], float64 on the GPU: out, the
    weighted mean of |v|, the largest scale * sum |q||k|."""
    q, k, v = q.double().transpose(0, 1), k.double(), v.double()
    s = torch.matmul(q, k.transpose(1, 2).contiguous()) * scale
    top = (torch.matmul(q.abs(), k.abs().transpose(1, 2).contiguous()) * abs(scale)).amax(-1)
    n, T = q.shape[1], k.shape[1]
    late = torch.arange(T, device=DEV)[None] > prefix + torch.arange(n, device=DEV)[:, None]
    p = torch.softmax(s.masked_fill(late, -float("inf")), -1)
    return [x.transpose(0, 1).cpu().numpy() for x in
            (torch.matmul(p, v), torch.matmul(p, v.abs()), top)]


@pytest.mark.parametrize("kind,B,hkv,group,D,ctx", [
    ("bf16", 1, 12, 1, 64, 190_000),  # shares of more than 64 tiles, a few rows
    ("f16", 2, 8, 5, 128, 70_003),  # the same of 32 keys, five tiles of rows
    ("bf16", 70, 2, 2, 256, 300),  # a batch beyond a wave
    ("f16", 700, 1, 3, 64, 90),  # beyond a workgroup
])
def test_attention_sizes(kind, B, hkv, group, D, ctx):
    say(f"attention sizes {kind} B={B} hkv={hkv} group={group} D={D} ctx={ctx}")
    _, dt, u = TYPES[kind]
    gamma, page, hq = 15, 256 if ctx > 1000 else 16, hkv * group
    rng = np.random.default_rng(B)
    lens = [16 if ctx > 1000 else int(x) for x in rng.integers(1, 17, B)]
    b = Batch(B, lens, [ctx - (ctx // 3) * (r % 3) for r in range(B)], gamma, page, False)
    cache = dv.alloc_kv_cache(b.nb, hkv, page, D, TYPES[kind][0], DEV)
    torch.manual_seed(B)
    cache.k.normal_()
    cache.v.normal_()
    # queries and outputs inside wider rows
    wide = torch.randn(b.rows, 2 * hq, D, device=DEV).to(dt)
    q = wide[:, hq:]
    res = torch.full((b.rows, 2 * hq, D), -7.0, device=DEV, dtype=dt)
    o = dv.alloc_attention_outputs(B, gamma, b.rows, hq, cache)._replace(out=res[:, :hq])
    dv.dspark_tree_attention(B, gamma, q, b.rows, *b.args(), cache, D ** -0.5, o)
    torch.cuda.synchronize()
    assert o.attention_meta.tolist() == [int(b.cu[-1]), 0]
    assert bool((res[:, hq:] == -7).all()) and bool((res[int(b.cu[-1]):] == -7).all())
    for r in range(B) if B < 10 else rng.choice(B, 8, replace=False):
        T = b.ctx[r] + b.lens[r]
        pages = torch.tensor(b.table[r][:-(-T // page)].tolist(), device=DEV)
        k, v = (t[pages].transpose(0, 1).reshape(hkv, -1, D)[:, :T].repeat_interleave(group, 0)
                for t in (cache.k, cache.v))
        c0, c1 = int(b.cu[r]), int(b.cu[r + 1])
        ref, mean_abs, top = ref_long(q[c0:c1], k, v, b.ctx[r], D ** -0.5)
        t = (D + 16) * W * top[..., None] + 2 * W
        bound = u * np.abs(ref) + (u + 2 * t + (T + 32) * W) * mean_abs
        if kind == "f16":
            bound += T * 2.0 ** -25 * float(v.abs().max())
        within(f64(res[c0:c1, :hq]), ref, bound, f"request {r}")


def test_two_calls_at_once():
    """Two streams with a workspace each, over one cache: the result of one."""
    say("two calls at once")
    D, hkv, hq, gamma, page = 128, 2, 16, 8, 32
    b = Batch(3, [9, 4, 7], [3000, 100, 900], gamma, page, True)
    cache = make_cache("e4m3", b.nb, hkv, page, D)
    rng = np.random.default_rng(0)
    for r in range(b.B):
        T = b.ctx[r] + b.lens[r]
        put(cache, b.slots(r, 0, T), *rng.normal(0, 1, (2, T, hkv, D)).astype(np.float32))
    qs = [torch.randn(b.rows, hq, D, device=DEV).bfloat16() for _ in range(2)]
    args, par = b.args(), b.par()
    outs = [dv.alloc_attention_outputs(b.B, gamma, b.rows, hq, cache) for _ in range(2)]
    want = []
    for q, o in zip(qs, outs):
        dv.dspark_tree_attention(b.B, gamma, q, b.rows, *args, cache, 0.1, o, tree_parents=par)
        torch.cuda.synchronize()
        want.append(o.out[:int(b.cu[-1])].clone())
        o.out.zero_()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for q, o, s in zip(qs, outs, streams):
            with torch.cuda.stream(s):
                dv.dspark_tree_attention(b.B, gamma, q, b.rows, *args, cache, 0.1, o,
                                         tree_parents=par)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o.out[:int(b.cu[-1])], w)


@pytest.mark.parametrize("gamma", [5, 40])
def test_status_of_every_request_of_a_large_batch(gamma):
    """One bad request anywhere in a batch of 300 shows in the status of append,
    read and commit, and nothing else changes."""
    say(f"status of large batches gamma={gamma}")
    B, D, page = 300, 64, 16
    rng = np.random.default_rng(gamma)
    lens = rng.integers(2, gamma + 2, B).tolist()
    b = Batch(1, lens, rng.integers(0, 70, B).tolist(), gamma, page, True)
    cache = make_cache("bf16", b.nb, 1, page, D)
    q = torch.randn(b.rows, 1, D, device=DEV).bfloat16()
    ap = dv.alloc_append_outputs(b.rows, 1, cache)
    rd = dv.alloc_kv_read_outputs(b.rows, cache)
    cm = torch.empty(2, dtype=torch.int32, device=DEV)
    path = np.zeros((B, gamma + 1), np.int32)
    path[:, 1] = 2 if gamma > 1 else 1
    num = np.ones(B, np.int32)
    num[np.array(lens) < 3] = 0
    n = int(num.sum())

    def run(parents, ctx, table, path, num):
        dv.dspark_kv_append(B, gamma, q, q, q, b.rows, i32(b.cu), i32(ctx), i32(table), cache, ap,
                            tree_parents=i32(parents))
        dv.dspark_kv_read(B, b.rows, i32(b.cu), i32(ctx), i32(table), cache, rd)
        dv.dspark_kv_commit(B, gamma, i32(path), i32(num), i32(ctx), i32(table), cache, cm)
        torch.cuda.synchronize()
        return ap.append_meta.tolist()[1], rd.read_meta.tolist()[1], cm.tolist()

    assert run(b.parents, b.ctx, b.table, path, num) == (0, 0, [n, 0])
    # what was appended to rows that no commit moved comes back
    dv.dspark_kv_append(B, gamma, q, q, q, b.rows, *b.args(), cache, ap)
    dv.dspark_kv_read(B, b.rows, *b.args(), cache, rd)
    torch.cuda.synchronize()
    assert torch.equal(rd.k_out[:int(b.cu[-1])], q[:int(b.cu[-1])])
    L, T, P = oracle.DATA_BAD_LENS, oracle.DATA_BAD_TREE, oracle.DATA_BAD_PAGE
    for r in (0, 15, 16, 63, 64, 255, 256, 299):
        ctx, parents, table, p, c = (x.copy() for x in (np.array(b.ctx), b.parents, b.table, path, num))
        ctx[r] = -3
        assert run(b.parents, ctx, table, path, num)[:2] == (L, L)
        assert cm.tolist() == [n - num[r], L]
        parents[r, 0] = 1
        assert run(parents, b.ctx, table, path, num) == (T, 0, [n, 0])
        table[r, (b.ctx[r] + lens[r] - 1) // page] = b.nb
        bad = num[r] and (b.ctx[r] + 2) // page == (b.ctx[r] + lens[r] - 1) // page
        got = run(b.parents, b.ctx, table, path, num)
        assert got[:2] == (P, P)
        assert got[2] == ([n - 1, P] if bad else [n, 0])
        p[r, 0], c[r] = 1, 1
        assert run(b.parents, b.ctx, b.table, p, c)[2] == [n - num[r], T]


def test_commit_of_many_layers():
    """A number of layers that no group of layers divides."""
    say("commit of 7 layers")
    for kind in ("e4m3", "f16"):
        cache = make_cache(kind, 6, 3, 16, 128, layers=7)
        for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
            if t is not None:
                t.view(torch.uint8).random_(0, 120)
        table, path = [[4, 1], [0, 3]], [[0, 2, 3, 5], [0, 1, 3, -1]]
        num, ctx = [3, 2], [14, 9]
        pools = [t for t in (cache.k, cache.v, cache.k_scale, cache.v_scale) if t is not None]
        want = [t.view(torch.uint8).clone() for t in pools]
        for r in range(2):
            for s, d in oracle.commit_moves(path[r], num[r], ctx[r], 5):
                for w in want:
                    w[:, table[r][d // 16], :, d % 16] = w[:, table[r][s // 16], :, s % 16]
        cm = torch.empty(2, dtype=torch.int32, device=DEV)
        pad = np.array([p + [-1, -1] for p in path])
        dv.dspark_kv_commit(2, 5, i32(pad), i32(num), i32(ctx), i32(table), cache, cm)
        torch.cuda.synchronize()
        assert cm.tolist() == [4, 0]
        for t, w in zip(pools, want):
            assert torch.equal(t.view(torch.uint8), w)


@pytest.mark.parametrize("B", [4, 300])
def test_read_beside_requests_out_of_order(B):
    """Malformed lengths leave the rows of the well-formed requests as they are."""
    say(f"read with lengths out of order B={B}")
    D, page = 64, 16
    rng = np.random.default_rng(B)
    lens = rng.integers(2, 5, B).tolist()
    b = Batch(3, lens, rng.integers(0, 40, B).tolist(), 4, page, False)
    cache = make_cache("bf16", b.nb, 1, page, D)
    rows = torch.randn(b.rows, 1, D, device=DEV).bfloat16()
    ap = dv.alloc_append_outputs(b.rows, 1, cache)
    dv.dspark_kv_append(B, 4, rows, rows, rows, b.rows, *b.args(), cache, ap)
    for value in (10 ** 6, -5, int(b.cu[-1]), 0):
        cu = b.cu.copy()
        at = B // 2
        cu[at] = value
        rd = dv.alloc_kv_read_outputs(b.rows, cache)
        rd.k_out.fill_(-7)
        dv.dspark_kv_read(B, b.rows, i32(cu), i32(b.ctx), i32(b.table), cache, rd)
        torch.cuda.synchronize()
        assert rd.read_meta.tolist() == [int(b.cu[-1]), oracle.DATA_BAD_LENS] or value in (
            0, int(b.cu[-1]))
        for r in range(B):
            if r in (at - 1, at):
                continue  # the two that the word bounds
            c = slice(int(b.cu[r]), int(b.cu[r + 1]))
            if value in (0, int(b.cu[-1])) and not torch.equal(rd.k_out[c], rows[c]):
                # such a word makes another request long, which may claim the row
                assert (r < at) == (value == 0)
                continue
            assert torch.equal(rd.k_out[c], rows[c]), (value, r)
