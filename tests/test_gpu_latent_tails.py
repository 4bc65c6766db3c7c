"""GPU tests of what small weights add in float16 attention over latents, and of the
largest scale.

Float16 weights round to the nearest of 2^-24 of a power of two that the kernels put them
on: as include/dspark.h has it they count down to 2^-34 (absorbed) or 2^-36 (expanded) of
the row's largest, which is half their step. So a weight errs by 2^-11 of itself or by that
part of the largest, and an output by

    u |out| + 2^-25 + (u + 2 t + (n + 32) w) sum w_k |v_k| + 2^-34 (2^-36) max w sum |v_k|

with the weights w_k in the sums divided by their sum, u = 2^-11, w = 2^-24, 2^-25 half the
output's own smallest step, and t = 80 w max |s| the scores' error, whose one term has 64
zeros beside it and is turned into log2."""

import numpy as np
import pytest
import torch

import dspark_verify_scheduling_amd as dv
from _gpu import DEV, say
from test_gpu_latent import R, latent_setup, lget, lput, make_latent, typed
from test_gpu_target import TYPES, Batch, W, f64, within

pytestmark = pytest.mark.gpu
U, LN2 = 2.0 ** -11, float(np.float32(np.log(2)))


@pytest.fixture(scope="module", autouse=True)
def _need_gpu(hip):
    return hip


def tails(T, shape, rng):
    """Scores in log2 of T keys, and which keys hold values: some of weight 1, or rising to
    it by 32 a step, without; all others 2^-26 to 2^-30 of it, with."""
    s = rng.integers(-30 * 64, -26 * 64 + 1, T) / 64
    large = np.arange(T) % 61 == 40 if shape == "often" else np.zeros(T, bool)
    if shape == "first":
        large[0] = True
    elif shape == "late":
        large[T * 3 // 4] = True
    elif shape == "rising":
        at = np.linspace(5, T - 9, 25).astype(int)
        large[at] = True
        s[at] = -5.0 * np.arange(24, -1, -1)
    if shape != "rising":
        s[large] = 0.0
    return s, ~large


def setup(T, L, shape, page, seed):
    """A request of two rows over T keys whose scores are `tails`, through the rotated
    part alone; its latents are large, so that what the small weights add is seen."""
    rng = np.random.default_rng(seed)
    b = Batch(seed, [2], [T - 2], 3, page, False)
    s, small = tails(T, shape, rng)
    lat = rng.integers(10000, 60001, (T, L)) // 32 * 32.0 * small[:, None]  # float16 numbers
    rope = np.zeros((T, R))
    rope[:, 3] = s
    cache = make_latent("f16", b.nb, page, L)
    lput(cache, b.slots(0, 0, T), lat, rope)
    got, turned = lget(cache, b.slots(0, 0, T))
    assert np.array_equal(got, lat) and np.array_equal(turned, rope)
    return b, cache, lat, s


def expect(got, lse, v, s, factor, n, least):
    """One row of `got` against the formula over its n keys' values v and scores."""
    x = s[:n] * factor * LN2
    w = np.exp(x - x.max())
    total = w.sum()
    w = w / total
    ref, mean_abs = w @ v[:n], w @ np.abs(v[:n])
    t = 80 * W * np.abs(x).max()
    bound = (U * np.abs(ref) + 2.0 ** -25 + (U + 2 * t + (n + 32) * W) * mean_abs
             + least * w.max() * np.abs(v[:n]).sum(0))
    # the small weights are what the row consists of, and far above the bound
    if factor == 1:
        assert np.all(bound < 0.1 * np.abs(ref))
    within(got, ref, bound, ("out", n, factor))
    want = x.max() + np.log(total)
    within(lse, want, t + (n + 32) * W + 4 * W * abs(want) + 1e-6, ("lse", n, factor))


SHAPES = ["often", "first", "late", "rising"]


@pytest.mark.parametrize("L,H", [(512, 2), (256, 40)])
@pytest.mark.parametrize("T", [700, 6000])
@pytest.mark.parametrize("shape", SHAPES)
def test_small_weights_count_in_the_absorbed_form(shape, T, L, H):
    say(f"latent attention, float16 tails {shape} T={T} L={L}")
    b, cache, lat, s = setup(T, L, shape, 64, 3)
    ql = torch.zeros(b.rows, H, L, dtype=torch.float16, device=DEV)
    qr = torch.zeros(b.rows, H, R, dtype=torch.float16, device=DEV)
    qr[:, 0::2, 3], qr[:, 1::2, 3] = 1.0, 0.5
    o = dv.alloc_latent_attention_outputs(1, 3, b.rows, H, cache, lse=True)
    dv.dspark_latent_attention(1, 3, ql, qr, b.rows, *b.args(), cache, LN2, o)
    torch.cuda.synchronize()
    got, lse = f64(o.out), f64(o.lse)
    for j in range(2):
        for h in {0, 1, H - 1}:
            expect(got[j, h], lse[j, h], lat, s, 1.0 if h % 2 == 0 else 0.5, T - 1 + j, 2.0 ** -34)


@pytest.mark.parametrize("L,H", [(512, 2), (256, 9)])
@pytest.mark.parametrize("T", [700, 6000])
@pytest.mark.parametrize("shape", SHAPES)
def test_small_weights_count_in_the_expanded_form(shape, T, L, H):
    say(f"latent prefill, float16 tails {shape} T={T} L={L}")
    n = 64
    b, cache, lat, s = setup(T, L, shape, 64, 4)
    q = torch.zeros(b.rows, H, n + R, dtype=torch.float16, device=DEV)
    q[:, 0::2, n + 3], q[:, 1::2, n + 3] = 1.0, 0.5
    w = torch.zeros(H, 2 * n, L, dtype=torch.float16, device=DEV)
    for c in range(n):  # values are the latents' last elements
        w[:, n + c, L - n + c] = 1.0
    o = dv.alloc_latent_prefill_outputs(1, b.rows, T, H, n, cache, lse=True)
    dv.dspark_latent_prefill(1, q, w[:, :n], w[:, n:], b.rows, T, *b.args(), cache, LN2, o)
    torch.cuda.synchronize()
    got, lse = f64(o.out), f64(o.lse)
    for j in range(2):
        for h in {0, 1, H - 1}:
            expect(got[j, h], lse[j, h], lat[:, L - n:], s, 1.0 if h % 2 == 0 else 0.5, T - 1 + j,
                   2.0 ** -36)


@pytest.mark.parametrize("kind,L", [("bf16", 512), ("f16", 256), ("e4m3", 512)])
@pytest.mark.parametrize("scale", [3.4e38, -3.4e38])
def test_the_largest_scale_ends_and_keeps_to_its_rows(kind, L, scale):
    """Scores past float32 have no meaning, but the status has, and rows past the last are
    left as they were."""
    say(f"latent attention and prefill, scale {scale} {kind}")
    H, n = 4, 64
    b = Batch(9, [3, 2], [70, 5], 3, 16, False)
    cache, ql, qr = latent_setup(b, kind, H, L)
    q = typed(b.rng, (b.rows, H, n + R), TYPES[kind][1]).to(DEV)
    w = typed(b.rng, (H, 2 * n, L), TYPES[kind][1], L ** -0.5).to(DEV)
    a = dv.alloc_latent_attention_outputs(2, 3, b.rows, H, cache, lse=True)
    p = dv.alloc_latent_prefill_outputs(2, b.rows, 80, H, n, cache, lse=True)
    for o in (a, p):
        o.out.fill_(-7)
        o.lse.fill_(-7)
    dv.dspark_latent_attention(2, 3, ql, qr, b.rows, *b.args(), cache, scale, a)
    dv.dspark_latent_prefill(2, q, w[:, :n], w[:, n:], b.rows, 80, *b.args(), cache, scale, p)
    torch.cuda.synchronize()
    for o in (a, p):
        assert o.attention_meta.tolist() == [5, 0]
        assert bool((o.out[5:] == -7).all()) and bool((o.lse[5:] == -7).all())
        assert bool((o.out[:5] != -7).any(-1).all()) and bool((o.lse[:5] != -7).all())
