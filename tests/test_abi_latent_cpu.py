"""Argument checks of the latent cache's entry points and of the append with
positions on several axes, without a GPU: every call here is refused on the
host, before any launch."""

import ctypes

import pytest
import torch

import dspark_verify_scheduling_amd as dv
from dspark_verify_scheduling_amd import _lib

NULL = None
FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: every call below fails validation
ODD = ctypes.c_void_p(0x1008)
INV, UNS, WSP = _lib.E_INVALID, _lib.E_UNSUPPORTED, _lib.E_WORKSPACE


def _cache(**kw):
    a = dict(latent=0x1000, rope=0x2000, scale=None, block_stride=16 * 512,
             rope_block_stride=16 * 64, scale_block_stride=0, layer_stride=0, rope_layer_stride=0,
             scale_layer_stride=0, num_layers=1, num_blocks=8, block_size=16, latent_dim=512,
             dtype=_lib.BF16)
    a.update(kw)
    return _lib.LatentCacheDesc(*a.values())


def _e8(**kw):
    return _cache(**{**dict(scale=0x3000, scale_block_stride=64, dtype=_lib.E4M3), **kw})


def _ref(c):
    return ctypes.cast(ctypes.pointer(c), ctypes.c_void_p)


def _call(name, a, cache, kw):
    a["cache"] = _ref(_cache() if cache is None else cache)
    a.update(kw)
    return getattr(_lib.lib(), name)(*a.values())


def _append(cache=None, **kw):  # meta NULL: refused at the latest there
    return _call("dspark_latent_append", dict(
        B=2, gamma=4, hq=4, dt=_lib.BF16, kv=FAKE, kvld=576, q=FAKE, qld=256, qhld=64, max_rows=10,
        cu=FAKE, prefix=FAKE, parents=NULL, table=FAKE, width=4, w=NULL, eps=1e-6, rope=NULL,
        rope_rows=0, inter=0, out=FAKE, old=256, ohld=64, cache=NULL, meta=NULL, stream=NULL),
        cache, kw)


def _read(cache=None, **kw):
    return _call("dspark_latent_read", dict(
        B=2, max_rows=10, cu=FAKE, starts=FAKE, table=FAKE, width=4, cache=NULL, lat=FAKE, ld=512,
        rope=FAKE, rld=64, meta=NULL, stream=NULL), cache, kw)


def _commit(cache=None, **kw):
    return _call("dspark_latent_commit", dict(
        B=2, gamma=4, path=FAKE, num=FAKE, prefix=FAKE, table=FAKE, width=4, cache=NULL, meta=NULL,
        stream=NULL), cache, kw)


def _attn(cache=None, **kw):  # refused for its workspace at the latest
    return _call("dspark_latent_attention", dict(
        B=2, gamma=4, hq=4, dt=_lib.BF16, ql=FAKE, qlld=2048, qlhld=512, qr=FAKE, qrld=256,
        qrhld=64, max_rows=10, cu=FAKE, prefix=FAKE, parents=NULL, table=FAKE, width=4, cache=NULL,
        scale=0.1, out=FAKE, old=2048, lse=NULL, meta=FAKE, ws=NULL, wsb=1 << 40, stream=NULL),
        cache, kw)


def _prefill(cache=None, **kw):
    return _call("dspark_latent_prefill", dict(
        B=2, hq=4, nope=128, dt=_lib.BF16, q=FAKE, qld=768, wk=FAKE, wv=FAKE, wld=128 * 512,
        max_rows=10, max_keys=100, cu=FAKE, prefix=FAKE, table=FAKE, width=4, cache=NULL, scale=0.1,
        out=FAKE, old=512, lse=NULL, meta=FAKE, ws=NULL, wsb=1 << 40, stream=NULL), cache, kw)


BAD_CACHES = [
    (_cache(dtype=_lib.F32), UNS), (_cache(dtype=9), UNS), (_cache(latent_dim=128), UNS),
    (_cache(latent_dim=576), UNS), (_cache(block_size=8), UNS), (_cache(block_size=512), UNS),
    (_cache(num_blocks=0), INV), (_cache(latent=None), INV), (_cache(latent=0x1008), INV),
    (_cache(rope=None), INV), (_cache(rope=0x2008), INV), (_cache(block_stride=16 * 512 - 8), INV),
    (_cache(block_stride=16 * 512 + 4), INV), (_cache(rope_block_stride=16 * 64 - 8), INV),
    (_cache(rope_block_stride=16 * 64 + 4), INV), (_e8(scale=None), INV), (_e8(scale=0x3004), INV),
    (_e8(scale_block_stride=48), INV), (_e8(scale_block_stride=72), INV),
    (_e8(block_stride=16 * 512 + 8), INV),
]


@pytest.mark.parametrize("call", [_append, _read, _commit, _attn, _prefill])
@pytest.mark.parametrize("i", range(len(BAD_CACHES)))
def test_cache_refusals(call, i):
    cache, code = BAD_CACHES[i]
    assert call(cache) == code, _lib.last_error()
    assert "dspark_latent" in _lib.last_error()


CALLS = {"a": _append, "r": _read, "c": _commit, "q": _attn, "p": _prefill}
SHARED = [  # (calls that take it, changed arguments, status)
    ("arcqp", dict(B=-1), INV), ("arcqp", dict(B=8193), UNS), ("arcqp", dict(table=NULL), INV),
    ("arcqp", dict(width=0), INV), ("acqp", dict(prefix=NULL), INV), ("r", dict(starts=NULL), INV),
    ("cq", dict(gamma=0), INV), ("acq", dict(gamma=65), INV), ("a", dict(gamma=-1), INV),
    ("arqp", dict(max_rows=-1), INV), ("arqp", dict(cu=NULL), INV),
    ("aqp", dict(dt=_lib.F32), UNS), ("aqp", dict(dt=_lib.E4M3), UNS), ("aqp", dict(dt=_lib.F16), UNS),
    ("qp", dict(hq=0), INV), ("a", dict(hq=-1), INV), ("aqp", dict(hq=129), INV),
    ("qp", dict(out=NULL), INV), ("aqp", dict(out=ODD), INV), ("aqp", dict(old=248), INV),
]


@pytest.mark.parametrize("calls,kw,code", SHARED)
def test_shared_refusals(calls, kw, code):
    for c in calls:
        assert CALLS[c](**kw) == code, (c, _lib.last_error())


@pytest.mark.parametrize("kw,code", [
    (dict(), INV), (dict(kv=NULL), INV), (dict(kv=ODD), INV), (dict(kvld=568), INV),
    (dict(kvld=580), INV), (dict(q=NULL), INV), (dict(q=ODD), INV), (dict(qhld=56), INV),
    (dict(qhld=68), INV), (dict(qld=248), INV), (dict(qld=260), INV), (dict(ohld=32), INV),
    (dict(out=NULL), INV), (dict(out=FAKE, old=264), INV), (dict(meta=FAKE, eps=-1.0), INV),
    (dict(meta=FAKE, eps=float("nan")), INV), (dict(meta=FAKE, w=ODD), INV),
    (dict(meta=FAKE, rope=ODD, rope_rows=5), INV), (dict(meta=FAKE, rope=FAKE, rope_rows=0), INV),
    (dict(meta=FAKE, gamma=0, parents=FAKE), INV),
])
def test_append_refusals(kw, code):
    assert _append(**kw) == code, _lib.last_error()


@pytest.mark.parametrize("kw", [
    dict(), dict(lat=NULL), dict(lat=ODD), dict(ld=504), dict(ld=516), dict(rope=NULL),
    dict(rope=ODD), dict(rld=56), dict(rld=68),
])
def test_read_refusals(kw):
    assert _read(**kw) == INV, _lib.last_error()


@pytest.mark.parametrize("cache,kw", [
    (_cache(num_layers=0), {}), (_cache(num_layers=1025), {}),
    (_cache(num_layers=2, layer_stride=8, rope_layer_stride=16 * 64), {}),
    (_cache(num_layers=2, layer_stride=16 * 512, rope_layer_stride=16 * 64 + 4), {}),
    (_e8(num_layers=2, layer_stride=16 * 512, rope_layer_stride=16 * 64, scale_layer_stride=8), {}),
    (None, dict(path=NULL)), (None, dict(num=NULL)), (None, {}),
])
def test_commit_refusals(cache, kw):
    assert _commit(cache, **kw) == INV, _lib.last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(), WSP), (dict(ws=ctypes.c_void_p(0x1010)), WSP), (dict(ws=FAKE, wsb=1024), WSP),
    (dict(meta=NULL), INV), (dict(scale=float("inf")), INV), (dict(scale=float("nan")), INV),
    (dict(ql=NULL), INV), (dict(ql=ODD), INV), (dict(qlld=2040), INV), (dict(qlhld=504), INV),
    (dict(qlhld=516), INV), (dict(qr=NULL), INV), (dict(qr=ODD), INV), (dict(qrhld=60), INV),
    (dict(qrld=200), INV), (dict(old=2040), INV),
])
def test_attention_refusals(kw, code):
    assert _attn(**kw) == code, _lib.last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(), WSP), (dict(ws=ctypes.c_void_p(0x1010)), WSP), (dict(ws=FAKE, wsb=1024), WSP),
    (dict(meta=NULL), INV), (dict(scale=float("inf")), INV), (dict(nope=96), UNS),
    (dict(max_keys=-1), INV), (dict(max_keys=_lib.LATENT_MAX_KEYS + 1), UNS), (dict(q=NULL), INV),
    (dict(qld=760), INV), (dict(wk=NULL), INV), (dict(wv=ODD), INV), (dict(wld=512), INV),
    (dict(wld=128 * 512 + 4), INV), (dict(old=504), INV),
])
def test_prefill_refusals(kw, code):
    assert _prefill(**kw) == code, _lib.last_error()


def test_no_cache():
    for c in CALLS.values():
        assert c(cache=None) != _lib.OK
    assert _lib.lib().dspark_latent_commit(2, 4, FAKE, FAKE, FAKE, FAKE, 4, NULL, FAKE, NULL) == INV


def test_workspace_sizes():
    f, g = dv.dspark_latent_attention_workspace_size, dv.dspark_latent_prefill_workspace_size
    assert f(4, 4, 16, 512) > 0 and f(4, 4, 128, 256) > 0
    for bad in [(-1, 4, 16, 512), (8193, 4, 16, 512), (4, 0, 16, 512), (4, 65, 16, 512),
                (4, 4, 0, 512), (4, 4, 129, 512), (4, 4, 16, 384)]:
        assert f(*bad) == 0
    one = g(1, 64, 1000, 8, 128, 512)
    # dense rows, keys and values of every head
    assert one >= 1000 * (512 * 2 + 64 * 2 + 8 * 256 * 2)
    assert g(0, 0, 0, 8, 128, 512) >= 0 and g(3, 64, 1000, 8, 128, 512) >= one
    for bad in [(-1, 4, 9, 8, 128, 512), (1, -1, 9, 8, 128, 512), (1, 4, -1, 8, 128, 512),
                (1, 4, 9, 0, 128, 512), (1, 4, 9, 8, 96, 512), (1, 4, 9, 8, 128, 300),
                (1, 4, _lib.LATENT_MAX_KEYS + 1, 8, 128, 512)]:
        assert g(*bad) == 0


# ------------------------------------------------------------------ positions on several axes

def _axes(**kw):
    kv = _lib.KvCacheDesc(0x1000, 0x2000, None, None, 2 * 16 * 64, 0, 0, 0, 1, 8, 2, 16, 64, _lib.BF16)
    pairs = kw.pop("pairs", [0] * 32)
    host = (ctypes.c_int32 * len(pairs))(*pairs)
    a = dict(B=2, hq=4, dt=_lib.BF16, q=FAKE, qld=256, k=FAKE, kld=128, v=FAKE, vld=128, max_rows=10,
             cu=FAKE, prefix=FAKE, pos=FAKE, pld=10, axes=3, pair=ctypes.cast(host, ctypes.c_void_p),
             table=FAKE, width=4, qw=NULL, kw=NULL, eps=1e-6, rope=FAKE, rope_rows=100, rope_dim=64,
             inter=0, out=FAKE, old=256, cache=_ref(kv), meta=FAKE, stream=NULL)
    a.update(kw)
    return _lib.lib().dspark_kv_append_axes(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(axes=0), INV), (dict(axes=5), INV), (dict(pos=NULL), INV), (dict(pld=9), INV),
    (dict(pair=NULL), INV), (dict(pairs=[0] * 31 + [3]), INV), (dict(pairs=[-1] + [0] * 31), INV),
    (dict(rope=NULL), INV), (dict(rope_dim=24), INV), (dict(rope_dim=80), INV),
    (dict(rope_rows=0), INV), (dict(meta=NULL), INV), (dict(B=-1), INV), (dict(B=8193), UNS),
    (dict(cu=NULL), INV), (dict(table=NULL), INV), (dict(hq=3), INV), (dict(dt=_lib.F16), UNS),
    (dict(q=ODD), INV), (dict(vld=120), INV), (dict(out=FAKE, old=264), INV),
    (dict(cache=NULL), INV), (dict(eps=-1.0), INV), (dict(kw=ODD), INV), (dict(max_rows=-1), INV),
])
def test_axes_refusals(kw, code):
    assert _axes(**kw) == code, _lib.last_error()


# ------------------------------------------------------------------ the binding's own checks

def test_latent_cache_checks():
    lat, rope = torch.zeros(4, 16, 512), torch.zeros(4, 16, 64)
    with pytest.raises(TypeError):
        dv.LatentCache(lat, rope)  # float32
    with pytest.raises(TypeError):
        dv.LatentCache(None, rope)
    with pytest.raises(ValueError):
        dv.LatentCache(lat.bfloat16(), rope.bfloat16())  # not on a GPU
    with pytest.raises(ValueError):
        dv.LatentCache(lat[0].bfloat16(), rope[0].bfloat16())
    with pytest.raises(ValueError):
        dv.alloc_latent_cache(4, 16, 512, dv.F32, "cpu")
