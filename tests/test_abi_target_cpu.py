"""Argument checks of the target-pass entry points, without a GPU: every call
here is refused on the host, before any launch."""

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
    a = dict(k=0x1000, v=0x2000, k_scale=None, v_scale=None, block_stride=2 * 16 * 64,
             scale_block_stride=0, layer_stride=0, scale_layer_stride=0, num_layers=1,
             num_blocks=8, num_kv_heads=2, block_size=16, head_dim=64, dtype=_lib.BF16)
    a.update(kw)
    return _lib.KvCacheDesc(*a.values())


def _e8(**kw):
    return _cache(**{**dict(k_scale=0x3000, v_scale=0x4000, scale_block_stride=32,
                            dtype=_lib.E4M3), **kw})


def _ref(c):
    return ctypes.cast(ctypes.pointer(c), ctypes.c_void_p) if c is not None else None


def _append(cache=None, **kw):
    cache = _cache() if cache is None else cache
    a = dict(B=2, gamma=4, hq=4, dt=_lib.BF16, q=FAKE, qld=256, k=FAKE, kld=128, v=FAKE, vld=128,
             max_rows=10, cu=FAKE, prefix=FAKE, parents=NULL, table=FAKE, width=4, qw=NULL,
             kw=NULL, eps=1e-6, rope=NULL, rope_rows=0, rope_dim=0, inter=0, out=FAKE, old=256,
             cache=_ref(cache), meta=NULL, stream=NULL)  # meta NULL: refused at the latest there
    a.update(kw)
    return _lib.lib().dspark_kv_append(*a.values())


def _attn(cache=None, **kw):
    cache = _cache() if cache is None else cache
    a = dict(B=2, gamma=4, hq=4, dt=_lib.BF16, q=FAKE, qld=256, max_rows=10, cu=FAKE, prefix=FAKE,
             parents=NULL, table=FAKE, width=4, cache=_ref(cache), scale=0.1, out=FAKE, old=256,
             lse=NULL, meta=FAKE, ws=NULL, wsb=1 << 30, stream=NULL)  # refused for ws at the latest
    a.update(kw)
    return _lib.lib().dspark_tree_attention(*a.values())


def _read(cache=None, **kw):
    cache = _cache() if cache is None else cache
    a = dict(B=2, max_rows=10, cu=FAKE, starts=FAKE, table=FAKE, width=4, cache=_ref(cache), k=FAKE,
             v=FAKE, ld=128, meta=NULL, stream=NULL)
    a.update(kw)
    return _lib.lib().dspark_kv_read(*a.values())


def _commit(cache=None, **kw):
    cache = _cache() if cache is None else cache
    a = dict(B=2, gamma=4, path=FAKE, num=FAKE, prefix=FAKE, table=FAKE, width=4,
             cache=_ref(cache), meta=NULL, stream=NULL)
    a.update(kw)
    return _lib.lib().dspark_kv_commit(*a.values())


BAD_CACHES = [
    (_cache(dtype=_lib.F32), UNS), (_cache(dtype=9), UNS), (_cache(head_dim=96), UNS),
    (_cache(head_dim=0), UNS), (_cache(block_size=8), UNS), (_cache(block_size=48), UNS),
    (_cache(block_size=512), UNS), (_cache(num_kv_heads=0), INV), (_cache(num_kv_heads=257), INV),
    (_cache(num_blocks=0), INV), (_cache(k=None), INV), (_cache(v=0x1008), INV),
    (_cache(block_stride=2047), INV), (_cache(block_stride=2052), INV),
    (_e8(k_scale=None), INV), (_e8(v_scale=None), INV), (_e8(scale_block_stride=31), INV),
    (_e8(block_stride=2056), INV), (_e8(k_scale=0x3004), INV), (_e8(scale_block_stride=40), INV),
]


@pytest.mark.parametrize("call", [_append, _attn, _read, _commit])
@pytest.mark.parametrize("i", range(len(BAD_CACHES)))
def test_cache_refusals(call, i):
    cache, code = BAD_CACHES[i]
    assert call(cache) == code, _lib.last_error()
    assert "dspark_" in _lib.last_error()


SHARED = [  # (calls that take it, changed arguments, status)
    ("arqc", dict(B=-1), INV), ("arqc", dict(B=8193), UNS), ("arqc", dict(table=NULL), INV),
    ("arqc", dict(width=0), INV), ("aqc", dict(prefix=NULL), INV), ("aqc", dict(gamma=0), INV),
    ("aqc", dict(gamma=65), INV), ("arq", dict(max_rows=-1), INV), ("arq", dict(cu=NULL), INV),
    ("aq", dict(dt=_lib.F32), UNS), ("aq", dict(dt=_lib.E4M3), UNS), ("aq", dict(dt=_lib.F16), UNS),
    ("aq", dict(hq=0), INV), ("aq", dict(hq=3), INV), ("aq", dict(hq=258), INV),
    ("aq", dict(hq=130), INV), ("aq", dict(q=NULL), INV), ("aq", dict(q=ODD), INV),
    ("aq", dict(qld=255), INV), ("aq", dict(qld=260), INV), ("aq", dict(old=248), INV),
]
CALLS = {"a": _append, "r": _read, "q": _attn, "c": _commit}


@pytest.mark.parametrize("calls,kw,code", SHARED)
def test_shared_refusals(calls, kw, code):
    for c in calls:
        assert CALLS[c](**kw) == code, (c, _lib.last_error())


def test_no_cache():
    lib = _lib.lib()
    assert lib.dspark_kv_commit(2, 4, FAKE, FAKE, FAKE, FAKE, 4, NULL, FAKE, NULL) == INV
    assert lib.dspark_kv_read(2, 4, FAKE, FAKE, FAKE, 4, NULL, FAKE, FAKE, 128, FAKE, NULL) == INV
    assert "cache is NULL" in _lib.last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(), INV),  # append_meta NULL
    (dict(kld=120), INV), (dict(v=NULL), INV), (dict(vld=132), INV), (dict(k=ODD), INV),
    (dict(out=ODD), INV), (dict(qld=264), INV),  # q_out is q with another stride
    (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(eps=float("inf")), INV),
    (dict(qw=ODD), INV), (dict(kw=ODD), INV),
    (dict(rope=FAKE, rope_rows=0, rope_dim=32), INV), (dict(rope=ODD, rope_rows=9, rope_dim=32), INV),
    (dict(rope=FAKE, rope_rows=9, rope_dim=8), INV), (dict(rope=FAKE, rope_rows=9, rope_dim=80), INV),
    (dict(rope=FAKE, rope_rows=9, rope_dim=40), INV),
])
def test_append_refusals(kw, code):
    # (the meta pointer is given, so that each of these is refused for its own fault)
    if kw:
        kw = dict(meta=FAKE, **kw)
    assert _append(**kw) == code, _lib.last_error()


def test_attention_refusals():
    assert _attn() == WSP
    assert _attn(ws=ctypes.c_void_p(0x1010)) == WSP  # not 256-byte aligned
    assert _attn(ws=FAKE, wsb=16) == WSP
    assert _attn(scale=float("inf")) == INV and _attn(scale=float("nan")) == INV
    assert _attn(out=NULL) == INV and _attn(meta=NULL) == INV
    assert _attn(_e8(), dt=_lib.F16) == UNS  # an 8-bit cache goes with bfloat16
    size = dv.dspark_tree_attention_workspace_size
    assert size(2, 4, 4, 2, 64) >= 256
    for bad in ((-1, 4, 4, 2, 64), (2, 0, 4, 2, 64), (2, 65, 4, 2, 64), (2, 4, 3, 2, 64),
                (2, 4, 4, 0, 64), (2, 4, 4, 2, 80), (8193, 4, 4, 2, 64), (2, 4, 130, 2, 64)):
        assert size(*bad) == 0


def test_read_and_commit_refusals():
    assert _read() == INV and "read_meta" in _lib.last_error()
    assert _read(meta=FAKE, k=ODD) == INV and _read(meta=FAKE, v=NULL) == INV
    assert _read(meta=FAKE, ld=120) == INV and _read(meta=FAKE, starts=NULL) == INV
    assert _commit() == INV and "commit_meta" in _lib.last_error()
    assert _commit(meta=FAKE, path=NULL) == INV and _commit(meta=FAKE, num=NULL) == INV
    assert _commit(_cache(num_layers=0), meta=FAKE) == INV
    assert _commit(_cache(num_layers=1025), meta=FAKE) == INV
    assert _commit(_cache(num_layers=2, layer_stride=1024), meta=FAKE) == INV  # layers overlap
    assert _commit(_e8(num_layers=2, layer_stride=2048, scale_layer_stride=40), meta=FAKE) == INV


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), INV), (dict(gamma=65), INV), (dict(V=0), INV), (dict(dt=_lib.F16), UNS),
    (dict(path=NULL), INV), (dict(cu=NULL), INV), (dict(drafts=NULL), INV), (dict(ws=NULL), WSP),
    (dict(newseq=FAKE, prefix=NULL), INV), (dict(ld=1000), INV),
])
def test_tree_accept_refusals(kw, code):
    a = dict(B=2, gamma=4, V=1024, dt=_lib.BF16, logits=FAKE, ld=1024, max_rows=10, cu=FAKE,
             drafts=FAKE, parents=NULL, prefix=NULL, am=FAKE, nc=FAKE, bonus=FAKE, commit=FAKE,
             out=FAKE, path=FAKE, newseq=NULL, meta=FAKE, ws=ctypes.c_void_p(0x10000), wsb=1 << 20,
             stream=NULL)
    a.update(kw)
    assert _lib.lib().dspark_tree_accept(*a.values()) == code, _lib.last_error()
    assert "dspark_tree_accept" in _lib.last_error()


def test_binding_refuses_host_tensors_and_wrong_kinds():
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        dv.KvCache(k, k.clone())
    with pytest.raises(TypeError):
        dv.KvCache(k.float(), k.float())
    with pytest.raises(TypeError):
        dv.KvCache(None, k)
    with pytest.raises(ValueError):
        dv.KvCache(k, k[:2])
    with pytest.raises(ValueError, match="dtype code"):
        dv.alloc_kv_cache(4, 2, 16, 64, dv.F32, "cpu")
