"""Which strides of queries the latent cache's entry points take, without a GPU: every
call here is refused on the host, at the latest for its workspace or status words."""

import pytest

from dspark_verify_scheduling_amd import _lib
from test_abi_latent_cpu import INV, WSP, _append, _attn


@pytest.mark.parametrize("kw,code", [
    # a head's rows together, max_rows = 10 of them
    (dict(qlhld=10 * 512, qlld=512), WSP), (dict(qrhld=10 * 64, qrld=64), WSP),
    (dict(qlhld=1 << 40, qlld=512), WSP), (dict(qlhld=8192, qlld=520), WSP),
    (dict(qlhld=10 * 512, qlld=512, qrhld=10 * 64, qrld=64), WSP),
    (dict(qlhld=512, qlld=512, hq=1), WSP), (dict(qlhld=512, qlld=512, max_rows=1), WSP),
    # rows of two heads that overlap
    (dict(qlhld=9 * 512, qlld=512), INV), (dict(qlhld=5200, qlld=528), INV),
    (dict(qlhld=512, qlld=512), INV), (dict(qlhld=1024, qlld=512), INV),
    (dict(qlhld=512, qlld=512, max_rows=2), INV), (dict(qlhld=512, qlld=1 << 40, max_rows=2 ** 31 - 1), WSP),
    (dict(qlhld=(1 << 40) + 8, qlld=512), INV), (dict(qlhld=10 * 512 + 4, qlld=512), INV),
    (dict(qlhld=10 * 512, qlld=508), INV),
])
def test_attention_takes_rows_and_heads_in_both_orders(kw, code):
    assert _attn(**kw) == code, _lib.last_error()


@pytest.mark.parametrize("kw,ok", [
    (dict(qhld=640, qld=64), True), (dict(ohld=640, old=64), True),
    (dict(qhld=640, qld=64, ohld=1280, old=128, out=0x4000), True),
    (dict(qhld=576, qld=64), False), (dict(ohld=576, old=64), False),
])
def test_append_takes_rows_and_heads_in_both_orders(kw, ok):
    kw = {"out": 0x4000, **kw}
    assert _append(**kw) == INV  # its status words are NULL, which is seen last
    assert ("append_meta" in _lib.last_error()) == ok, _lib.last_error()
