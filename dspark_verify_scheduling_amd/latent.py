"""The target pass over a cache of one latent vector a token: append, read,
commit, and attention in the absorbed and in the expanded form.

Conventions as in ``target``. ``LatentCache`` describes a cache once; calls of a
layer take ``cache.layer(i)``.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import _lib
from . import _stream
from ._lib import E4M3, LATENT_GROUP, LATENT_ROPE
from .target import _CODE, _I32, _TORCH, AttentionOutputs, _device, _on, _strides, _table


def _heads(t: torch.Tensor, name: str, dtype, rows: int, heads: int, dim: int, dev: int):
    """Pointer, row stride and head stride of [rows, heads, dim] with dense elements,
    whose rows or whose heads may be the outer ones."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the current device cuda:{dev}, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[0] < rows or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{name} must be [>= {rows}, {heads}, {dim}], got {tuple(shape)}")
    s = t.stride()
    if s[2] != 1:
        raise ValueError(f"the elements of a head of {name} must be dense")
    # a single head or row has no stride of its own
    head = s[1] if heads > 1 else dim
    return t.data_ptr(), (s[0] if shape[0] > 1 else (heads - 1) * head + dim), head


def _lines(t: torch.Tensor, name: str, dtype, rows: int, dim: int, dev: int):
    """Pointer and row stride of [rows, dim] with dense rows."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the current device cuda:{dev}, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2 or t.shape[0] < rows or t.shape[1] != dim:
        raise ValueError(f"{name} must be [>= {rows}, {dim}], got {tuple(t.shape)}")
    if t.stride(1) != 1:
        raise ValueError(f"the rows of {name} must be dense")
    return t.data_ptr(), (t.stride(0) if t.shape[0] > 1 else dim)


def _dense_out(t: torch.Tensor, name: str, dtype, rows: int, heads: int, dim: int, dev: int):
    ptr, ld, head = _heads(t, name, dtype, rows, heads, dim, dev)
    if head != dim:
        raise ValueError(f"the heads of {name} must be dense")
    return ptr, ld


# ------------------------------------------------------------------ cache

class LatentCache:
    """A paged cache: ``latent`` [num_blocks, block_size, latent_dim] in
    bfloat16, float16 or float8_e4m3fn and ``rope`` [num_blocks, block_size, 64]
    in 16 bits, or both with a leading layer dimension. With float8_e4m3fn,
    ``scale`` (uint8, [..., latent_dim / 128]) holds the exponent bytes of every
    128 elements: value = code * 2^(byte - 127), and ``rope`` is bfloat16. The
    strides of pages and layers are free; the last two dimensions are dense."""

    def __init__(self, latent: torch.Tensor, rope: torch.Tensor,
                 scale: Optional[torch.Tensor] = None):
        if not isinstance(latent, torch.Tensor) or not isinstance(rope, torch.Tensor):
            raise TypeError("latent and rope must be torch.Tensors")
        if latent.dtype not in _CODE:
            raise TypeError(f"a cache is bfloat16, float16 or float8_e4m3fn, got {latent.dtype}")
        if latent.dim() not in (3, 4):
            raise ValueError("latent must be [(layers,) num_blocks, block_size, latent_dim]")
        if not latent.is_cuda:
            raise ValueError(f"the cache must be on a CUDA device, got {latent.device}")
        e8 = latent.dtype == torch.float8_e4m3fn
        #: type of the rows that go in and come out
        self.row_dtype = torch.bfloat16 if e8 else latent.dtype
        if rope.dtype != self.row_dtype:
            raise TypeError(f"rope must be {self.row_dtype}, got {rope.dtype}")
        if e8 and (not isinstance(scale, torch.Tensor) or scale.dtype != torch.uint8):
            raise TypeError("scale must be a uint8 tensor")
        if not e8 and scale is not None:
            raise ValueError("only a float8_e4m3fn cache has a scale")
        lead, dim = latent.shape[:-1], latent.shape[-1]
        parts = [("latent", latent, dim), ("rope", rope, LATENT_ROPE)]
        if e8:
            parts.append(("scale", scale, dim // LATENT_GROUP))
        strides = []
        for name, t, n in parts:
            if t.shape != lead + (n,) or t.device != latent.device:
                raise ValueError(f"{name} must be {tuple(lead + (n,))} on {latent.device}")
            s = _strides(t)
            if s[-2:] != (n, 1):
                raise ValueError(f"{name} must be dense in its last two dimensions")
            strides.append(s)
        if not e8:
            strides.append((0,) * latent.dim())
        self.latent, self.rope, self.scale = latent, rope, scale
        self.dtype = _CODE[latent.dtype]
        self.num_blocks, self.block_size, self.latent_dim = latent.shape[-3:]
        layered = latent.dim() == 4
        self.num_layers = latent.shape[0] if layered else 1
        self.device = latent.device
        self.device_index = latent.get_device()
        self._desc = _lib.LatentCacheDesc(
            latent.data_ptr(), rope.data_ptr(), scale.data_ptr() if e8 else None,
            *(s[-3] for s in strides), *(s[0] if layered else 0 for s in strides),
            self.num_layers, self.num_blocks, self.block_size, self.latent_dim, self.dtype)
        self._ref = ctypes.cast(ctypes.pointer(self._desc), ctypes.c_void_p)

    def layer(self, i: int) -> "LatentCache":
        """The cache of one layer."""
        if self.latent.dim() != 4:
            raise ValueError("the cache has no layer dimension")
        return LatentCache(self.latent[i], self.rope[i],
                           self.scale[i] if self.scale is not None else None)

    def _one_layer(self):
        if self.latent.dim() != 3:
            raise ValueError("this call takes one layer: cache.layer(i)")
        return self._ref


def alloc_latent_cache(num_blocks: int, block_size: int, latent_dim: int, dtype: int, device,
                       layers: int = 0) -> LatentCache:
    """A cache of uninitialized pages (dtype BF16, F16 or E4M3), with a layer
    dimension if ``layers`` > 0."""
    if dtype not in _TORCH:
        raise ValueError(f"a cache is BF16, F16 or E4M3, got dtype code {dtype}")
    lead = ((layers,) if layers else ()) + (num_blocks, block_size)
    kind = _TORCH[dtype]
    row = torch.bfloat16 if dtype == E4M3 else kind
    pools = [torch.empty(lead + (latent_dim,), dtype=kind, device=device),
             torch.empty(lead + (LATENT_ROPE,), dtype=row, device=device)]
    if dtype == E4M3:
        pools.append(torch.empty(lead + (latent_dim // LATENT_GROUP,), dtype=torch.uint8,
                                 device=device))
    return LatentCache(*pools)


# ------------------------------------------------------------------ append

class LatentAppendOutputs(NamedTuple):
    q_rope: Optional[torch.Tensor]  # [max_rows, num_heads, 64]
    append_meta: torch.Tensor  # [2] int32


def alloc_latent_append_outputs(max_rows: int, num_heads: int,
                                cache: LatentCache) -> LatentAppendOutputs:
    q = None
    if num_heads:
        q = torch.empty(max_rows, num_heads, LATENT_ROPE, dtype=cache.row_dtype,
                        device=cache.device)
    return LatentAppendOutputs(q, torch.empty(2, dtype=_I32, device=cache.device))


def dspark_latent_append(B: int, kv: torch.Tensor, max_rows: int, cu_seqlens: torch.Tensor,
                         prefix_lens: torch.Tensor, block_table: torch.Tensor,
                         cache: LatentCache, out: LatentAppendOutputs,
                         q_rope: Optional[torch.Tensor] = None,
                         weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                         rope: Optional[torch.Tensor] = None, rope_interleaved: bool = False,
                         gamma: int = 0, tree_parents: Optional[torch.Tensor] = None,
                         stream=None) -> LatentAppendOutputs:
    """Norm (``weight`` [latent_dim]) and rotation (``rope`` [positions, 64]
    float32, cosines then sines) of the packed rows ``kv`` [max_rows, latent_dim
    + 64], their write into the cache, and the rotation of ``q_rope`` [max_rows,
    num_heads, 64], also as [num_heads, max_rows, 64] transposed; ``out.q_rope`` may
    be ``q_rope``. ``gamma`` 0: requests have
    any number of rows; otherwise up to gamma + 1, in a chain or in the trees of
    ``tree_parents`` [B, gamma]."""
    dev = _device(cache)
    dt, L = cache.row_dtype, cache.latent_dim
    table, width = _table(block_table, B, dev)
    hq, q_args, out_args = 0, (None, 0, 0), (None, 0, 0)
    if q_rope is not None:
        hq = q_rope.shape[1] if q_rope.dim() == 3 else 0
        q_args = _heads(q_rope, "q_rope", dt, max_rows, hq, LATENT_ROPE, dev)
        if out.q_rope is None:
            raise ValueError("out.q_rope is required with q_rope")
        out_args = _heads(out.q_rope, "out.q_rope", dt, max_rows, hq, LATENT_ROPE, dev)
        if hq == 0:
            raise ValueError("q_rope has no heads")
    rope_rows = 0
    if rope is not None:
        if rope.dim() != 2 or rope.shape[1] != LATENT_ROPE:
            raise ValueError(f"rope must be [positions, {LATENT_ROPE}]")
        rope_rows = rope.shape[0]
    args = (
        B, gamma, hq, _CODE[dt],
        *_lines(kv, "kv", dt, max_rows, L + LATENT_ROPE, dev),
        *q_args, max_rows,
        _on(cu_seqlens, "cu_seqlens", _I32, B + 1, dev),
        _on(prefix_lens, "prefix_lens", _I32, B, dev),
        _on(tree_parents, "tree_parents", _I32, B * gamma, dev, required=False),
        table, width,
        _on(weight, "weight", dt, L, dev, required=False), eps,
        _on(rope, "rope", torch.float32, 1, dev, required=False), rope_rows,
        1 if rope_interleaved else 0,
        *out_args, cache._one_layer(),
        _on(out.append_meta, "append_meta", _I32, 2, dev),
        _stream(stream),
    )
    _lib.check("dspark_latent_append", _lib.lib().dspark_latent_append(*args))
    return out


# ------------------------------------------------------------------ read

class LatentReadOutputs(NamedTuple):
    latent_out: torch.Tensor  # [max_rows, latent_dim]
    rope_out: torch.Tensor  # [max_rows, 64]
    read_meta: torch.Tensor  # [2] int32


def alloc_latent_read_outputs(max_rows: int, cache: LatentCache) -> LatentReadOutputs:
    return LatentReadOutputs(
        torch.empty(max_rows, cache.latent_dim, dtype=cache.row_dtype, device=cache.device),
        torch.empty(max_rows, LATENT_ROPE, dtype=cache.row_dtype, device=cache.device),
        torch.empty(2, dtype=_I32, device=cache.device),
    )


def dspark_latent_read(B: int, max_rows: int, cu_seqlens: torch.Tensor, starts: torch.Tensor,
                       block_table: torch.Tensor, cache: LatentCache, out: LatentReadOutputs,
                       stream=None) -> LatentReadOutputs:
    """Row ``cu_seqlens[r] + j`` of the outputs is cache index ``starts[r] + j``
    of request r (an 8-bit cache comes back in bfloat16)."""
    dev = _device(cache)
    dt = cache.row_dtype
    table, width = _table(block_table, B, dev)
    args = (
        B, max_rows,
        _on(cu_seqlens, "cu_seqlens", _I32, B + 1, dev),
        _on(starts, "starts", _I32, B, dev),
        table, width, cache._one_layer(),
        *_lines(out.latent_out, "latent_out", dt, max_rows, cache.latent_dim, dev),
        *_lines(out.rope_out, "rope_out", dt, max_rows, LATENT_ROPE, dev),
        _on(out.read_meta, "read_meta", _I32, 2, dev),
        _stream(stream),
    )
    _lib.check("dspark_latent_read", _lib.lib().dspark_latent_read(*args))
    return out


# ------------------------------------------------------------------ commit

def dspark_latent_commit(B: int, gamma: int, path_rows: torch.Tensor, num_correct: torch.Tensor,
                         prefix_lens: torch.Tensor, block_table: torch.Tensor, cache: LatentCache,
                         commit_meta: torch.Tensor, stream=None) -> torch.Tensor:
    """Moves the accepted path's cache rows to consecutive slots, in every layer
    of ``cache``. ``commit_meta`` [2] int32 receives rows moved and status."""
    dev = _device(cache)
    table, width = _table(block_table, B, dev)
    args = (
        B, gamma,
        _on(path_rows, "path_rows", _I32, B * (gamma + 1), dev),
        _on(num_correct, "num_correct", _I32, B, dev),
        _on(prefix_lens, "prefix_lens", _I32, B, dev),
        table, width, cache._ref,
        _on(commit_meta, "commit_meta", _I32, 2, dev),
        _stream(stream),
    )
    _lib.check("dspark_latent_commit", _lib.lib().dspark_latent_commit(*args))
    return commit_meta


# ------------------------------------------------------------------ attention, absorbed

def dspark_latent_attention_workspace_size(B: int, gamma: int, num_heads: int,
                                           latent_dim: int) -> int:
    return int(_lib.lib().dspark_latent_attention_workspace_size(B, gamma, num_heads, latent_dim))


def _outputs(max_rows: int, num_heads: int, dim: int, ws: int, cache: LatentCache,
             lse: bool) -> AttentionOutputs:
    dev = cache.device
    return AttentionOutputs(
        torch.empty(max_rows, num_heads, dim, dtype=cache.row_dtype, device=dev),
        torch.empty(max_rows, num_heads, dtype=torch.float32, device=dev) if lse else None,
        torch.empty(2, dtype=_I32, device=dev),
        torch.empty(max(ws, 256), dtype=torch.uint8, device=dev),
    )


def alloc_latent_attention_outputs(B: int, gamma: int, max_rows: int, num_heads: int,
                                   cache: LatentCache, lse: bool = False) -> AttentionOutputs:
    ws = dspark_latent_attention_workspace_size(B, gamma, num_heads, cache.latent_dim)
    return _outputs(max_rows, num_heads, cache.latent_dim, ws, cache, lse)


def dspark_latent_attention(B: int, gamma: int, q_latent: torch.Tensor, q_rope: torch.Tensor,
                            max_rows: int, cu_seqlens: torch.Tensor, prefix_lens: torch.Tensor,
                            block_table: torch.Tensor, cache: LatentCache, scale: float,
                            out: AttentionOutputs, tree_parents: Optional[torch.Tensor] = None,
                            stream=None) -> AttentionOutputs:
    """Attention of the packed rows over the latents of each request's context
    and its own tree (``tree_parents`` [B, gamma]; None: a chain). ``q_latent``
    [max_rows, num_heads, latent_dim] are the queries taken through the heads'
    key weights, ``q_rope`` [max_rows, num_heads, 64] their turned parts, both also
    transposed from a product for each head; the
    outputs are means of latents, for the heads' value weights."""
    dev = _device(cache)
    dt, L = cache.row_dtype, cache.latent_dim
    hq = q_latent.shape[1] if q_latent.dim() == 3 else 0
    table, width = _table(block_table, B, dev)
    args = (
        B, gamma, hq, _CODE[dt],
        *_heads(q_latent, "q_latent", dt, max_rows, hq, L, dev),
        *_heads(q_rope, "q_rope", dt, max_rows, hq, LATENT_ROPE, dev), max_rows,
        _on(cu_seqlens, "cu_seqlens", _I32, B + 1, dev),
        _on(prefix_lens, "prefix_lens", _I32, B, dev),
        _on(tree_parents, "tree_parents", _I32, B * gamma, dev, required=False),
        table, width, cache._one_layer(), scale,
        *_dense_out(out.out, "out", dt, max_rows, hq, L, dev),
        _on(out.lse, "lse", torch.float32, max_rows * hq, dev, required=False),
        _on(out.attention_meta, "attention_meta", _I32, 2, dev),
        _on(out.workspace, "workspace", torch.uint8, 1, dev), out.workspace.numel(),
        _stream(stream),
    )
    _lib.check("dspark_latent_attention", _lib.lib().dspark_latent_attention(*args))
    return out


# ------------------------------------------------------------------ attention, expanded

def dspark_latent_prefill_workspace_size(B: int, max_rows: int, max_keys: int, num_heads: int,
                                         nope: int, latent_dim: int) -> int:
    return int(_lib.lib().dspark_latent_prefill_workspace_size(B, max_rows, max_keys, num_heads,
                                                               nope, latent_dim))


def alloc_latent_prefill_outputs(B: int, max_rows: int, max_keys: int, num_heads: int, nope: int,
                                 cache: LatentCache, lse: bool = False) -> AttentionOutputs:
    ws = dspark_latent_prefill_workspace_size(B, max_rows, max_keys, num_heads, nope,
                                              cache.latent_dim)
    return _outputs(max_rows, num_heads, nope, ws, cache, lse)


def dspark_latent_prefill(B: int, q: torch.Tensor, w_k: torch.Tensor, w_v: torch.Tensor,
                          max_rows: int, max_keys: int, cu_seqlens: torch.Tensor,
                          prefix_lens: torch.Tensor, block_table: torch.Tensor,
                          cache: LatentCache, scale: float, out: AttentionOutputs,
                          stream=None) -> AttentionOutputs:
    """Causal attention of prompt rows ``q`` [max_rows, num_heads, nope + 64]
    over their requests' cached tokens and themselves, with keys and values
    expanded by ``w_k`` and ``w_v`` [num_heads, nope, latent_dim] (which may be
    parts of one weight). ``max_keys``: cached tokens of all requests together,
    their rows included, at most. The workspace grows with heads times keys; a share of
    the heads at a time (``q[:, a:b]``, ``w_k[a:b]``, ``w_v[a:b]``, an output
    ``out[:, a:b]``) needs that share of it."""
    dev = _device(cache)
    dt, L = cache.row_dtype, cache.latent_dim
    hq, dim = (q.shape[1], q.shape[2]) if q.dim() == 3 else (0, 0)
    n = dim - LATENT_ROPE
    table, width = _table(block_table, B, dev)
    weights = []
    for name, t in (("w_k", w_k), ("w_v", w_v)):
        ptr, head, row = _heads(t, name, dt, hq, n, L, dev)
        if t.shape[0] != hq:
            raise ValueError(f"{name} holds {t.shape[0]} heads, q has {hq}")
        if row != L:
            raise ValueError(f"the rows of {name} must be dense")
        weights.append((ptr, head))
    if weights[0][1] != weights[1][1]:
        raise ValueError("w_k and w_v need the same strides")
    args = (
        B, hq, n, _CODE[dt],
        *_dense_out(q, "q", dt, max_rows, hq, dim, dev),
        weights[0][0], weights[1][0], weights[0][1], max_rows, max_keys,
        _on(cu_seqlens, "cu_seqlens", _I32, B + 1, dev),
        _on(prefix_lens, "prefix_lens", _I32, B, dev),
        table, width, cache._one_layer(), scale,
        *_dense_out(out.out, "out", dt, max_rows, hq, n, dev),
        _on(out.lse, "lse", torch.float32, max_rows * hq, dev, required=False),
        _on(out.attention_meta, "prefill_meta", _I32, 2, dev),
        _on(out.workspace, "workspace", torch.uint8, 1, dev), out.workspace.numel(),
        _stream(stream),
    )
    _lib.check("dspark_latent_prefill", _lib.lib().dspark_latent_prefill(*args))
    return out
