"""The target pass between pack and accept: paged cache, attention, tree accept.

Like the rest of the binding, the functions carry the names of the C entry
points, check their tensors, pass raw pointers and the current HIP stream, and
raise ``DsparkError`` on a non-OK status. Every tensor of a call must live on
the current device. ``KvCache`` describes a cache once; calls of a layer take
``cache.layer(i)``.
"""

from __future__ import annotations

import ctypes
from array import array
from typing import NamedTuple, Optional, Sequence

import torch

from . import _lib
from . import _logit_dtype, _stream, dspark_accept_workspace_size
from ._lib import BF16, E4M3, F16

_I32 = torch.int32
_CODE = {torch.bfloat16: BF16, torch.float16: F16, torch.float8_e4m3fn: E4M3}
_TORCH = {code: t for t, code in _CODE.items()}


def _on(t: Optional[torch.Tensor], name: str, dtype, numel: int, dev: int, required: bool = True):
    """The pointer of a dense tensor of at least ``numel`` elements on device ``dev``."""
    if t is None:
        if required and numel > 0:
            raise ValueError(f"{name} is required")
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the current device cuda:{dev}, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < numel:
        raise ValueError(f"{name} holds {t.numel()} elements, needs {numel}")
    return t.data_ptr()


def _rows(t: torch.Tensor, name: str, dtype, rows: int, heads: int, dim: int, dev: int):
    """Pointer and row stride of [rows, heads, dim] with dense heads."""
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
    if s[2] != 1 or (heads > 1 and s[1] != dim):
        raise ValueError(f"the heads of {name} must be dense")
    # a single row has no stride of its own
    return t.data_ptr(), (s[0] if shape[0] > 1 else heads * dim)


def _table(block_table: torch.Tensor, B: int, dev: int):
    if block_table is None or block_table.dim() != 2:
        raise ValueError("block_table must be [B, table_width]")
    width = block_table.shape[1]
    return _on(block_table, "block_table", _I32, B * width, dev), width


def _device(cache: "KvCache") -> int:
    dev = torch.cuda.current_device()
    if cache.device_index != dev:
        raise ValueError(f"the cache is on cuda:{cache.device_index}, the current device is cuda:{dev}")
    return dev


# ------------------------------------------------------------------ cache

def _strides(t: torch.Tensor) -> tuple:
    """Strides in which a dimension of one has its dense one: it has none of its own."""
    out, dense = [], 1
    for n, s in zip(reversed(t.shape), reversed(t.stride())):
        out.append(s if n != 1 else dense)
        dense = out[-1] * n
    return tuple(reversed(out))


class KvCache:
    """A paged cache: ``k`` and ``v`` [num_blocks, num_kv_heads, block_size,
    head_dim] in bfloat16, float16 or float8_e4m3fn, or with a leading layer
    dimension. With float8_e4m3fn, ``k_scale`` and ``v_scale`` (uint8, the same
    shape without head_dim) hold the exponent bytes: value = code * 2^(byte -
    127). The strides of pages and layers are free, so ``k`` and ``v`` may be
    views of one pool; those of the last three dimensions are dense."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: Optional[torch.Tensor] = None,
                 v_scale: Optional[torch.Tensor] = None):
        if not isinstance(k, torch.Tensor) or not isinstance(v, torch.Tensor):
            raise TypeError("k and v must be torch.Tensors")
        if k.dtype not in _CODE:
            raise TypeError(f"a cache is bfloat16, float16 or float8_e4m3fn, got {k.dtype}")
        if k.dim() not in (4, 5) or k.shape != v.shape or k.dtype != v.dtype or k.device != v.device:
            raise ValueError("k and v must be [(layers,) num_blocks, num_kv_heads, block_size, "
                             "head_dim] alike")
        if not k.is_cuda:
            raise ValueError(f"the cache must be on a CUDA device, got {k.device}")
        heads, size, dim = k.shape[-3:]
        dense = (size * dim, dim, 1)
        ks = _strides(k)
        if ks != _strides(v) or ks[-3:] != dense:
            raise ValueError("k and v need the same strides, dense in their last three dimensions")
        e8 = k.dtype == torch.float8_e4m3fn
        ss = None
        if e8:
            for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
                if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8:
                    raise TypeError(f"{name} must be a uint8 tensor")
                if t.shape != k.shape[:-1] or t.device != k.device:
                    raise ValueError(f"{name} must be {tuple(k.shape[:-1])} on {k.device}")
                ss = ss or _strides(t)
                if ss[-2:] != (size, 1) or _strides(t) != ss:
                    raise ValueError("k_scale and v_scale need the same strides, dense in their "
                                     "last two dimensions")
        elif k_scale is not None or v_scale is not None:
            raise ValueError("only a float8_e4m3fn cache has scales")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.dtype = _CODE[k.dtype]
        self.num_blocks, self.num_kv_heads, self.block_size, self.head_dim = k.shape[-4:]
        self.num_layers = k.shape[0] if k.dim() == 5 else 1
        #: type of the rows that go in and come out
        self.row_dtype = torch.bfloat16 if e8 else k.dtype
        self.device = k.device
        self.device_index = k.get_device()
        self._desc = _lib.KvCacheDesc(
            k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if e8 else None,
            v_scale.data_ptr() if e8 else None,
            ks[-4], ss[-3] if e8 else 0,
            ks[0] if k.dim() == 5 else 0, ss[0] if e8 and k.dim() == 5 else 0,
            self.num_layers, self.num_blocks, heads, size, dim, self.dtype)
        self._ref = ctypes.cast(ctypes.pointer(self._desc), ctypes.c_void_p)

    def layer(self, i: int) -> "KvCache":
        """The cache of one layer."""
        if self.k.dim() != 5:
            raise ValueError("the cache has no layer dimension")
        sc = self.k_scale is not None
        return KvCache(self.k[i], self.v[i], self.k_scale[i] if sc else None,
                       self.v_scale[i] if sc else None)

    def _one_layer(self):
        if self.k.dim() != 4:
            raise ValueError("this call takes one layer: cache.layer(i)")
        return self._ref


def alloc_kv_cache(num_blocks: int, num_kv_heads: int, block_size: int, head_dim: int, dtype: int,
                   device, layers: int = 0) -> KvCache:
    """A cache of uninitialized pages (dtype BF16, F16 or E4M3), with a layer
    dimension if ``layers`` > 0."""
    if dtype not in _TORCH:
        raise ValueError(f"a cache is BF16, F16 or E4M3, got dtype code {dtype}")
    shape = ((layers,) if layers else ()) + (num_blocks, num_kv_heads, block_size, head_dim)
    pools = [torch.empty(shape, dtype=_TORCH[dtype], device=device) for _ in range(2)]
    if dtype == E4M3:
        pools += [torch.empty(shape[:-1], dtype=torch.uint8, device=device) for _ in range(2)]
    return KvCache(*pools)


# ------------------------------------------------------------------ append

class AppendOutputs(NamedTuple):
    q_out: torch.Tensor  # [max_rows, num_heads, head_dim]
    append_meta: torch.Tensor  # [2] int32


def alloc_append_outputs(max_rows: int, num_heads: int, cache: KvCache) -> AppendOutputs:
    return AppendOutputs(
        torch.empty(max_rows, num_heads, cache.head_dim, dtype=cache.row_dtype, device=cache.device),
        torch.empty(2, dtype=_I32, device=cache.device),
    )


def dspark_kv_append(B: int, gamma: int, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                     max_rows: int, cu_seqlens: torch.Tensor, prefix_lens: torch.Tensor,
                     block_table: torch.Tensor, cache: KvCache, out: AppendOutputs,
                     q_weight: Optional[torch.Tensor] = None,
                     k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                     rope: Optional[torch.Tensor] = None, rope_interleaved: bool = False,
                     tree_parents: Optional[torch.Tensor] = None, stream=None) -> AppendOutputs:
    """Norms (``q_weight``, ``k_weight``: [head_dim]) and rotation (``rope``:
    [positions, rope_dim] float32, cosines then sines) of the packed rows ``q``
    [max_rows, num_heads, head_dim] and ``k``, and the write of ``k`` and ``v``
    [max_rows, num_kv_heads, head_dim] into the cache. ``out.q_out`` may be
    ``q``. The three may be parts of one buffer's rows."""
    dev = _device(cache)
    dt, D, hkv = cache.row_dtype, cache.head_dim, cache.num_kv_heads
    hq = q.shape[1] if q.dim() == 3 else 0
    table, width = _table(block_table, B, dev)
    rope_rows = rope_dim = 0
    if rope is not None:
        if rope.dim() != 2:
            raise ValueError("rope must be [positions, rope_dim]")
        rope_rows, rope_dim = rope.shape
    args = (
        B, gamma, hq, _CODE[dt],
        *_rows(q, "q", dt, max_rows, hq, D, dev),
        *_rows(k, "k", dt, max_rows, hkv, D, dev),
        *_rows(v, "v", dt, max_rows, hkv, D, dev), max_rows,
        _on(cu_seqlens, "cu_seqlens", _I32, B + 1, dev),
        _on(prefix_lens, "prefix_lens", _I32, B, dev),
        _on(tree_parents, "tree_parents", _I32, B * gamma, dev, required=False),
        table, width,
        _on(q_weight, "q_weight", dt, D, dev, required=False),
        _on(k_weight, "k_weight", dt, D, dev, required=False), eps,
        _on(rope, "rope", torch.float32, 1, dev, required=False), rope_rows, rope_dim,
        1 if rope_interleaved else 0,
        *_rows(out.q_out, "q_out", dt, max_rows, hq, D, dev),
        cache._one_layer(),
        _on(out.append_meta, "append_meta", _I32, 2, dev),
        _stream(stream),
    )
    _lib.check("dspark_kv_append", _lib.lib().dspark_kv_append(*args))
    return out


def dspark_kv_append_axes(B: int, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, max_rows: int,
                          cu_seqlens: torch.Tensor, prefix_lens: torch.Tensor,
                          positions: torch.Tensor, pair_axis: Sequence[int],
                          block_table: torch.Tensor, cache: KvCache, out: AppendOutputs,
                          rope: torch.Tensor, q_weight: Optional[torch.Tensor] = None,
                          k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                          rope_interleaved: bool = False, stream=None) -> AppendOutputs:
    """dspark_kv_append for rows whose pairs turn by positions on several axes:
    pair i by ``positions[pair_axis[i]]`` (``positions``: [axes, >= max_rows]
    int32, rows dense; ``pair_axis``: rope_dim / 2 whole numbers). Requests have
    any number of rows."""
    dev = _device(cache)
    dt, D, hkv = cache.row_dtype, cache.head_dim, cache.num_kv_heads
    hq = q.shape[1] if q.dim() == 3 else 0
    table, width = _table(block_table, B, dev)
    if rope is None or rope.dim() != 2:
        raise ValueError("rope must be [positions, rope_dim]")
    rope_rows, rope_dim = rope.shape
    # (5 us less per call than a ctypes array)
    axes = array("i", pair_axis)
    if len(axes) != rope_dim // 2:
        raise ValueError(f"pair_axis holds {len(axes)} axes, needs {rope_dim // 2}")
    if not isinstance(positions, torch.Tensor) or positions.dtype != _I32:
        raise TypeError("positions must be an int32 tensor")
    if positions.get_device() != dev:
        raise ValueError(f"positions must be on the current device cuda:{dev}, got {positions.device}")
    if positions.dim() != 2 or positions.shape[1] < max_rows:
        raise ValueError(f"positions must be [axes, >= {max_rows}], got {tuple(positions.shape)}")
    ld = positions.stride(0) if positions.shape[0] > 1 else max(max_rows, positions.shape[1])
    if positions.shape[1] > 1 and positions.stride(1) != 1:
        raise ValueError("the rows of positions must be dense")
    args = (
        B, hq, _CODE[dt],
        *_rows(q, "q", dt, max_rows, hq, D, dev),
        *_rows(k, "k", dt, max_rows, hkv, D, dev),
        *_rows(v, "v", dt, max_rows, hkv, D, dev), max_rows,
        _on(cu_seqlens, "cu_seqlens", _I32, B + 1, dev),
        _on(prefix_lens, "prefix_lens", _I32, B, dev),
        positions.data_ptr(), ld, positions.shape[0], axes.buffer_info()[0],
        table, width,
        _on(q_weight, "q_weight", dt, D, dev, required=False),
        _on(k_weight, "k_weight", dt, D, dev, required=False), eps,
        _on(rope, "rope", torch.float32, 1, dev), rope_rows, rope_dim,
        1 if rope_interleaved else 0,
        *_rows(out.q_out, "q_out", dt, max_rows, hq, D, dev),
        cache._one_layer(),
        _on(out.append_meta, "append_meta", _I32, 2, dev),
        _stream(stream),
    )
    _lib.check("dspark_kv_append_axes", _lib.lib().dspark_kv_append_axes(*args))
    return out


# ------------------------------------------------------------------ read

class KvReadOutputs(NamedTuple):
    k_out: torch.Tensor  # [max_rows, num_kv_heads, head_dim]
    v_out: torch.Tensor
    read_meta: torch.Tensor  # [2] int32


def alloc_kv_read_outputs(max_rows: int, cache: KvCache) -> KvReadOutputs:
    shape = (max_rows, cache.num_kv_heads, cache.head_dim)
    return KvReadOutputs(
        torch.empty(shape, dtype=cache.row_dtype, device=cache.device),
        torch.empty(shape, dtype=cache.row_dtype, device=cache.device),
        torch.empty(2, dtype=_I32, device=cache.device),
    )


def dspark_kv_read(B: int, max_rows: int, cu_seqlens: torch.Tensor, starts: torch.Tensor,
                   block_table: torch.Tensor, cache: KvCache, out: KvReadOutputs,
                   stream=None) -> KvReadOutputs:
    """Row ``cu_seqlens[r] + j`` of the outputs is cache index ``starts[r] + j``
    of request r (an 8-bit cache comes back in bfloat16)."""
    dev = _device(cache)
    dt, D, hkv = cache.row_dtype, cache.head_dim, cache.num_kv_heads
    table, width = _table(block_table, B, dev)
    k_ptr, ld = _rows(out.k_out, "k_out", dt, max_rows, hkv, D, dev)
    v_ptr, v_ld = _rows(out.v_out, "v_out", dt, max_rows, hkv, D, dev)
    if ld != v_ld:
        raise ValueError("k_out and v_out need the same row stride")
    args = (
        B, max_rows,
        _on(cu_seqlens, "cu_seqlens", _I32, B + 1, dev),
        _on(starts, "starts", _I32, B, dev),
        table, width, cache._one_layer(), k_ptr, v_ptr, ld,
        _on(out.read_meta, "read_meta", _I32, 2, dev),
        _stream(stream),
    )
    _lib.check("dspark_kv_read", _lib.lib().dspark_kv_read(*args))
    return out


# ------------------------------------------------------------------ attention

class AttentionOutputs(NamedTuple):
    out: torch.Tensor  # [max_rows, num_heads, head_dim]
    lse: Optional[torch.Tensor]  # [max_rows, num_heads] float32
    attention_meta: torch.Tensor  # [2] int32
    workspace: torch.Tensor  # uint8 scratch (no initialization needed)


def dspark_tree_attention_workspace_size(B: int, gamma: int, num_heads: int, num_kv_heads: int,
                                         head_dim: int) -> int:
    return int(_lib.lib().dspark_tree_attention_workspace_size(B, gamma, num_heads, num_kv_heads,
                                                               head_dim))


def alloc_attention_outputs(B: int, gamma: int, max_rows: int, num_heads: int, cache: KvCache,
                            lse: bool = False) -> AttentionOutputs:
    dev = cache.device
    ws = dspark_tree_attention_workspace_size(B, gamma, num_heads, cache.num_kv_heads,
                                              cache.head_dim)
    return AttentionOutputs(
        torch.empty(max_rows, num_heads, cache.head_dim, dtype=cache.row_dtype, device=dev),
        torch.empty(max_rows, num_heads, dtype=torch.float32, device=dev) if lse else None,
        torch.empty(2, dtype=_I32, device=dev),
        torch.empty(max(ws, 256), dtype=torch.uint8, device=dev),
    )


def dspark_tree_attention(B: int, gamma: int, q: torch.Tensor, max_rows: int,
                          cu_seqlens: torch.Tensor, prefix_lens: torch.Tensor,
                          block_table: torch.Tensor, cache: KvCache, scale: float,
                          out: AttentionOutputs, tree_parents: Optional[torch.Tensor] = None,
                          stream=None) -> AttentionOutputs:
    """Attention of the packed rows ``q`` [max_rows, num_heads, head_dim] over
    each request's context and its own tree (``tree_parents`` [B, gamma]; None:
    a chain). The step's keys and values must be in the cache."""
    dev = _device(cache)
    dt, D = cache.row_dtype, cache.head_dim
    hq = q.shape[1] if q.dim() == 3 else 0
    table, width = _table(block_table, B, dev)
    args = (
        B, gamma, hq, _CODE[dt],
        *_rows(q, "q", dt, max_rows, hq, D, dev), max_rows,
        _on(cu_seqlens, "cu_seqlens", _I32, B + 1, dev),
        _on(prefix_lens, "prefix_lens", _I32, B, dev),
        _on(tree_parents, "tree_parents", _I32, B * gamma, dev, required=False),
        table, width, cache._one_layer(), scale,
        *_rows(out.out, "out", dt, max_rows, hq, D, dev),
        _on(out.lse, "lse", torch.float32, max_rows * hq, dev, required=False),
        _on(out.attention_meta, "attention_meta", _I32, 2, dev),
        _on(out.workspace, "workspace", torch.uint8, 1, dev), out.workspace.numel(),
        _stream(stream),
    )
    _lib.check("dspark_tree_attention", _lib.lib().dspark_tree_attention(*args))
    return out


# ------------------------------------------------------------------ tree accept

class TreeAcceptOutputs(NamedTuple):
    row_argmax: torch.Tensor  # [max_rows] int32
    num_correct: torch.Tensor  # [B] int32
    bonus: torch.Tensor
    commit_lens: torch.Tensor
    out_tokens: torch.Tensor  # [B, gamma+1] int32
    path_rows: torch.Tensor  # [B, gamma+1] int32
    new_seq_lens: Optional[torch.Tensor]
    accept_meta: torch.Tensor  # [2] int32
    workspace: torch.Tensor  # uint8 scratch (no initialization needed)


def alloc_tree_accept_outputs(B: int, gamma: int, max_rows: int, V: int, dt: int, device,
                              new_seq=True) -> TreeAcceptOutputs:
    ws = dspark_accept_workspace_size(max_rows, V, dt)
    return TreeAcceptOutputs(
        torch.empty(max(max_rows, 1), dtype=_I32, device=device),
        torch.empty(B, dtype=_I32, device=device),
        torch.empty(B, dtype=_I32, device=device),
        torch.empty(B, dtype=_I32, device=device),
        torch.empty(B, gamma + 1, dtype=_I32, device=device),
        torch.empty(B, gamma + 1, dtype=_I32, device=device),
        torch.empty(B, dtype=_I32, device=device) if new_seq else None,
        torch.empty(2, dtype=_I32, device=device),
        torch.empty(max(ws, 256), dtype=torch.uint8, device=device),
    )


def dspark_tree_accept(B: int, gamma: int, V: int, dt: int, packed_logits: torch.Tensor, ld: int,
                       max_rows: int, cu_seqlens: torch.Tensor, draft_tokens: torch.Tensor,
                       tree_parents: Optional[torch.Tensor], prefix_lens,
                       out: TreeAcceptOutputs, stream=None) -> TreeAcceptOutputs:
    """Greedy accept along each request's draft tree (``tree_parents`` None: a
    chain, the result of dspark_accept)."""
    dev = torch.cuda.current_device()
    args = (
        B, gamma, V, dt,
        _on(packed_logits, "packed_logits", _logit_dtype(dt), max_rows * ld if max_rows else 0, dev),
        ld, max_rows,
        _on(cu_seqlens, "cu_seqlens", _I32, B + 1, dev),
        _on(draft_tokens, "draft_tokens", _I32, B * gamma, dev),
        _on(tree_parents, "tree_parents", _I32, B * gamma, dev, required=False),
        _on(prefix_lens, "prefix_lens", _I32, B, dev, required=False),
        _on(out.row_argmax, "row_argmax", _I32, max_rows, dev),
        _on(out.num_correct, "num_correct", _I32, B, dev),
        _on(out.bonus, "bonus", _I32, B, dev),
        _on(out.commit_lens, "commit_lens", _I32, B, dev),
        _on(out.out_tokens, "out_tokens", _I32, B * (gamma + 1), dev),
        _on(out.path_rows, "path_rows", _I32, B * (gamma + 1), dev),
        _on(out.new_seq_lens, "new_seq_lens", _I32, B, dev, required=False),
        _on(out.accept_meta, "accept_meta", _I32, 2, dev),
        _on(out.workspace, "workspace", torch.uint8, 1, dev), out.workspace.numel(),
        _stream(stream),
    )
    _lib.check("dspark_tree_accept", _lib.lib().dspark_tree_accept(*args))
    return out


# ------------------------------------------------------------------ commit

def dspark_kv_commit(B: int, gamma: int, path_rows: torch.Tensor, num_correct: torch.Tensor,
                     prefix_lens: torch.Tensor, block_table: torch.Tensor, cache: KvCache,
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
    _lib.check("dspark_kv_commit", _lib.lib().dspark_kv_commit(*args))
    return commit_meta
