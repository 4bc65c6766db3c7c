"""ctypes loader for libdspark.so, with the C signatures of include/dspark.h.

Loading never touches a GPU, so the library can be loaded (and its host-side
argument checks exercised) on a machine without one. If the library has not
been built, ``lib()`` raises: there is no fallback implementation.
"""

from __future__ import annotations

import ctypes
from ctypes import c_double, c_float, c_int, c_int32, c_int64, c_size_t, c_void_p
from pathlib import Path

_PKG = Path(__file__).resolve().parent
LIB_PATH = _PKG / "libdspark.so"
HOSTCHECK_PATH = _PKG / "libdspark_hostcheck.so"

OK, E_INVALID, E_UNSUPPORTED, E_WORKSPACE, E_LAUNCH = 0, 1, 2, 3, 4
F32, BF16, F16, E4M3 = 0, 1, 2, 3
IN_CONF_LOGITS, IN_COND, IN_SURVIVAL = 0, 1, 2
DATA_BAD_COST, DATA_BAD_CONF, DATA_BAD_LENS, DATA_BAD_LOGITS = 1, 2, 4, 8
DATA_BAD_TREE, DATA_BAD_PAGE, DATA_BAD_POS = 16, 32, 64
MAX_GAMMA, MAX_CANDIDATES, MAX_BATCH, MAX_TIERS, MAX_VOCAB = 64, 8192, 8192, 32, 262144
MAX_SPS_PROBES = 512
STS_MAX_GRID, STS_MAX_BINS, STS_MAX_RECORDS = 128, 64, 4194304
COST_ADDITIVE, COST_SPS1D = 0, 1
MAX_HEADS, MAX_GROUP, MAX_LAYERS = 256, 64, 1024
MAX_AXES, LATENT_MAX_HEADS, LATENT_ROPE, LATENT_GROUP = 4, 128, 64, 128
LATENT_MAX_KEYS = 134217728


class PlanOptions(ctypes.Structure):
    """dspark_plan_options of include/dspark.h."""
    _fields_ = [("cost_mode", c_int), ("sps_m", c_void_p), ("sps", c_void_p),
                ("sps_len", c_int32), ("align_to_tier", c_int32)]


class KvCacheDesc(ctypes.Structure):
    """dspark_kv_cache of include/dspark.h."""
    _fields_ = [("k", c_void_p), ("v", c_void_p), ("k_scale", c_void_p), ("v_scale", c_void_p),
                ("block_stride", c_int64), ("scale_block_stride", c_int64),
                ("layer_stride", c_int64), ("scale_layer_stride", c_int64),
                ("num_layers", c_int32), ("num_blocks", c_int32), ("num_kv_heads", c_int32),
                ("block_size", c_int32), ("head_dim", c_int32), ("dtype", c_int)]


class LatentCacheDesc(ctypes.Structure):
    """dspark_latent_cache of include/dspark.h."""
    _fields_ = [("latent", c_void_p), ("rope", c_void_p), ("scale", c_void_p),
                ("block_stride", c_int64), ("rope_block_stride", c_int64),
                ("scale_block_stride", c_int64), ("layer_stride", c_int64),
                ("rope_layer_stride", c_int64), ("scale_layer_stride", c_int64),
                ("num_layers", c_int32), ("num_blocks", c_int32), ("block_size", c_int32),
                ("latent_dim", c_int32), ("dtype", c_int)]


# name -> (restype, argtypes), mirroring include/dspark.h
SIGNATURES = {
    "dspark_plan": (c_int, [
        c_int32, c_int32, c_int, c_void_p, c_void_p, c_int32, c_int32, c_float, c_int32,
        c_int32, c_float, c_void_p, c_int32, c_void_p, c_int32, c_void_p, c_void_p, c_void_p,
        c_void_p, c_void_p, c_void_p]),
    "dspark_plan_pack": (c_int, [
        c_int32, c_int32, c_int, c_void_p, c_void_p, c_int32, c_int32, c_float, c_int32,
        c_int32, c_float, c_void_p, c_int32, c_void_p, c_int32, c_void_p, c_void_p, c_void_p,
        c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_int32, c_void_p, c_void_p,
        c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]),
    "dspark_plan_pack_ex": (c_int, [
        c_int32, c_int32, c_int, c_void_p, c_void_p, c_int32, c_int32, c_float, c_int32,
        c_int32, c_float, c_void_p, c_int32, c_void_p, c_int32, c_void_p, c_void_p, c_void_p,
        c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_int32, c_void_p, c_void_p,
        c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]),
    "dspark_pack": (c_int, [
        c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_void_p, c_int32, c_void_p, c_void_p,
        c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]),
    "dspark_accept": (c_int, [
        c_int32, c_int32, c_int32, c_int, c_void_p, c_int64, c_int32, c_void_p, c_void_p,
        c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
        c_void_p, c_void_p, c_size_t, c_void_p]),
    "dspark_accept_noalloc": (c_int, [
        c_int32, c_int32, c_int32, c_int, c_void_p, c_int64, c_int32, c_void_p, c_void_p,
        c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
        c_void_p, c_void_p]),
    "dspark_cap_accept": (c_int, [
        c_int32, c_int32, c_int32, c_int, c_void_p, c_int64, c_void_p, c_void_p, c_void_p,
        c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
        c_void_p, c_void_p, c_size_t, c_void_p]),
    "dspark_scatter_to_strided": (c_int, [
        c_int32, c_int32, c_void_p, c_int32, c_void_p, c_int64, c_void_p, c_int64, c_int64,
        c_void_p, c_void_p]),
    "dspark_accept_workspace_size": (c_size_t, [c_int32, c_int32, c_int]),
    "dspark_accept_sampling": (c_int, [
        c_int32, c_int32, c_int32, c_int, c_void_p, c_int64, c_int32, c_void_p, c_void_p,
        c_int64, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
        c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "dspark_accept_sampling_workspace_size": (c_size_t, [c_int32, c_int32, c_int32, c_int]),
    "dspark_sts_fit": (c_int, [
        c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_int32, c_int32, c_void_p, c_void_p,
        c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "dspark_sts_workspace_size": (c_size_t, [c_int32, c_int32, c_int32, c_int32]),
    "dspark_tv_accept": (c_int, [
        c_int32, c_int32, c_int32, c_int, c_void_p, c_int64, c_void_p, c_int64, c_int32,
        c_void_p, c_void_p, c_void_p]),
    "dspark_kv_append": (c_int, [
        c_int32, c_int32, c_int32, c_int, c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int64,
        c_int32, c_void_p, c_void_p, c_void_p, c_void_p, c_int32, c_void_p, c_void_p, c_float,
        c_void_p, c_int32, c_int32, c_int32, c_void_p, c_int64, c_void_p, c_void_p, c_void_p]),
    "dspark_kv_read": (c_int, [
        c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_int32, c_void_p, c_void_p, c_void_p,
        c_int64, c_void_p, c_void_p]),
    "dspark_tree_attention": (c_int, [
        c_int32, c_int32, c_int32, c_int, c_void_p, c_int64, c_int32, c_void_p, c_void_p,
        c_void_p, c_void_p, c_int32, c_void_p, c_float, c_void_p, c_int64, c_void_p, c_void_p,
        c_void_p, c_size_t, c_void_p]),
    "dspark_tree_attention_workspace_size": (c_size_t, [
        c_int32, c_int32, c_int32, c_int32, c_int32]),
    "dspark_tree_accept": (c_int, [
        c_int32, c_int32, c_int32, c_int, c_void_p, c_int64, c_int32, c_void_p, c_void_p,
        c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
        c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "dspark_kv_commit": (c_int, [
        c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_void_p, c_int32, c_void_p, c_void_p,
        c_void_p]),
    "dspark_kv_append_axes": (c_int, [
        c_int32, c_int32, c_int, c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int64, c_int32,
        c_void_p, c_void_p, c_void_p, c_int64, c_int32, c_void_p, c_void_p, c_int32, c_void_p,
        c_void_p, c_float, c_void_p, c_int32, c_int32, c_int32, c_void_p, c_int64, c_void_p,
        c_void_p, c_void_p]),
    "dspark_latent_append": (c_int, [
        c_int32, c_int32, c_int32, c_int, c_void_p, c_int64, c_void_p, c_int64, c_int64, c_int32,
        c_void_p, c_void_p, c_void_p, c_void_p, c_int32, c_void_p, c_float, c_void_p, c_int32,
        c_int32, c_void_p, c_int64, c_int64, c_void_p, c_void_p, c_void_p]),
    "dspark_latent_read": (c_int, [
        c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_int32, c_void_p, c_void_p, c_int64,
        c_void_p, c_int64, c_void_p, c_void_p]),
    "dspark_latent_commit": (c_int, [
        c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_void_p, c_int32, c_void_p, c_void_p,
        c_void_p]),
    "dspark_latent_attention": (c_int, [
        c_int32, c_int32, c_int32, c_int, c_void_p, c_int64, c_int64, c_void_p, c_int64, c_int64,
        c_int32, c_void_p, c_void_p, c_void_p, c_void_p, c_int32, c_void_p, c_float, c_void_p,
        c_int64, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "dspark_latent_attention_workspace_size": (c_size_t, [c_int32, c_int32, c_int32, c_int32]),
    "dspark_latent_prefill": (c_int, [
        c_int32, c_int32, c_int32, c_int, c_void_p, c_int64, c_void_p, c_void_p, c_int64, c_int32,
        c_int32, c_void_p, c_void_p, c_void_p, c_int32, c_void_p, c_float, c_void_p, c_int64,
        c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "dspark_latent_prefill_workspace_size": (c_size_t, [
        c_int32, c_int32, c_int32, c_int32, c_int32, c_int32]),
    "dspark_status_str": (ctypes.c_char_p, [c_int]),
    "dspark_last_error": (ctypes.c_char_p, []),
    "dspark_version": (c_int32, []),
}

_lib = None
_hostcheck = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not LIB_PATH.exists():
            raise RuntimeError(
                f"{LIB_PATH} is not built; run `python -m dspark_verify_scheduling_amd.build` "
                "(or __graft_entry__.build())")
        handle = ctypes.CDLL(str(LIB_PATH))
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def hostcheck() -> ctypes.CDLL:
    """Host-only build of the device sigmoid and of the cache read's search
    (CPU tests of their logic)."""
    global _hostcheck
    if _hostcheck is None:
        if not HOSTCHECK_PATH.exists():
            raise RuntimeError(f"{HOSTCHECK_PATH} is not built")
        handle = ctypes.CDLL(str(HOSTCHECK_PATH))
        handle.dspark_hostcheck_sigmoid.restype = None
        handle.dspark_hostcheck_sigmoid.argtypes = [c_void_p, c_void_p, c_void_p, c_int64, c_int]
        handle.dspark_hostcheck_request_search.restype = None
        handle.dspark_hostcheck_request_search.argtypes = [c_void_p, c_int32, c_void_p, c_void_p,
                                                           c_int64]
        _hostcheck = handle
    return _hostcheck


def last_error() -> str:
    return lib().dspark_last_error().decode()


def status_str(st: int) -> str:
    return lib().dspark_status_str(st).decode()


class DsparkError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} -> {status_str(status)}: {last_error()}")


def check(fn: str, status: int) -> None:
    if status != OK:
        raise DsparkError(fn, status)


__all__ = ["lib", "hostcheck", "check", "DsparkError", "SIGNATURES", "c_double"]
