"""ctypes binding of the eviction of libpfkv.so (argument marshalling only).

Every function has the name of the C entry point that it calls (see
``include/pfkv_evict.h`` for the full contract); caches, tables, streams and
errors are those of ``binding``.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import binding as B
from . import prefix as P
from . import rope as R

# every symbol include/pfkv_evict.h declares
EXPORTED: tuple = ("pfkv_kv_evict_workspace_size", "pfkv_kv_evict")


def lib() -> ctypes.CDLL:
    """libpfkv.so with these calls' signatures set."""
    L = B.lib()
    if not getattr(L, "_evict_calls", False):
        P_, I32, I64, Z = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        cache, pages = ctypes.POINTER(B._CCache), ctypes.POINTER(B._CPages)
        L.pfkv_kv_evict_workspace_size.argtypes = [cache, pages, I32, I32, ctypes.POINTER(Z)]
        L.pfkv_kv_evict.argtypes = [cache, pages, pages, P_, I32, I32, P_, I64, I64, I32, I32, P_, Z,
                                    P_, P_, I64, I64, I32, P_, I64, I64, P_, P_]
        for name in EXPORTED:
            getattr(L, name).restype = ctypes.c_int
        L._evict_calls = True
    return L


def _rows(t: Optional[torch.Tensor], dtype, name: str, batch: int, heads: int, least: int):
    """(stride_b, stride_h, length) of rows [B][Hkv][length] with unit stride along tokens."""
    if t is None:
        return 0, 0, 0
    shape, stride = t.shape, t.stride()
    if (t.dtype is not dtype or len(shape) != 3 or shape[0] != batch or shape[1] != heads
            or shape[2] < least or (stride[2] != 1 and shape[2] > 1)):
        raise ValueError(f"{name}: {dtype} [B][Hkv][>= {least}] with unit stride along tokens")
    return stride[0], stride[1], shape[2]


def _lengths(t: torch.Tensor, pages: B.Pages, heads: int, name: str, dev: int):
    """Address of int32 numbers that lie as the lengths of `pages` do."""
    last = (pages.batch - 1) * pages.len_stride_b + (heads - 1) * pages.len_stride_h
    if not t.is_contiguous() or t.numel() <= last:
        spans = sum((n - 1) * s for n, s in zip(t.shape, t.stride())) if t.numel() else -1
        if pages.batch > 0 and spans < last:
            raise ValueError(f"{name}: int32, one at every place that the lengths of pages have")
    return R._i32(t, name, dev)


def pfkv_kv_evict_workspace_size(cache: B.Cache, pages: B.Pages, max_seq_len: int,
                                 max_keep_len: int) -> int:
    dev = R._current()
    c, p = P.cache_struct(cache, dev), P.pages_struct(pages, dev)
    n = ctypes.c_size_t(0)
    B._check(lib().pfkv_kv_evict_workspace_size(ctypes.byref(c), ctypes.byref(p), int(max_seq_len),
                                                int(max_keep_len), ctypes.byref(n)),
             "pfkv_kv_evict_workspace_size")
    return int(n.value)


def pfkv_kv_evict(cache: B.Cache, pages: B.Pages, new_pages: B.Pages, keep_lens: torch.Tensor,
                  attn_mass: torch.Tensor, max_seq_len: int, max_keep_len: int,
                  workspace: torch.Tensor, new_lens: torch.Tensor,
                  new_mass: Optional[torch.Tensor] = None, kept: Optional[torch.Tensor] = None,
                  keep_first: int = 0, keep_last: int = 0, flags: Optional[torch.Tensor] = None,
                  stream=None) -> None:
    """``pages``: the tokens as they are; ``new_pages``: the tables that receive the kept ones
    (its lengths are not read and may be None); keep_lens, new_lens: int32 with the length strides of ``pages``;
    attn_mass: float32 [B][Hkv][>= max_seq_len]; new_mass: float32 [B][Hkv][>= max_keep_len];
    kept: int32 [B][Hkv][>= max_keep_len]; workspace: uint8 of at least
    pfkv_kv_evict_workspace_size(...) bytes; flags uint8 [>= round_up(B, 4)]."""
    dev = R._current()
    heads = cache.k_pages.shape[1]
    ms = _rows(attn_mass, torch.float32, "attn_mass", pages.batch, heads, max_seq_len)
    ns = _rows(new_mass, torch.float32, "new_mass", pages.batch, heads, max_keep_len)
    ks = _rows(kept, torch.int32, "kept", pages.batch, heads, max_keep_len)
    if workspace.dtype is not torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace: contiguous uint8")
    kl = _lengths(keep_lens, pages, heads, "keep_lens", dev)
    nl = _lengths(new_lens, pages, heads, "new_lens", dev)
    c, p, x = P.cache_struct(cache, dev), P.pages_struct(pages, dev), P.pages_struct(new_pages, dev)
    B._check(lib().pfkv_kv_evict(
        ctypes.byref(c), ctypes.byref(p), ctypes.byref(x), kl,
        int(keep_first), int(keep_last), R._ptr(attn_mass, dev), ms[0], ms[1], int(max_seq_len),
        int(max_keep_len), R._ptr(workspace, dev), workspace.nbytes,
        nl, R._ptr(new_mass, dev), ns[0], ns[1], ns[2],
        R._ptr(kept, dev), ks[0], ks[1], R._ptr(flags, dev), R._stream(stream, dev)), "pfkv_kv_evict")
