"""ctypes binding of the attention over shared prefixes of libpfkv.so (argument
marshalling only).

Every function has the name of the C entry point that it calls (see
``include/pfkv_prefix.h`` for the full contract); caches, tables, streams and
errors are those of ``binding``, row layouts those of ``rope``.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import binding as B
from . import rope as R

PFKV_PREFIX_MAX = 4096

# every symbol include/pfkv_prefix.h declares
EXPORTED: tuple = ("pfkv_prefix_decode_workspace_size", "pfkv_prefix_decode_attn",
                   "pfkv_selftest_prefix_decode")


def lib() -> ctypes.CDLL:
    """libpfkv.so with these calls' signatures set."""
    L = R.lib()
    if not getattr(L, "_prefix_calls", False):
        P, I32, I64, F, Z = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                             ctypes.c_size_t)
        cache, pages, rows = (ctypes.POINTER(t) for t in (B._CCache, B._CPages, R._CRows))
        L.pfkv_prefix_decode_workspace_size.argtypes = [cache, pages, pages, I32, I32, I32, I32, I32,
                                                        I32, ctypes.POINTER(Z)]
        L.pfkv_prefix_decode_attn.argtypes = [cache, pages, pages, I32, P, rows, I32, I32, F, I32, I32,
                                              P, Z, rows, P, I64, I64, P, P]
        L.pfkv_selftest_prefix_decode.argtypes = [I32, *L.pfkv_prefix_decode_attn.argtypes]
        for name in EXPORTED:
            getattr(L, name).restype = ctypes.c_int
        L._prefix_calls = True
    return L


def cache_struct(cache: B.Cache, dev: int) -> B._CCache:
    """The pool of a call on device `dev`, its tensors checked."""
    k, v = cache.k_pages, cache.v_pages
    if v.shape != k.shape or v.dtype != k.dtype:
        raise ValueError("k_pages and v_pages: alike")
    NP, heads, PS, D = k.shape
    R._pool(k, cache.k_scale, cache.page_tags, NP * heads)
    R._pool(v, cache.v_scale, None, NP * heads)
    return B._CCache(NP, heads, PS, D, cache.dtype, R._ptr(k, dev), R._ptr(v, dev),
                     R._ptr(cache.k_scale, dev), R._ptr(cache.v_scale, dev),
                     R._ptr(cache.page_tags, dev))


def pages_struct(p: Optional[B.Pages], dev: int) -> Optional[B._CPages]:
    """A batch's tables of a call on device `dev`, their types checked (lengths may be None
    where a call does not read them)."""
    if p is None:
        return None
    if (p.block_tables.dtype is not torch.int32
            or p.seq_lens is not None and p.seq_lens.dtype is not torch.int32
            or p.expected_tags is not None and p.expected_tags.dtype not in R._TAGS):
        raise ValueError("block_tables, seq_lens and expected_tags: int32")
    return R._pages(p, dev)


def pfkv_prefix_decode_workspace_size(cache: B.Cache, pages: Optional[B.Pages], prefixes: B.Pages,
                                      batch: int, num_q_heads: int, num_query_tokens: int,
                                      max_seq_len: int, max_prefix_len: int,
                                      mass: bool = False) -> int:
    dev = R._current()
    c, p, x = cache_struct(cache, dev), pages_struct(pages, dev), pages_struct(prefixes, dev)
    n = ctypes.c_size_t(0)
    B._check(lib().pfkv_prefix_decode_workspace_size(ctypes.byref(c), R._ref(p), ctypes.byref(x),
                                                     int(batch), int(num_q_heads),
                                                     int(num_query_tokens), int(max_seq_len),
                                                     int(max_prefix_len), int(bool(mass)),
                                                     ctypes.byref(n)),
             "pfkv_prefix_decode_workspace_size")
    return int(n.value)


def pfkv_prefix_decode_attn(cache: B.Cache, pages: Optional[B.Pages], prefixes: B.Pages,
                            prefix_of: torch.Tensor, q: torch.Tensor, sm_scale: float,
                            max_seq_len: int, max_prefix_len: int, workspace: torch.Tensor,
                            out: torch.Tensor, attn_mass: Optional[torch.Tensor] = None,
                            flags: Optional[torch.Tensor] = None, stream=None) -> None:
    """q, out: bf16 [B][kq][Hq][D] of any strides that leave rows contiguous (out may be q);
    ``pages``: the requests' own tokens, or None; ``prefixes``: a Pages of the prefixes;
    prefix_of int32 [B] (-1: none); attn_mass: float32 [B][Hkv][>= max_seq_len], added to;
    workspace: uint8 of at least pfkv_prefix_decode_workspace_size(...) bytes; flags uint8
    [>= round_up(B, 4)].  The pool is in device memory."""
    _attn((), cache, pages, prefixes, prefix_of, q, sm_scale, max_seq_len, max_prefix_len, workspace, out,
          attn_mass, flags, stream)


def pfkv_selftest_prefix_decode(tries: int, *args, attn_mass: Optional[torch.Tensor] = None,
                                flags: Optional[torch.Tensor] = None, stream=None) -> None:
    """pfkv_prefix_decode_attn (whose positional arguments up to ``out`` follow) with waits that
    give up after ``tries`` tries."""
    _attn((int(tries),), *args, attn_mass, flags, stream)


def _attn(tries, cache, pages, prefixes, prefix_of, q, sm_scale, max_seq_len, max_prefix_len, workspace, out,
          attn_mass, flags, stream) -> None:
    dev = R._current()
    if q.dim() != 4 or q.shape != out.shape:
        raise ValueError("q and out: bfloat16 [B][kq][Hq][D]")
    if not (cache.k_pages.is_cuda and cache.v_pages.is_cuda):
        raise ValueError("a pool in device memory")
    if not workspace.is_contiguous():
        raise ValueError("workspace: contiguous")
    batch, kq, hq, D = q.shape
    if prefix_of.numel() != batch or not prefix_of.is_contiguous():
        raise ValueError("prefix_of: contiguous int32, one a request")
    rq, ro = (R._rows(t, False, True, n, cache.k_pages.shape[3], dev) for t, n in ((q, "q"), (out, "out")))
    c, p, x = cache_struct(cache, dev), pages_struct(pages, dev), pages_struct(prefixes, dev)
    sb = sh = 0
    if attn_mass is not None:
        if (attn_mass.dtype != torch.float32 or attn_mass.dim() != 3 or attn_mass.stride(2) != 1
                or attn_mass.shape[0] != batch or attn_mass.shape[1] != cache.k_pages.shape[1]
                or attn_mass.shape[2] < max_seq_len):
            raise ValueError("attn_mass: float32 [B][Hkv][>= max_seq_len] with unit stride along tokens")
        sb, sh = attn_mass.stride(0), attn_mass.stride(1)
    name = "pfkv_selftest_prefix_decode" if tries else "pfkv_prefix_decode_attn"
    B._check(getattr(lib(), name)(
        *tries, ctypes.byref(c), R._ref(p), ctypes.byref(x), batch, R._i32(prefix_of, "prefix_of", dev),
        ctypes.byref(rq), hq, kq, float(sm_scale), int(max_seq_len), int(max_prefix_len),
        R._ptr(workspace, dev), workspace.nbytes, ctypes.byref(ro), R._ptr(attn_mass, dev), sb, sh,
        R._ptr(flags, dev), R._stream(stream, dev)), name)
