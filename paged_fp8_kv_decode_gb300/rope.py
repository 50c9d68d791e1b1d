"""ctypes binding of the rotary append of libpfkv.so (argument marshalling only).

Every function has the name of the C entry point that it calls (see
``include/pfkv_rope.h`` for the full contract); caches, tables, streams and
errors are those of ``binding``.
"""
from __future__ import annotations

import ctypes
import dataclasses
from typing import Optional

import torch

from . import binding as B

# every symbol include/pfkv_rope.h declares
EXPORTED = ("pfkv_rope_append",)


class _CRope(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("scale", ctypes.c_float)]


class _CRows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride_b", ctypes.c_int64),
                ("stride_t", ctypes.c_int64), ("stride_h", ctypes.c_int64)]


class _CNewTokens(ctypes.Structure):
    _fields_ = [("num_new_tokens", ctypes.c_int32), ("positions", ctypes.c_void_p),
                ("new_lens", ctypes.c_void_p), ("rope_positions", ctypes.c_void_p),
                ("row_starts", ctypes.c_void_p), ("total_rows", ctypes.c_int64)]


@dataclasses.dataclass
class Rope:
    """The rotation: inv_freq float32 CUDA tensor [rot_dim / 2] (radians per
    position), pairs interleaved or half the rotated part apart, and a factor
    on the turned elements."""
    inv_freq: torch.Tensor
    interleaved: bool = False
    scale: float = 1.0

    def c_struct(self, dev: Optional[int] = None) -> _CRope:
        dev = _current() if dev is None else dev
        if self.inv_freq.dtype != torch.float32 or not self.inv_freq.is_contiguous():
            raise ValueError("inv_freq: contiguous float32")
        return _CRope(_ptr(self.inv_freq, dev), 2 * self.inv_freq.numel(), int(bool(self.interleaved)),
                      float(self.scale))


_BF16, _I32, _byref = torch.bfloat16, torch.int32, ctypes.byref


def _current() -> int:
    """The kernels run on the current device, whose stream `None` stands for: device
    memory of any argument of a call is that device's."""
    return torch.cuda.current_device() if torch.cuda.is_initialized() else -1


def _ptr(t, dev: int) -> Optional[int]:
    """binding._ptr of memory of device `dev` or of the host."""
    if t is None or t.__class__ is int:
        return t
    d = t.get_device()
    if d == dev and d >= 0:
        return t.data_ptr()
    if d >= 0:
        raise ValueError("tensors of another device than the current one")
    return B._ptr(t)


_CODES = (torch.uint8, torch.float8_e4m3fn)
_TAGS = (_I32, torch.uint32)


def _pool(pages: torch.Tensor, scale, tags, units: int) -> None:
    """One pool's tensors: bfloat16, or e4m3 codes with a float32 scale a unit; a tag a unit."""
    if pages.dtype != _BF16:
        if pages.dtype not in _CODES:
            raise ValueError("pages: bfloat16, or uint8 for e4m3 codes")
        if (scale is None or scale.dtype != torch.float32 or scale.numel() < units
                or not scale.is_contiguous()):
            raise ValueError("pages of e4m3 codes need a contiguous float32 scale each")
    if tags is not None and (tags.dtype not in _TAGS or tags.numel() < units
                             or not tags.is_contiguous()):
        raise ValueError("page_tags: contiguous int32, one each")
    if not pages.is_contiguous():
        raise ValueError("pages: contiguous")


def _stream(stream, dev: int) -> Optional[int]:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else B._stream(stream)


def _pages(p: B.Pages, dev: int) -> B._CPages:
    return B._CPages(p.batch, p.max_pages, _ptr(p.block_tables, dev), p.bt_stride_b, p.bt_stride_h,
                     _ptr(p.seq_lens, dev), p.len_stride_b, p.len_stride_h,
                     _ptr(p.expected_tags, dev))


def _rows(x: torch.Tensor, packed: bool, heads: bool, name: str, dim: int, dev: int) -> _CRows:
    """bf16 rows as the C ABI takes them: [B][T][H][D] padded or [rows][H][D]
    packed, without H where the rows are shared by all heads; any strides that
    leave a row's elements contiguous."""
    s = x.stride()
    want = 2 + (not packed) + heads
    if x.dtype != _BF16 or len(s) != want or s[-1] != 1:
        raise ValueError(f"{name}: bfloat16 tensor of {want} dimensions with contiguous rows")
    if x.size(-1) != dim:
        raise ValueError(f"{name}: rows of {dim} elements")
    p = _ptr(x, dev)
    if packed:
        return _CRows(p, 0, s[0], s[1] if heads else 0)
    return _CRows(p, s[0], s[1], s[2] if heads else 0)


def _i32(t: Optional[torch.Tensor], name: str, dev: int):
    if t is not None and t.dtype != _I32:
        raise ValueError(f"{name}: int32")
    return _ptr(t, dev)


def _new_tokens(first: torch.Tensor, batch: int, positions, new_lens, rope_positions, row_starts,
                max_new_tokens, dev: int) -> _CNewTokens:
    """`first`: the tensor of new rows that gives T or the number of rows."""
    if row_starts is None:
        if first.shape[0] != batch:
            raise ValueError("padded rows: one entry per request")
        T, total = first.shape[1], 0
        if max_new_tokens is not None and int(max_new_tokens) != T:
            raise ValueError("padded rows: max_new_tokens is their second dimension")
    else:
        if max_new_tokens is None:
            raise ValueError("packed rows need max_new_tokens")
        if row_starts.numel() != batch + 1:
            raise ValueError("row_starts: batch + 1 entries")
        T, total = int(max_new_tokens), first.shape[0]
    return _CNewTokens(T, _i32(positions, "positions", dev), _i32(new_lens, "new_lens", dev),
                       _i32(rope_positions, "rope_positions", dev),
                       _i32(row_starts, "row_starts", dev), total)


def _queries(q, q_out, first, packed, dim, dev):
    """(q rows, q_out rows, heads), or three empty ones without queries."""
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out: both or neither")
    if q is None:
        return None, None, 0
    lead = 1 if packed else 2
    if q.shape != q_out.shape or q.shape[:lead] != first.shape[:lead]:
        raise ValueError("q and q_out: rows for the same tokens as the new keys")
    return (_rows(q, packed, True, "q", dim, dev), _rows(q_out, packed, True, "q_out", dim, dev),
            q.shape[-2])


def _ref(s):
    return None if s is None else _byref(s)


def lib() -> ctypes.CDLL:
    """libpfkv.so with these calls' signatures set."""
    L = B.lib()
    if not getattr(L, "_rope_calls", False):
        P, I32 = ctypes.c_void_p, ctypes.c_int32
        rows = ctypes.POINTER(_CRows)
        L.pfkv_rope_append.argtypes = [ctypes.POINTER(B._CCache), ctypes.POINTER(B._CPages),
                                       ctypes.POINTER(_CRope), ctypes.POINTER(_CNewTokens), rows,
                                       rows, rows, rows, I32, P, P]
        L.pfkv_rope_append.restype = ctypes.c_int
        L._rope_calls = True
    return L


def pfkv_rope_append(cache: B.Cache, pages: B.Pages, rope: Rope, positions: torch.Tensor,
                     k_new: torch.Tensor, v_new: torch.Tensor, q: Optional[torch.Tensor] = None,
                     q_out: Optional[torch.Tensor] = None,
                     new_lens: Optional[torch.Tensor] = None,
                     rope_positions: Optional[torch.Tensor] = None,
                     row_starts: Optional[torch.Tensor] = None,
                     max_new_tokens: Optional[int] = None, flags: Optional[torch.Tensor] = None,
                     stream=None) -> None:
    """k_new, v_new: bf16 [B][T][Hkv][D] (padded), or [rows][Hkv][D] with
    row_starts (int32 [B + 1]) and max_new_tokens; q, q_out the same with the
    query heads (q_out may be q); positions, new_lens int32 with the length
    strides of ``pages``, rope_positions int32 [B]; flags uint8
    [>= round_up(B, 4)] (OR-ed)."""
    dev = _current()
    packed = row_starts is not None
    NP, heads, PS, D = cache.k_pages.shape
    if cache.v_pages.shape != cache.k_pages.shape or cache.v_pages.dtype != cache.k_pages.dtype:
        raise ValueError("k_pages and v_pages: alike")
    _pool(cache.k_pages, cache.k_scale, cache.page_tags, NP * heads)
    _pool(cache.v_pages, cache.v_scale, None, NP * heads)
    tok = _new_tokens(k_new, pages.batch, positions, new_lens, rope_positions, row_starts,
                      max_new_tokens, dev)
    if k_new.shape != v_new.shape or k_new.shape[-2] != heads:
        raise ValueError("k_new and v_new: one row per kv head")
    k = _rows(k_new, packed, True, "k_new", D, dev)
    v = _rows(v_new, packed, True, "v_new", D, dev)
    qr, qo, hq = _queries(q, q_out, k_new, packed, D, dev)
    c = B._CCache(NP, heads, PS, D, cache.dtype, _ptr(cache.k_pages, dev), _ptr(cache.v_pages, dev),
                  _ptr(cache.k_scale, dev), _ptr(cache.v_scale, dev), _ptr(cache.page_tags, dev))
    p, r = _pages(pages, dev), rope.c_struct(dev)
    B._check(lib().pfkv_rope_append(_byref(c), _byref(p), _byref(r),
                                    _byref(tok), _byref(k), _byref(v), _ref(qr),
                                    _ref(qo), hq, _ptr(flags, dev), _stream(stream, dev)),
             "pfkv_rope_append")
