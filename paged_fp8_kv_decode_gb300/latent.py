"""ctypes binding of the latent cache of libpfkv.so (argument marshalling only).

Every function has the name of the C entry point that it calls (see
``include/pfkv_latent.h`` for the full contract); tables, streams and errors are
those of ``binding``, rotations and row layouts those of ``rope``.
"""
from __future__ import annotations

import ctypes
import dataclasses
from typing import Optional

import torch

from . import binding as B
from . import rope as R

PFKV_LATENT_DIM = 512
PFKV_LATENT_ROPE = 64
PFKV_LATENT_NOPE = 128
PFKV_LATENT_VDIM = 128

# every symbol include/pfkv_latent.h declares
EXPORTED = ("pfkv_latent_append", "pfkv_latent_gather", "pfkv_latent_decode_workspace_size",
            "pfkv_latent_decode_attn", "pfkv_latent_prefill_attn", "pfkv_selftest_latent_decode",
            "pfkv_selftest_latent_prefill")


class _CLatentCache(ctypes.Structure):
    _fields_ = [("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("latent_dim", ctypes.c_int32), ("rope_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("c_pages", ctypes.c_void_p),
                ("r_pages", ctypes.c_void_p), ("c_scale", ctypes.c_void_p),
                ("page_tags", ctypes.c_void_p)]


@dataclasses.dataclass
class LatentCache:
    """The page pool (caller-owned CUDA tensors).

    c_pages: [num_pages][16][512], torch.bfloat16 or torch.uint8 (e4m3 codes);
    r_pages: bfloat16 [num_pages][16][64]; c_scale: float32 [num_pages] (FP8);
    page_tags: int32 (uint32 bit patterns) [num_pages] or None."""
    c_pages: torch.Tensor
    r_pages: torch.Tensor
    c_scale: Optional[torch.Tensor] = None
    page_tags: Optional[torch.Tensor] = None

    @property
    def dtype(self) -> int:
        return B.PFKV_KV_BF16 if self.c_pages.dtype == torch.bfloat16 else B.PFKV_KV_FP8_E4M3

    def c_struct(self, dev: Optional[int] = None) -> _CLatentCache:
        dev = R._current() if dev is None else dev
        c, r = self.c_pages, self.r_pages
        NP, PS, D = c.shape
        rNP, rPS, rD = r.shape
        if rNP != NP or rPS != PS or r.dtype != torch.bfloat16 or not r.is_contiguous():
            raise ValueError("c_pages [pages][16][512] and bfloat16 r_pages [pages][16][64], contiguous")
        R._pool(c, self.c_scale, self.page_tags, NP)
        return _CLatentCache(NP, PS, D, rD, self.dtype, R._ptr(c, dev), R._ptr(r, dev),
                             R._ptr(self.c_scale, dev), R._ptr(self.page_tags, dev))


def lib() -> ctypes.CDLL:
    """libpfkv.so with these calls' signatures set."""
    L = R.lib()
    if not getattr(L, "_latent_calls", False):
        P, I32, I64, F, Z = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                             ctypes.c_size_t)
        cache, pages, rows = (ctypes.POINTER(t) for t in (_CLatentCache, B._CPages, R._CRows))
        L.pfkv_latent_append.argtypes = [cache, pages, ctypes.POINTER(R._CRope),
                                         ctypes.POINTER(R._CNewTokens), rows, rows, rows, rows, I32,
                                         P, P]
        L.pfkv_latent_gather.argtypes = [cache, pages, P, I64, I32, P, I64, P, I64, P, P]
        L.pfkv_latent_decode_workspace_size.argtypes = [cache, pages, I32, I32, I32,
                                                        ctypes.POINTER(Z)]
        L.pfkv_latent_decode_attn.argtypes = [cache, pages, rows, rows, I32, I32, F, I32, P, Z,
                                              rows, P, P]
        L.pfkv_selftest_latent_decode.argtypes = [I32, *L.pfkv_latent_decode_attn.argtypes]
        L.pfkv_latent_prefill_attn.argtypes = [I32, I32, P, P, I64, I64, I32, rows, rows, rows,
                                               rows, rows, F, I32, rows, P, P]
        L.pfkv_selftest_latent_prefill.argtypes = [I32, *L.pfkv_latent_prefill_attn.argtypes]
        for name in EXPORTED:
            getattr(L, name).restype = ctypes.c_int
        L._latent_calls = True
    return L


def pfkv_latent_append(cache: LatentCache, pages: B.Pages, rope: R.Rope, positions: torch.Tensor,
                       c_new: torch.Tensor, r_new: torch.Tensor, q: Optional[torch.Tensor] = None,
                       q_out: Optional[torch.Tensor] = None,
                       new_lens: Optional[torch.Tensor] = None,
                       rope_positions: Optional[torch.Tensor] = None,
                       row_starts: Optional[torch.Tensor] = None,
                       max_new_tokens: Optional[int] = None, flags: Optional[torch.Tensor] = None,
                       stream=None) -> None:
    """c_new: bf16 [B][T][512], r_new: bf16 [B][T][64] (padded), or [rows][512]
    and [rows][64] with row_starts and max_new_tokens; q, q_out: bf16
    [B][T][H][64] or [rows][H][64]; the rest as in pfkv_rope_append."""
    dev = R._current()
    packed = row_starts is not None
    tok = R._new_tokens(c_new, pages.batch, positions, new_lens, rope_positions, row_starts,
                        max_new_tokens, dev)
    if c_new.shape[:-1] != r_new.shape[:-1]:
        raise ValueError("c_new and r_new: rows for the same tokens")
    c = R._rows(c_new, packed, False, "c_new", cache.c_pages.shape[2], dev)
    r = R._rows(r_new, packed, False, "r_new", cache.r_pages.shape[2], dev)
    qr, qo, hq = R._queries(q, q_out, c_new, packed, cache.r_pages.shape[2], dev)
    k, p, t = cache.c_struct(dev), R._pages(pages, dev), rope.c_struct(dev)
    B._check(lib().pfkv_latent_append(ctypes.byref(k), ctypes.byref(p), ctypes.byref(t),
                                      ctypes.byref(tok), ctypes.byref(c), ctypes.byref(r),
                                      R._ref(qr), R._ref(qo), hq, R._ptr(flags, dev),
                                      R._stream(stream, dev)), "pfkv_latent_append")


def pfkv_latent_gather(cache: LatentCache, pages: B.Pages, row_starts: torch.Tensor,
                       max_seq_len: int, c_out: torch.Tensor, r_out: torch.Tensor,
                       flags: Optional[torch.Tensor] = None, stream=None) -> None:
    """row_starts: int32 [B + 1]; c_out: bf16 [rows][512], r_out: bf16
    [rows][64], rows of any stride."""
    dev = R._current()
    c = R._rows(c_out, True, False, "c_out", cache.c_pages.shape[2], dev)
    r = R._rows(r_out, True, False, "r_out", cache.r_pages.shape[2], dev)
    if c_out.shape[0] != r_out.shape[0] or row_starts.numel() != pages.batch + 1:
        raise ValueError("as many rows of c_out as of r_out, and batch + 1 row_starts")
    k, p = cache.c_struct(dev), R._pages(pages, dev)
    B._check(lib().pfkv_latent_gather(ctypes.byref(k), ctypes.byref(p),
                                      R._i32(row_starts, "row_starts", dev), c_out.shape[0],
                                      int(max_seq_len), c.data, c.stride_t, r.data, r.stride_t,
                                      R._ptr(flags, dev), R._stream(stream, dev)),
             "pfkv_latent_gather")


def pfkv_latent_decode_workspace_size(cache: LatentCache, pages: B.Pages, num_q_heads: int,
                                      num_query_tokens: int, max_seq_len: int) -> int:
    dev = R._current()
    k, p = cache.c_struct(dev), R._pages(pages, dev)
    n = ctypes.c_size_t(0)
    B._check(lib().pfkv_latent_decode_workspace_size(ctypes.byref(k), ctypes.byref(p),
                                                     int(num_q_heads), int(num_query_tokens),
                                                     int(max_seq_len), ctypes.byref(n)),
             "pfkv_latent_decode_workspace_size")
    return int(n.value)


def pfkv_latent_decode_attn(cache: LatentCache, pages: B.Pages, q_c: torch.Tensor,
                            q_r: torch.Tensor, sm_scale: float, max_seq_len: int,
                            workspace: torch.Tensor, out: torch.Tensor,
                            flags: Optional[torch.Tensor] = None, stream=None) -> None:
    """q_c, out: bf16 [B][kq][H][512], q_r: bf16 [B][kq][H][64], any strides
    that leave rows contiguous: the last kq tokens of every request; workspace:
    uint8 of at least pfkv_latent_decode_workspace_size(...) bytes.  The pool is in
    device memory (tensor copies fetch it)."""
    _decode((), cache, pages, q_c, q_r, sm_scale, max_seq_len, workspace, out, flags, stream)


def pfkv_selftest_latent_decode(tries: int, *args, flags: Optional[torch.Tensor] = None,
                                stream=None) -> None:
    """pfkv_latent_decode_attn (whose positional arguments follow) with waits that give
    up after ``tries`` tries."""
    _decode((int(tries),), *args, flags, stream)


def _decode(tries, cache, pages, q_c, q_r, sm_scale, max_seq_len, workspace, out, flags,
            stream) -> None:
    if not (cache.c_pages.is_cuda and cache.r_pages.is_cuda):
        raise ValueError("a pool in device memory")
    if (q_c.shape != out.shape or q_c.shape[:-1] != q_r.shape[:-1]
            or q_c.shape[0] != pages.batch):
        raise ValueError("q_c and out [B][kq][H][512], q_r [B][kq][H][64]")
    dev = R._current()
    qc = R._rows(q_c, False, True, "q_c", cache.c_pages.shape[2], dev)
    qr = R._rows(q_r, False, True, "q_r", cache.r_pages.shape[2], dev)
    o = R._rows(out, False, True, "out", cache.c_pages.shape[2], dev)
    k, p = cache.c_struct(dev), R._pages(pages, dev)
    name = "pfkv_selftest_latent_decode" if tries else "pfkv_latent_decode_attn"
    B._check(getattr(lib(), name)(
        *tries, ctypes.byref(k), ctypes.byref(p), ctypes.byref(qc), ctypes.byref(qr), q_c.shape[2],
        q_c.shape[1], float(sm_scale), int(max_seq_len), R._ptr(workspace, dev),
        workspace.nbytes, ctypes.byref(o), R._ptr(flags, dev),
        R._stream(stream, dev)), name)


def pfkv_latent_prefill_attn(q_nope: torch.Tensor, q_rope: torch.Tensor, k_nope: torch.Tensor,
                             k_rope: torch.Tensor, v: torch.Tensor, q_starts: torch.Tensor,
                             k_starts: torch.Tensor, max_q_len: int, sm_scale: float, causal: bool,
                             out: torch.Tensor, flags: Optional[torch.Tensor] = None,
                             stream=None) -> None:
    """Packed rows: q_nope, out: bf16 [rows][H][128], q_rope: [rows][H][64],
    k_nope, v: [key rows][H][128], k_rope: [key rows][64]; q_starts, k_starts:
    int32 [B + 1]; any strides that leave rows contiguous; the rows in device memory."""
    _prefill((), q_nope, q_rope, k_nope, k_rope, v, q_starts, k_starts, max_q_len, sm_scale, causal,
             out, flags, stream)


def pfkv_selftest_latent_prefill(tries: int, *args, flags: Optional[torch.Tensor] = None,
                                 stream=None) -> None:
    """pfkv_latent_prefill_attn (whose positional arguments follow) with waits that
    give up after ``tries`` tries."""
    _prefill((int(tries),), *args, flags, stream)


def _prefill(tries, q_nope, q_rope, k_nope, k_rope, v, q_starts, k_starts, max_q_len, sm_scale,
             causal, out, flags, stream) -> None:
    (Tq, H), Tk = q_nope.shape[:2], k_nope.shape[0]
    if (q_nope.shape[:2] != q_rope.shape[:2] or q_nope.shape[:2] != out.shape[:2]
            or k_nope.shape[:2] != v.shape[:2] or k_nope.shape[1] != H or k_rope.shape[0] != Tk
            or q_starts.numel() != k_starts.numel() or q_starts.numel() < 1):
        raise ValueError("query rows [Tq][H], key rows [Tk][H], and batch + 1 starts of both")
    dev = R._current()
    if not (q_nope.is_cuda and q_rope.is_cuda and k_nope.is_cuda and k_rope.is_cuda and v.is_cuda):
        raise ValueError("rows in device memory")
    rows = [R._rows(t, True, h, n, d, dev) for t, h, n, d in (
        (q_nope, True, "q_nope", PFKV_LATENT_NOPE), (q_rope, True, "q_rope", PFKV_LATENT_ROPE),
        (k_nope, True, "k_nope", PFKV_LATENT_NOPE), (k_rope, False, "k_rope", PFKV_LATENT_ROPE),
        (v, True, "v", PFKV_LATENT_VDIM), (out, True, "out", PFKV_LATENT_VDIM))]
    name = "pfkv_selftest_latent_prefill" if tries else "pfkv_latent_prefill_attn"
    B._check(getattr(lib(), name)(
        *tries, int(q_starts.numel()) - 1, H, R._i32(q_starts, "q_starts", dev),
        R._i32(k_starts, "k_starts", dev),
        Tq, Tk, int(max_q_len), *[ctypes.byref(r) for r in rows[:5]], float(sm_scale),
        int(bool(causal)), ctypes.byref(rows[5]), R._ptr(flags, dev), R._stream(stream, dev)), name)
