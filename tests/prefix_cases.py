"""Inputs and 64-bit references of the attention over shared prefixes and of the
eviction, shared by their GPU tests.  The references are written from the
definitions, head by head, without the library.

Pools are filled with NaN (values and scales) wherever no live token lies, tables
with an id outside the pool wherever no live page does."""
import math

import torch

from latent_cases import BF16, F16, PAGE, close, gen, i32, rows, score_error, softmax_attend
from paged_fp8_kv_decode_gb300 import binding as B
from paged_fp8_kv_decode_gb300 import evict as E
from paged_fp8_kv_decode_gb300 import prefix as P


def pages_of(n):
    return (n + PAGE - 1) // PAGE


def per_head(lens, H):
    """Lengths as lists of one number a head."""
    return [list(x) if isinstance(x, (list, tuple)) else [x] * H for x in lens]


class Pool:
    """A pool of `num` pages for heads H of D elements."""

    def __init__(self, num, H, D, fp8, tags=False, seed=0):
        self.H, self.D, self.fp8, self.g = H, D, fp8, gen(seed)
        self.free = torch.randperm(num, generator=torch.Generator().manual_seed(seed)).tolist()
        shape = (num, H, PAGE, D)
        if fp8:
            k, v = (torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
            ks, vs = (torch.full(shape[:2], math.nan, device="cuda") for _ in range(2))
        else:
            k, v = (torch.full(shape, math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2))
            ks = vs = None
        t = None
        if tags:
            t = torch.randint(-2 ** 31, 2 ** 31 - 1, shape[:2], generator=self.g, device="cuda", dtype=torch.int32)
        self.cache = B.Cache(k, v, ks, vs, t)

    def tables(self, lens, heads_apart=False, fill=True, lens_apart=None, wide=0):
        """A Pages whose row i holds lens[i] tokens (a number, or one a head; heads that share a
        table take pages for the longest), filled with random keys and values."""
        H = self.H
        lens = per_head(lens, H)
        most = max(1, max([pages_of(n) for r in lens for n in r], default=1)) + wide
        T = H if heads_apart else 1
        bt = torch.full((len(lens), T, most), -7, dtype=torch.int32)
        for i, r in enumerate(lens):
            for t in range(T):
                for p in range(pages_of(r[t] if heads_apart else max(r))):
                    bt[i, t, p] = self.free.pop()
        bt = bt.cuda()
        apart = any(len(set(r)) > 1 for r in lens) if lens_apart is None else lens_apart
        n = i32(lens if apart else [r[:1] for r in lens]).reshape(len(lens), -1)
        want = None
        if self.cache.page_tags is not None:
            want = self.cache.page_tags[bt.long().clamp(min=0), torch.arange(T, device="cuda")[None, :, None]].contiguous()
            if not heads_apart:  # one tag a page for all heads
                ids = bt[bt >= 0].long()
                self.cache.page_tags[ids] = self.cache.page_tags[ids][:, :1].expand(-1, H).contiguous()
        pages = B.Pages(len(lens), most, bt, bt.stride(0), bt.stride(1) if heads_apart else 0, n, n.shape[1],
                        1 if apart else 0, want)
        pages.lens = lens
        if fill:
            self.fill(pages)
        return pages

    def fill(self, pages):
        c, D = self.cache, self.D
        for i, r in enumerate(pages.lens):
            for h, n in enumerate(r):
                ids = self.row(pages, i, h)[:pages_of(n)]
                for pool, scale in ((c.k_pages, c.k_scale), (c.v_pages, c.v_scale)):
                    if n == 0:
                        continue
                    if self.fp8:
                        x = torch.randn(n, D, generator=self.g, device="cuda") * 100
                        x = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                        scale[ids, h] = torch.exp(torch.randn(len(ids), generator=self.g, device="cuda") * 0.3 - 4.6)
                    else:
                        x = rows(self.g, n, D)
                    j = torch.arange(n, device="cuda")
                    pool[ids[j // PAGE], h, j % PAGE] = x

    @staticmethod
    def row(pages, i, h):
        bt = pages.block_tables
        return bt[i, h if bt.shape[1] > 1 else 0].long()

    def values(self, pages, i, h, n, which):
        """The first n tokens of row i and head h in 64 bits: [n, D]."""
        pool, scale = getattr(self.cache, which + "_pages"), getattr(self.cache, which + "_scale")
        ids = self.row(pages, i, h)[:pages_of(n)]
        x = pool[ids, h]
        if self.fp8:
            x = x.view(torch.float8_e4m3fn).double() * scale[ids, h].double()[:, None, None]
        return x.double().reshape(-1, self.D)[:n]


def attend(pool, own, pre, of, q, scale, mass=None):
    """What the call has to give: (out, tolerance, mass or None, its tolerance)."""
    Bn, kq, Hq, D = q.shape
    H = pool.H
    G = Hq // H
    out, tol = torch.zeros(q.shape, dtype=torch.float64, device="cuda"), torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    m_out = None if mass is None else mass.double().clone()
    m_tol = None if mass is None else mass.double().abs() * 2.0 ** -24
    for b in range(Bn):
        for h in range(H):
            n = own.lens[b][h] if own else 0
            N = pre.lens[of[b]][h] if of[b] >= 0 else 0
            k = [pool.values(own, b, h, n, "k")] if own else []
            v = [pool.values(own, b, h, n, "v")] if own else []
            if of[b] >= 0:
                k, v = [pool.values(pre, of[b], h, N, "k")] + k, [pool.values(pre, of[b], h, N, "v")] + v
            if not k:
                continue
            k, v = torch.cat(k), torch.cat(v)
            for t in range(kq):
                seen = N + (max(0, n - kq + 1 + t) if own else 0)
                if seen == 0:
                    continue
                heads = slice(h * G, (h + 1) * G)
                qq, kk, vv = q[b, t, heads].double(), k[:seen], v[:seen]
                s = qq @ kk.T * scale
                err = score_error(qq, kk, scale)
                if pool.fp8:  # a query's pair of e4m3 values: 2^-17 of the row's largest
                    err = err + 2.0 ** -17 * qq.abs().amax(-1) * kk.abs().sum(-1).amax() * abs(scale)
                o, e = softmax_attend(s, vv, F16 if pool.fp8 else BF16, err)
                out[b, t, heads], tol[b, t, heads] = o, e + seen * 2.0 ** -31 * vv.abs().amax()
                if mass is not None:
                    w = torch.softmax(s, -1)[:, N:]
                    m_out[b, h, :n] += w.sum(0)
                    # scores' errors, the exponential's (2^-21 of the weight) and the logarithm of the sum's
                    # (2^-20 of its size, at most 40), and the total's rounding
                    m_tol[b, h, :n] += (w * (2 * err[:, None] + 40 * 2.0 ** -20)).sum(0) + w.sum(0) * 2.0 ** -22
    return out, tol, m_out, m_tol


def call(pool, own, pre, of, q, scale, out=None, mass=None, flags=None, max_len=None, max_pre=None, ws=None, stream=None,
         guard=True):
    """The library's call; returns (out, flags)."""
    Bn, kq, Hq, _ = q.shape
    most = lambda p: max((n for r in p.lens for n in r), default=0) if p and p.batch else 0  # noqa: E731
    max_len = most(own) if max_len is None else max_len
    max_pre = most(pre) if max_pre is None else max_pre
    if ws is None:
        n = P.pfkv_prefix_decode_workspace_size(pool.cache, own, pre, Bn, Hq, kq, max_len, max_pre, mass=mass is not None)
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, math.nan) if out is None else out
    flags = torch.full(((Bn + 3) // 4 * 4,), 0xAA, dtype=torch.uint8, device="cuda") if flags is None else flags
    P.pfkv_prefix_decode_attn(pool.cache, own, pre, of if torch.is_tensor(of) else i32(of), q, scale, max_len, max_pre, ws, out,
                              attn_mass=mass, flags=flags, stream=stream)
    return out, flags


def no_prefixes(H):
    p = B.Pages(0, 1, i32([[0]]), 1, 0, i32([0]), 1, 0)
    p.lens = []
    return p


def evict_call(pool, src, dst, keep, mass, first, last, room=None, kept=True, max_len=None, max_keep=None, stream=None,
               new_lens=None):
    """The library's call; keep: int32 with src's lengths' shape.  Returns (new_lens, new_mass, kept, flags)."""
    Bn, H = src.batch, pool.H
    n = max((x for r in src.lens for x in r), default=0) if max_len is None else max_len
    k = int(keep.max()) if max_keep is None else max_keep
    room = k + 9 if room is None else room
    ws = torch.full((E.pfkv_kv_evict_workspace_size(pool.cache, src, n, k),), 0xFF, dtype=torch.uint8, device="cuda")
    new_lens = torch.full_like(src.seq_lens, -5) if new_lens is None else new_lens
    new_mass = torch.full((Bn, H, room), math.nan, device="cuda")
    kept = torch.full((Bn, H, k), -3, dtype=torch.int32, device="cuda") if kept else None
    flags = torch.full(((Bn + 3) // 4 * 4,), 0xAA, dtype=torch.uint8, device="cuda")
    E.pfkv_kv_evict(pool.cache, src, dst, keep, mass, n, k, ws, new_lens, new_mass=new_mass, kept=kept, keep_first=first,
                    keep_last=last, flags=flags, stream=stream)
    return new_lens, new_mass, kept, flags


def kept_ids(mass, n, k, first, last):
    """Old indices of the tokens that one head keeps, in order (a list)."""
    k = min(k, n)
    f = min(first, k)
    z = min(last, k - f)
    x = mass[f:n - z].double().cpu()
    x = torch.where(torch.isnan(x), torch.full_like(x, math.inf), x)
    nan = torch.isnan(mass[f:n - z].cpu())
    order = sorted(range(len(x)), key=lambda j: (not bool(nan[j]), -float(x[j]), j))[:k - f - z]
    return list(range(f)) + sorted(j + f for j in order) + list(range(n - z, n))


__all__ = ["B", "BF16", "E", "F16", "P", "PAGE", "Pool", "attend", "call", "close", "evict_call", "gen", "i32", "kept_ids",
           "no_prefixes", "pages_of", "per_head", "rows"]
