"""Inputs and 64-bit references of the rotary append and of the latent cache's
calls, shared by their GPU tests.  The references are written from the
definitions, request by request, without the library."""
import math

import torch

from paged_fp8_kv_decode_gb300 import binding as B
from paged_fp8_kv_decode_gb300 import latent as L

PAGE = 16
# half a rounding step, relative to the value
BF16, F16, E4M3 = 2.0 ** -8, 2.0 ** -11, 2.0 ** -4
# fp32 rotation: sincospif within 2 ulp, the angle within 2^-25 of a half turn,
# two products and a sum, each within 2^-24: below 2^-20 (|a| + |b|) together
TURN = 2.0 ** -20


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rows(g, *shape, outliers=0.01):
    x = torch.randn(*shape, generator=g, device="cuda")
    if outliers:
        x = torch.where(torch.rand(*shape, generator=g, device="cuda") < outliers, x * 20, x)
    return x.to(torch.bfloat16)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def flags_for(batch):
    return torch.zeros((batch + 3) // 4 * 4 + 4, dtype=torch.uint8, device="cuda")


def tables(last, seed=0, spare=5, first=None):
    """Shuffled pages for every request's pages first[b] .. last[b] - 1."""
    first = first or [0] * len(last)
    need = sum(b - a for a, b in zip(first, last))
    perm = torch.randperm(need + spare, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    mp = max(1, max(last))
    bt = torch.full((len(last), mp), -7, dtype=torch.int32)
    at = 0
    for b, (x, y) in enumerate(zip(first, last)):
        bt[b, x:y] = perm[at:at + y - x]
        at += y - x
    return bt.cuda(), need + spare


def pages(bt, lens, tags=None, expected=None):
    return B.Pages(bt.shape[0], bt.shape[1], bt, bt.stride(0), 0, lens, 1, 0, expected)


def turned(x, pos, inv_freq, interleaved, scale=1.0):
    """x [tokens, heads, dim] in 64 bits, turned by pos * inv_freq; and |a| + |b|
    of each element's pair (what its rounding errors are relative to)."""
    x = x.double().clone()
    size = torch.zeros_like(x)
    h = inv_freq.numel()
    a = (pos.double()[:, None] * inv_freq.double())[:, None]
    re, im = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else (slice(0, h), slice(h, 2 * h))
    u, v = x[..., re].clone(), x[..., im].clone()
    x[..., re] = scale * (u * a.cos() - v * a.sin())
    x[..., im] = scale * (v * a.cos() + u * a.sin())
    size[..., re] = size[..., im] = abs(scale) * (u.abs() + v.abs())
    return x, size


def close(got, want, tol, what):
    got = got.double()
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4].tolist(), want[bad][:4].tolist(),
                           torch.broadcast_to(torch.as_tensor(tol), want.shape).to(want.device)[bad][:4].tolist())


def latent_pool(g, num_pages, fp8, tags=False, fill=None):
    """A pool of random latents (or of bytes `fill` everywhere)."""
    if fp8:
        x = torch.randn(num_pages, PAGE, 512, generator=g, device="cuda") * 100
        c = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        z = torch.exp(torch.randn(num_pages, generator=g, device="cuda") * 0.3 - 4.6)
    else:
        c, z = rows(g, num_pages, PAGE, 512), None
    r = rows(g, num_pages, PAGE, 64, outliers=0)
    t = torch.randint(-2 ** 31, 2 ** 31 - 1, (num_pages,), generator=g, device="cuda", dtype=torch.int32) if tags else None
    if fill is not None:
        c.view(torch.uint8).fill_(fill)
        r.view(torch.uint8).fill_(fill)
    return L.LatentCache(c, r, z, t)


def latent_values(cache, table_row, n):
    """Latents and rotated keys of a request's first n tokens, in 64 bits."""
    pg = table_row[:(n + PAGE - 1) // PAGE].long()
    c = cache.c_pages[pg]
    if c.dtype == torch.uint8:
        c = c.view(torch.float8_e4m3fn).double() * cache.c_scale[pg].double()[:, None, None]
    return c.double().reshape(-1, 512)[:n], cache.r_pages[pg].double().reshape(-1, 64)[:n]


def softmax_attend(s, v, weight_step, score_err, out_step=BF16):
    """Attention of scores s [rows, tokens] (-inf where hidden; a row of them
    gives zero) over v [tokens, dim]; and how far a result may be off when each
    weight is rounded once by weight_step (relative), the scores are off by
    score_err (absolute, per row) and the output by out_step.

    With w_j = p_j (1 + e_j), |e_j| <= e = weight_step + 2 score_err + 2^-20 (the
    exponential), and the sum taken of the same w: |sum w v / sum w - o| <=
    e (sum p |v| + |o|) / (1 - e)."""
    empty = torch.isinf(s).all(-1, keepdim=True)
    p = torch.softmax(torch.where(empty, 0.0, s), -1)
    p = torch.where(empty, 0.0, p)
    o = p @ v
    e = weight_step + 2 * score_err + 2.0 ** -20
    if torch.is_tensor(e):
        e = e[:, None]
    spread = p @ v.abs() + o.abs()
    return o, e / (1 - e) * spread + out_step * o.abs() + 1e-30


def score_error(q, k, scale):
    """fp32 accumulation of products: 2^-24 a step of a tree at most 40 deep,
    relative to the sum of magnitudes; largest over the tokens, per row."""
    return (q.abs() @ k.abs().T).amax(-1) * abs(scale) * 40 * 2.0 ** -24


SCALE = 1.0 / math.sqrt(192)
