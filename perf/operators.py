"""Cases, plain forms and exact values of the rotary-append and latent-attention operators.

Five operators that a serving program calls around a paged cache:

  rope_append     rotate q and k by position, write k and v into page slots (FP8 or BF16 pool)
  latent_append   the same for a cache of one latent vector and one rotated key a token
  latent_gather   pages of a latent cache -> contiguous bf16 rows, the input of the up-projection
  latent_decode   attention of single tokens (or a few candidates) in the absorbed form over that cache
  latent_prefill  ragged causal attention of prompts in the expanded form

``run`` computes them with elementary torch operations in 32 bits while ``own`` is
false, and through the library's entry points while it is true.
"""
import math
import random

import torch

own = False

PAGE = 16
LATENT, ROPE = 512, 64          # values of a latent vector and of its rotated key
NOPE, VDIM = 128, 128           # expanded head: unrotated part of q and k, and v


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decode step of a 32-query-head, 8-kv-head layer, FP8 pool (the benchmark's layer)
        dict(name="rope step fp8", op="rope_append", B=32, T=1, packed=False, Hq=32, Hkv=8, D=128, fp8=True,
             rot=128, inter=False, ctx_lo=512, ctx_hi=8192),
        # prompts of ragged lengths, packed, entering an FP8 pool
        dict(name="rope prompts fp8", op="rope_append", B=6, T=4096, packed=True, Hq=32, Hkv=8, D=128, fp8=True,
             rot=128, inter=False, ctx_lo=0, ctx_hi=200),
        # candidates of a verification step far into long contexts, BF16 pool, half of the head rotated
        dict(name="rope verify bf16", op="rope_append", B=24, T=5, packed=False, Hq=8, Hkv=2, D=64, fp8=False,
             rot=32, inter=True, ctx_lo=100000, ctx_hi=500000),
        # one decode step of a 128-head latent layer
        dict(name="latent step fp8", op="latent_append", B=64, T=1, packed=False, H=128, fp8=True, inter=True,
             ctx_lo=512, ctx_hi=8192),
        # ragged prompts entering a latent pool, 16 heads (one of eight shards)
        dict(name="latent prompts bf16", op="latent_append", B=7, T=2048, packed=True, H=16, fp8=False, inter=True,
             ctx_lo=0, ctx_hi=100),
        # cached prefixes read back for the expanded form
        dict(name="gather fp8", op="latent_gather", B=8, n_lo=1000, n_hi=16384, fp8=True),
        dict(name="gather short bf16", op="latent_gather", B=3, n_lo=1, n_hi=300, fp8=False),
        # a single conversation, 16 heads: latency
        dict(name="decode one bf16", op="latent_decode", B=1, kq=1, H=16, n_lo=1000, n_hi=1000, fp8=False),
        # a full batch, all 128 heads, FP8
        dict(name="decode batch fp8", op="latent_decode", B=32, kq=1, H=128, n_lo=512, n_hi=8192, fp8=True),
        # verification of two candidates over long contexts
        dict(name="decode verify bf16", op="latent_decode", B=4, kq=2, H=64, n_lo=16384, n_hi=65536, fp8=False),
        # ragged short prompts, some of them with a cached prefix
        dict(name="prefill ragged", op="latent_prefill", B=5, H=16, q_lo=1, q_hi=777, pre_hi=333),
        # one long prompt, all 128 heads
        dict(name="prefill long", op="latent_prefill", B=1, H=128, q_lo=4096, q_hi=4096, pre_hi=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope_append", "latent_append", "latent_gather", "latent_decode", "latent_decode",
                     "latent_prefill"])
    fp8 = rng.random() < 0.5
    if op in ("rope_append", "latent_append"):
        packed = rng.random() < 0.5
        B, T = _log(rng, 1, 96), _log(rng, 1, 8)
        if packed:
            T = _log(rng, 20, 4096)
            B = min(rng.randint(1, 12), max(1, 20000 // T))
        lo = rng.choice([0, 0, _log(rng, 1, 200000)])
        hi = lo + _log(rng, 1, 8000)
        if op == "latent_append":
            return dict(op=op, B=B, T=T, packed=packed, H=rng.choice([1, 5, 8, 16, 32, 64, 128]), fp8=fp8,
                        inter=rng.random() < 0.7, ctx_lo=lo, ctx_hi=hi)
        D = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        return dict(op=op, B=B, T=T, packed=packed, Hq=Hkv * rng.choice([1, 2, 4, 8]), Hkv=Hkv, D=D, fp8=fp8,
                    rot=rng.choice([D, D, D // 2]), inter=rng.random() < 0.5, ctx_lo=lo, ctx_hi=hi)
    if op == "latent_gather":
        hi = _log(rng, 1, 16384)
        return dict(op=op, B=rng.randint(1, 8), n_lo=rng.randint(0, hi), n_hi=hi, fp8=fp8)
    if op == "latent_decode":
        H, kq = rng.choice([1, 8, 16, 20, 32, 64, 128]), rng.choice([1, 1, 1, 2, 3, 4])
        hi = _log(rng, 10, 60000)
        B = min(_log(rng, 1, 48), max(1, 200000 // hi), max(1, 9000000 // (hi * H * kq) * 4))
        return dict(op=op, B=B, kq=kq, H=H, n_lo=rng.randint(1, hi), n_hi=hi, fp8=fp8)
    H = rng.choice([1, 8, 16, 32, 128])
    hi = _log(rng, 10, 4096)
    B = max(1, min(rng.randint(1, 8), 2 ** 31 // (hi * (hi + hi // 4) * H)))
    return dict(op=op, B=B, H=H, q_lo=rng.randint(1, hi), q_hi=hi, pre_hi=rng.choice([0, hi // 4]) if B > 1 else 0)


def _lens(lo, hi, B, salt=0):
    """B lengths in [lo, hi], the same for every seed (the outputs' shapes go by them)."""
    r = random.Random(lo * 1000003 + hi * 101 + B * 7 + salt)
    v = [r.randint(lo, hi) for _ in range(B)]
    v[0] = hi
    return v


def _starts(v):
    s = [0]
    for x in v:
        s.append(s[-1] + x)
    return s


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows(g, *shape, outliers=True):
    """N(0, 1), one value in a hundred 20 times as large: the values of keys and latents."""
    x = torch.randn(*shape, generator=g, device="cuda")
    if outliers:
        x = torch.where(torch.rand(*shape, generator=g, device="cuda") < 0.01, x * 20, x)
    return x.to(torch.bfloat16)


def _codes(g, *shape):
    """e4m3 codes of N(0, 100^2) values, as a page whose largest value is near 448 holds them."""
    x = torch.randn(*shape, generator=g, device="cuda") * 100
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _scales(g, *shape):
    return torch.exp(torch.randn(*shape, generator=g, device="cuda") * 0.3 - 4.6)


def _tables(seed, first, last, spare=8):
    """Tables that map pages first[b]..last[b]-1 of each request to shuffled pages; (table, pages in the pool)."""
    need = sum(b - a for a, b in zip(first, last))
    perm = torch.randperm(need + spare, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    mp = max(1, max(last))
    bt = torch.full((len(last), mp), -1, dtype=torch.int32)
    at = 0
    for b, (x, y) in enumerate(zip(first, last)):
        bt[b, x:y] = perm[at:at + y - x]
        at += y - x
    return bt.cuda(), need + spare


def _append_state(case, seed):
    B, T = case["B"], case["T"]
    n = _lens(max(1, T // 8), T, B) if case["packed"] else [T] * B
    ctx = _lens(case["ctx_lo"], case["ctx_hi"], B, salt=1)
    first = [c // PAGE for c in ctx]
    last = [(c + k - 1) // PAGE + 1 for c, k in zip(ctx, n)]
    bt, pages = _tables(seed, first, last)
    s = dict(case=case, positions=_i32(ctx), bt=bt, pages=pages, seq_lens=_i32([c + k for c, k in zip(ctx, n)]),
             T=T, B=B, R=sum(n), starts=_i32(_starts(n)) if case["packed"] else None,
             flags=torch.zeros((B + 3) // 4 * 4, dtype=torch.uint8, device="cuda"))
    rot = case["rot"] if case["op"] == "rope_append" else ROPE
    s["inv_freq"] = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()
    return s


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "rope_append":
        s = _append_state(case, seed)
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        lead = (s["R"],) if case["packed"] else (s["B"], s["T"])
        s["q"] = _rows(g, *lead, Hq, D, outliers=False)
        s["k"], s["v"] = _rows(g, *lead, Hkv, D), _rows(g, *lead, Hkv, D)
        s["q_out"] = torch.zeros_like(s["q"])
        shape = (s["pages"], Hkv, PAGE, D)
        if case["fp8"]:
            s["k_pages"], s["v_pages"] = _codes(g, *shape), _codes(g, *shape)
            s["k_scale"], s["v_scale"] = _scales(g, *shape[:2]), _scales(g, *shape[:2])
        else:
            s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"] = _rows(g, *shape), _rows(g, *shape), None, None
        return s
    if op == "latent_append":
        s = _append_state(case, seed)
        lead = (s["R"],) if case["packed"] else (s["B"], s["T"])
        s["q"] = _rows(g, *lead, case["H"], ROPE, outliers=False)
        s["c"], s["r"] = _rows(g, *lead, LATENT), _rows(g, *lead, ROPE, outliers=False)
        s["q_out"] = torch.zeros_like(s["q"])
        _latent_pool(s, g, s["pages"], case["fp8"])
        return s
    if op in ("latent_gather", "latent_decode"):
        n = _lens(case["n_lo"], case["n_hi"], case["B"])
        bt, pages = _tables(seed, [0] * case["B"], [(k + PAGE - 1) // PAGE for k in n])
        s = dict(case=case, bt=bt, seq_lens=_i32(n), R=sum(n), B=case["B"], max_len=max(n),
                 flags=torch.zeros((case["B"] + 3) // 4 * 4, dtype=torch.uint8, device="cuda"))
        _latent_pool(s, g, pages, case["fp8"])
        if op == "latent_gather":
            s["starts"] = _i32(_starts(n))
            s["c_out"] = torch.empty(sum(n), LATENT, dtype=torch.bfloat16, device="cuda")
            s["r_out"] = torch.empty(sum(n), ROPE, dtype=torch.bfloat16, device="cuda")
        else:
            lead = (case["B"], case["kq"], case["H"])
            # scores of a few units, as trained heads give: some tokens stand out, none alone
            s["q_c"] = _rows(g, *lead, LATENT, outliers=False)
            s["q_r"] = _rows(g, *lead, ROPE, outliers=False)
            s["scale"] = 1.0 / math.sqrt(NOPE + ROPE)
            s["out"] = torch.empty(*lead, LATENT, dtype=torch.bfloat16, device="cuda")
        return s
    # latent_prefill: packed rows; k_nope and v are the two halves of each head's row of the
    # up-projection's result, as a program has them
    B, H = case["B"], case["H"]
    nq = _lens(case["q_lo"], case["q_hi"], B)
    nk = [a + p for a, p in zip(nq, _lens(0, case["pre_hi"], B, salt=2))]
    kv = _rows(g, sum(nk), H, NOPE + VDIM, outliers=False)
    return dict(case=case, B=B, H=H, nq=max(nq), nk=max(nk), q_starts=_i32(_starts(nq)), k_starts=_i32(_starts(nk)),
                q_nope=_rows(g, sum(nq), H, NOPE, outliers=False), q_rope=_rows(g, sum(nq), H, ROPE, outliers=False),
                k_rope=_rows(g, sum(nk), ROPE, outliers=False), k_nope=kv[..., :NOPE], v=kv[..., NOPE:],
                scale=1.0 / math.sqrt(NOPE + ROPE),
                out=torch.empty(sum(nq), H, VDIM, dtype=torch.bfloat16, device="cuda"),
                flags=torch.zeros((B + 3) // 4 * 4, dtype=torch.uint8, device="cuda"))


def _latent_pool(s, g, pages, fp8):
    s["c_pages"] = _codes(g, pages, PAGE, LATENT) if fp8 else _rows(g, pages, PAGE, LATENT)
    s["c_scale"] = _scales(g, pages) if fp8 else None
    s["r_pages"] = _rows(g, pages, PAGE, ROPE, outliers=False)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return {"rope_append": _own_rope, "latent_append": _own_latent_append, "latent_gather": _own_gather,
                "latent_decode": _own_decode, "latent_prefill": _own_prefill}[op](s)
    return {"rope_append": _plain_rope, "latent_append": _plain_latent_append, "latent_gather": _plain_gather,
            "latent_decode": _plain_decode, "latent_prefill": _plain_prefill}[op](s)


def _pool_values(t):
    """A pool's bytes as the values they stand for."""
    return t.view(torch.float8_e4m3fn) if t.dtype == torch.uint8 else t


def _rope_result(s):
    out = [s["q_out"], _pool_values(s["k_pages"]), _pool_values(s["v_pages"])]
    return out + ([s["k_scale"], s["v_scale"]] if s["k_scale"] is not None else [])


def _latent_result(s):
    out = [s["q_out"], _pool_values(s["c_pages"]), s["r_pages"]]
    return out + ([s["c_scale"]] if s["c_scale"] is not None else [])


# --- the library's calls ---------------------------------------------------
def _pages(s):
    from paged_fp8_kv_decode_gb300 import binding as B
    mp = s["bt"].shape[1]
    return B.Pages(s["B"], mp, s["bt"], mp, 0, s["seq_lens"], 1, 0, None)


def _own_rope(s):
    from paged_fp8_kv_decode_gb300 import binding as B, rope as R
    c = s["case"]
    cache = B.Cache(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"])
    R.pfkv_rope_append(cache, _pages(s), R.Rope(s["inv_freq"], c["inter"]), s["positions"], s["k"], s["v"], s["q"],
                       s["q_out"], row_starts=s["starts"], max_new_tokens=s["T"], flags=s["flags"])
    return _rope_result(s)


def _own_latent_append(s):
    from paged_fp8_kv_decode_gb300 import latent as L, rope as R
    L.pfkv_latent_append(L.LatentCache(s["c_pages"], s["r_pages"], s["c_scale"]), _pages(s),
                         R.Rope(s["inv_freq"], s["case"]["inter"]), s["positions"], s["c"], s["r"], s["q"], s["q_out"],
                         row_starts=s["starts"], max_new_tokens=s["T"], flags=s["flags"])
    return _latent_result(s)


def _own_gather(s):
    from paged_fp8_kv_decode_gb300 import latent as L
    L.pfkv_latent_gather(L.LatentCache(s["c_pages"], s["r_pages"], s["c_scale"]), _pages(s), s["starts"], s["max_len"],
                         s["c_out"], s["r_out"], flags=s["flags"])
    return [s["c_out"], s["r_out"]]


def _own_decode(s):
    from paged_fp8_kv_decode_gb300 import latent as L
    c = s["case"]
    cache, pages = L.LatentCache(s["c_pages"], s["r_pages"], s["c_scale"]), _pages(s)
    if "workspace" not in s:  # a program allocates it once
        s["workspace"] = torch.empty(L.pfkv_latent_decode_workspace_size(cache, pages, c["H"], c["kq"], s["max_len"]),
                                     dtype=torch.uint8, device="cuda")
    L.pfkv_latent_decode_attn(cache, pages, s["q_c"], s["q_r"], s["scale"], s["max_len"], s["workspace"], s["out"],
                              flags=s["flags"])
    return s["out"]


def _own_prefill(s):
    from paged_fp8_kv_decode_gb300 import latent as L
    L.pfkv_latent_prefill_attn(s["q_nope"], s["q_rope"], s["k_nope"], s["k_rope"], s["v"], s["q_starts"], s["k_starts"],
                               s["nq"], s["scale"], True, s["out"], flags=s["flags"])
    return s["out"]


# --- plain forms -----------------------------------------------------------
def _token_rows(s):
    """Request and index within its new tokens of every row."""
    rows = torch.arange(s["R"], device="cuda")
    if s["starts"] is None:
        return rows // s["T"], rows % s["T"]
    b = torch.searchsorted(s["starts"][1:].long(), rows, right=True)
    return b, rows - s["starts"][b].long()


def _rotate(x, angle, inter):
    """x: [rows, heads, dim] in 32 bits; angle: [rows, pairs] in 64."""
    h = angle.shape[1]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if inter:
        a, b = x[..., 0:2 * h:2], x[..., 1:2 * h:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :h], x[..., h:2 * h]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., 2 * h:]), -1)


def _quantise(x, scale, page, opened):
    """x: [rows, heads, dim]; new scales of the pages that this call opens; e4m3 codes of x."""
    top = torch.zeros_like(scale).index_reduce_(0, page, x.abs().amax(-1), "amax")
    opens = torch.zeros(scale.shape[0], dtype=torch.bool, device="cuda")
    opens[page] = opened
    fresh = torch.where(top == 0, torch.ones_like(top), top / 448)
    scale.copy_(torch.where(opens[:, None], fresh, scale))
    y = (x / scale[page][..., None]).clamp(-448, 448)
    return y.to(torch.float8_e4m3fn).view(torch.uint8)


def _slots(s):
    b, t = _token_rows(s)
    pos = s["positions"][b].long() + t
    page, slot = s["bt"][b, pos // PAGE].long(), pos % PAGE
    opened = pos - slot >= s["positions"][b]  # the call writes the page's first slot
    return page, slot, opened, pos.double()[:, None] * s["inv_freq"].double()


def _plain_rope(s):
    c = s["case"]
    page, slot, opened, angle = _slots(s)
    q = s["q"].reshape(s["R"], c["Hq"], c["D"]).float()
    s["q_out"].copy_(_rotate(q, angle, c["inter"]).view_as(s["q_out"]))
    k = _rotate(s["k"].reshape(s["R"], c["Hkv"], c["D"]).float(), angle, c["inter"])
    v = s["v"].reshape(s["R"], c["Hkv"], c["D"]).float()
    if c["fp8"]:
        k, v = _quantise(k, s["k_scale"], page, opened), _quantise(v, s["v_scale"], page, opened)
    s["k_pages"][page, :, slot] = k.to(s["k_pages"].dtype)
    s["v_pages"][page, :, slot] = v.to(s["v_pages"].dtype)
    return _rope_result(s)


def _plain_latent_append(s):
    c = s["case"]
    page, slot, opened, angle = _slots(s)
    q = s["q"].reshape(s["R"], c["H"], ROPE).float()
    s["q_out"].copy_(_rotate(q, angle, c["inter"]).view_as(s["q_out"]))
    r = _rotate(s["r"].reshape(s["R"], 1, ROPE).float(), angle, c["inter"])
    s["r_pages"][page, slot] = r[:, 0].to(torch.bfloat16)
    x = s["c"].reshape(s["R"], LATENT)
    if c["fp8"]:
        x = _quantise(x.float()[:, None], s["c_scale"][:, None], page, opened)[:, 0]
    s["c_pages"][page, slot] = x
    return _latent_result(s)


def _values(s, pages):
    """Latents of the pages named, in 32 bits."""
    x = _pool_values(s["c_pages"])[pages].float() if s["c_scale"] is None else \
        s["c_pages"][pages].view(torch.float8_e4m3fn).float()
    return x if s["c_scale"] is None else x * s["c_scale"][pages][..., None, None]


def _plain_gather(s):
    rows = torch.arange(s["R"], device="cuda")
    b = torch.searchsorted(s["starts"][1:].long(), rows, right=True)
    j = rows - s["starts"][b].long()
    page, slot = s["bt"][b, j // PAGE].long(), j % PAGE
    if s["c_scale"] is None:
        c = s["c_pages"][page, slot]
    else:
        c = s["c_pages"][page, slot].view(torch.float8_e4m3fn).float() * s["c_scale"][page][:, None]
    s["c_out"].copy_(c)
    s["r_out"].copy_(s["r_pages"][page, slot])
    return [s["c_out"], s["r_out"]]


def _plain_decode(s):
    B, kq, H = s["case"]["B"], s["case"]["kq"], s["case"]["H"]
    bt = s["bt"].long().clamp(min=0)
    c = _values(s, bt).flatten(1, 2)                                   # [B, n, 512]
    r = s["r_pages"][bt].float().flatten(1, 2)
    j = torch.arange(c.shape[1], device="cuda")
    n = s["seq_lens"].long()
    live = (j[None] < n[:, None])[..., None]
    c, r = torch.where(live, c, 0.0), torch.where(live, r, 0.0)
    q = s["q_c"].float().reshape(B, kq * H, LATENT), s["q_r"].float().reshape(B, kq * H, ROPE)
    x = (q[0] @ c.transpose(1, 2) + q[1] @ r.transpose(1, 2)) * s["scale"]
    sees = n[:, None] - kq + 1 + torch.arange(kq * H, device="cuda")[None] // H  # tokens that a row attends to
    x = x.masked_fill_(j >= sees[..., None], -math.inf)
    p = (x - x.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    o = (p @ c) / p.sum(-1, keepdim=True)
    o = torch.where(sees[..., None] > 0, o, 0.0)
    s["out"].copy_(o.reshape(s["out"].shape))
    return s["out"]


def _padded(x, starts, width):
    """Packed rows [rows, ...] -> [B, width, ...]; rows past a request's end repeat its last."""
    i = torch.arange(width, device="cuda")
    n = (starts[1:] - starts[:-1]).long()
    at = starts[:-1].long()[:, None] + torch.minimum(i[None], (n - 1).clamp(min=0)[:, None])
    return x[at.clamp(max=x.shape[0] - 1)]


def _plain_prefill(s):
    q = torch.cat((_padded(s["q_nope"], s["q_starts"], s["nq"]), _padded(s["q_rope"], s["q_starts"], s["nq"])), -1)
    k = _padded(s["k_nope"], s["k_starts"], s["nk"])
    r = _padded(s["k_rope"], s["k_starts"], s["nk"])[:, :, None].expand(-1, -1, s["H"], -1)
    k, v = torch.cat((k, r), -1), _padded(s["v"], s["k_starts"], s["nk"])
    x = q.float().transpose(1, 2) @ k.float().permute(0, 2, 3, 1)      # [B, H, nq, nk]
    nq, nk = s["q_starts"][1:] - s["q_starts"][:-1], s["k_starts"][1:] - s["k_starts"][:-1]
    i, j = torch.arange(s["nq"], device="cuda"), torch.arange(s["nk"], device="cuda")
    hidden = (j[None, None] > i[None, :, None] + (nk - nq)[:, None, None]) | (j[None, None] >= nk[:, None, None])
    x = x.mul_(s["scale"]).masked_fill_(hidden[:, None], -math.inf)
    p = x.sub_(x.amax(-1, keepdim=True)).exp_()
    total = p.sum(-1, keepdim=True)
    o = ((p @ v.float().transpose(1, 2)) / total).transpose(1, 2)      # [B, nq, H, 128]
    rows = torch.arange(s["out"].shape[0], device="cuda")
    b = torch.searchsorted(s["q_starts"][1:].long(), rows, right=True)
    s["out"].copy_(o[b, rows - s["q_starts"][b].long()])
    return s["out"]


# ---------------------------------------------------------------------------
# the definition in 64 bits, request by request
# ---------------------------------------------------------------------------
def _turned(x, pos, inv_freq, inter):
    """x: [tokens, heads, dim] turned as complex numbers by pos * inv_freq."""
    x = x.double().clone()
    h = inv_freq.numel()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       torch.outer(pos.double(), inv_freq.double()))[:, None]
    re, im = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if inter else (slice(0, h), slice(h, 2 * h))
    z = torch.complex(x[..., re].contiguous(), x[..., im].contiguous()) * turn
    x[..., re], x[..., im] = z.real, z.imag
    return x


def _exact_append(s):
    case = s["case"]
    rope = case["op"] == "rope_append"
    heads = case["Hq"] if rope else case["H"]
    dim = case["D"] if rope else ROPE
    q = s["q"].reshape(s["R"], heads, dim)
    q_out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    names = [("k_pages", "k_scale"), ("v_pages", "v_scale")] if rope else [("c_pages", "c_scale")]
    pools = {p: _pool_values(s[p]).double() for p, _ in names}
    scales = {p: s[z].double() if s[z] is not None else None for p, z in names}
    r_pages = None if rope else s["r_pages"].double()
    table, ctx = s["bt"].tolist(), s["positions"].tolist()
    starts = s["starts"].tolist() if s["starts"] is not None else [i * s["T"] for i in range(s["B"] + 1)]
    for b in range(s["B"]):
        rows = slice(starts[b], starts[b + 1])
        n = starts[b + 1] - starts[b]
        pos = ctx[b] + torch.arange(n, device="cuda")
        q_out[rows] = _turned(q[rows], pos, s["inv_freq"], case["inter"])
        if rope:
            k = s["k"].reshape(s["R"], case["Hkv"], dim)[rows]
            new = {"k_pages": _turned(k, pos, s["inv_freq"], case["inter"]),
                   "v_pages": s["v"].reshape(s["R"], case["Hkv"], dim)[rows].double()}
        else:
            new = {"c_pages": s["c"].reshape(s["R"], 1, LATENT)[rows].double()}
            turned = _turned(s["r"].reshape(s["R"], 1, ROPE)[rows], pos, s["inv_freq"], case["inter"])[:, 0]
        at = 0
        while at < n:
            p = ctx[b] + at
            slot, count = p % PAGE, min(PAGE - p % PAGE, n - at)
            page = table[b][p // PAGE]
            for name, x in new.items():
                x = x[at:at + count]                                   # [count, heads, dim]
                if scales[name] is not None:
                    if slot == 0:
                        top = x.abs().amax((0, 2)) / 448
                        top = torch.where(top == 0, torch.ones_like(top), top)
                        scales[name][page] = top if rope else top[0]
                    z = scales[name][page]
                    x = (x / (z[:, None] if rope else z)).clamp(-448, 448)
                if rope:
                    pools[name][page, :, slot:slot + count] = x.transpose(0, 1)
                else:
                    pools[name][page, slot:slot + count] = x[:, 0]
            if not rope:
                r_pages[page, slot:slot + count] = turned[at:at + count]
            at += count
    out = [q_out.view(s["q_out"].shape)] + [pools[p] for p, _ in names] + ([] if rope else [r_pages])
    return out + [scales[p] for p, _ in names if scales[p] is not None]


def _exact_rows(s, b, n):
    pages = s["bt"][b, :(n + PAGE - 1) // PAGE].long()
    c = _pool_values(s["c_pages"])[pages].double()
    if s["c_scale"] is not None:
        c = c * s["c_scale"][pages].double()[:, None, None]
    return c.reshape(-1, LATENT)[:n], s["r_pages"][pages].double().reshape(-1, ROPE)[:n]


def exact(case, seed):
    if case["op"] == "latent_prefill" and case["B"] * case["H"] * case["q_hi"] ** 2 > 6e9:
        return None
    s = prepare(case, seed)
    if case["op"] in ("rope_append", "latent_append"):
        return _exact_append(s)
    if case["op"] == "latent_gather":
        got = [_exact_rows(s, b, n) for b, n in enumerate(s["seq_lens"].tolist())]
        return [torch.cat([x[0] for x in got]), torch.cat([x[1] for x in got])]
    if case["op"] == "latent_decode":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        for b, n in enumerate(s["seq_lens"].tolist()):
            c, r = _exact_rows(s, b, n)
            for t in range(case["kq"]):
                m = n - case["kq"] + 1 + t
                if m > 0:
                    w = torch.softmax((s["q_c"][b, t].double() @ c[:m].T + s["q_r"][b, t].double() @ r[:m].T)
                                      * s["scale"], -1)
                    out[b, t] = w @ c[:m]
        return out
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    qs, ks = s["q_starts"].tolist(), s["k_starts"].tolist()
    for b in range(s["B"]):
        a, z, u, w = qs[b], qs[b + 1], ks[b], ks[b + 1]
        seen = torch.ones(z - a, w - u, dtype=torch.bool, device="cuda").tril((w - u) - (z - a))
        for h in range(s["H"]):
            x = s["q_nope"][a:z, h].double() @ s["k_nope"][u:w, h].double().T
            x += s["q_rope"][a:z, h].double() @ s["k_rope"][u:w].double().T
            x = torch.where(seen, x * s["scale"], -math.inf)
            out[a:z, h] = torch.softmax(x, -1) @ s["v"][u:w, h].double()
    return out


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op, B = case["op"], case["B"]
    if op in ("rope_append", "latent_append"):
        rows = sum(_lens(max(1, case["T"] // 8), case["T"], B)) if case["packed"] else B * case["T"]
        el = 1 if case["fp8"] else 2
        if op == "rope_append":
            q, kv = case["Hq"] * case["D"], 2 * case["Hkv"] * case["D"]
            turned = (case["Hq"] + case["Hkv"]) * case["rot"]
        else:
            q, kv, turned = case["H"] * ROPE + ROPE, LATENT, (case["H"] + 1) * ROPE
        return {"bytes": rows * (4 * q + (2 + el) * kv), "flops": rows * 3 * turned}
    if op in ("latent_gather", "latent_decode"):
        n = _lens(case["n_lo"], case["n_hi"], B)
        cached = sum(n) * ((1 if case["fp8"] else 2) * LATENT + 2 * ROPE)
        if op == "latent_gather":
            return {"bytes": cached + sum(n) * 2 * (LATENT + ROPE), "flops": sum(n) * LATENT if case["fp8"] else 0}
        rows = case["kq"] * case["H"]
        seen = sum(max(0, k - case["kq"] + 1 + t) for k in n for t in range(case["kq"])) * case["H"]
        return {"bytes": cached + B * rows * 2 * (2 * LATENT + ROPE), "flops": 2 * seen * (2 * LATENT + ROPE)}
    nq = _lens(case["q_lo"], case["q_hi"], B)
    pre = _lens(0, case["pre_hi"], B, salt=2)
    pairs = sum(a * p + a * (a + 1) // 2 for a, p in zip(nq, pre))
    nk = sum(nq) + sum(pre)
    return {"bytes": 2 * case["H"] * (sum(nq) * (NOPE + ROPE + VDIM) + nk * (NOPE + VDIM)) + 2 * nk * ROPE,
            "flops": 2 * case["H"] * pairs * (NOPE + ROPE + VDIM)}
