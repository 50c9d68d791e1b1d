"""Cases, plain forms and exact values of attention over shared prefixes and of eviction.

Two operators that a serving program calls on a paged cache:

  prefix   decode attention of a batch whose requests share prefixes: each prefix is read once for all
           of its requests, their own tokens follow it; a few query tokens a request (candidates, or
           decoder tokens that attend to an encoder's states, which are a prefix without anything after it);
           on request the summed softmax weight of each of a request's own tokens is added to its total
  evict    the tokens of a cache with the largest totals (and the first and the last ones) move, in order,
           to new pages; per head, FP8 pages with new scales

``run`` computes them with elementary torch operations in 32 bits while ``own`` is
false, and through the library's entry points while it is true.
"""
import math
import random

import torch

own = False

PAGE = 16


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a few conversations just begun behind a short system prompt: latency
        dict(name="prefix few bf16", op="prefix", B=4, NP=1, alone=0, kq=1, Hq=32, Hkv=8, D=128, fp8=False,
             p_lo=1000, p_hi=1000, n_lo=1, n_hi=60, per_head=False, mass=False),
        # the benchmark's layer: a batch of 32 behind one long system prompt
        dict(name="prefix batch fp8", op="prefix", B=32, NP=1, alone=0, kq=1, Hq=32, Hkv=8, D=128, fp8=True,
             p_lo=16384, p_hi=16384, n_lo=64, n_hi=2048, per_head=False, mass=False),
        # a large batch with groups of 8 query heads: bound by arithmetic
        dict(name="prefix wide bf16", op="prefix", B=256, NP=1, alone=0, kq=1, Hq=64, Hkv=8, D=128, fp8=False,
             p_lo=8192, p_hi=8192, n_lo=16, n_hi=512, per_head=False, mass=False),
        # a long document shared by a few questions
        dict(name="prefix long bf16", op="prefix", B=16, NP=1, alone=0, kq=1, Hq=32, Hkv=8, D=128, fp8=False,
             p_lo=131072, p_hi=131072, n_lo=100, n_hi=1000, per_head=False, mass=False),
        # several prefixes of ragged lengths, requests without one among them, candidates to verify, heads of 64
        dict(name="prefix ragged fp8", op="prefix", B=45, NP=6, alone=5, kq=3, Hq=16, Hkv=4, D=64, fp8=True,
             p_lo=300, p_hi=30000, n_lo=3, n_hi=1500, per_head=False, mass=False),
        # decoder tokens that attend to encoder states of their own request: nothing follows the prefix
        dict(name="states bf16", op="prefix", B=8, NP=8, alone=0, kq=4, Hq=16, Hkv=16, D=64, fp8=False,
             p_lo=200, p_hi=1500, n_lo=0, n_hi=0, per_head=False, mass=False),
        # own tokens evicted per head before, and their weights wanted for the next eviction
        dict(name="prefix mass fp8", op="prefix", B=24, NP=3, alone=0, kq=1, Hq=32, Hkv=8, D=128, fp8=True,
             p_lo=2000, p_hi=9000, n_lo=500, n_hi=4000, per_head=True, mass=True),
        # one conversation grown past its budget
        dict(name="evict one bf16", op="evict", B=1, Hkv=8, D=128, fp8=False, n_lo=1000, n_hi=1000, part=4, first=4,
             last=64, per_head=True),
        # a batch, a quarter kept
        dict(name="evict batch fp8", op="evict", B=32, Hkv=8, D=128, fp8=True, n_lo=512, n_hi=8192, part=4, first=4,
             last=128, per_head=True),
        # heads of 64, lengths that differ from head to head, half kept
        dict(name="evict heads bf16", op="evict", B=16, Hkv=4, D=64, fp8=False, n_lo=33, n_hi=20000, part=2, first=0,
             last=16, per_head=True),
        # long contexts, an eighth kept
        dict(name="evict long fp8", op="evict", B=2, Hkv=8, D=128, fp8=True, n_lo=200000, n_hi=262144, part=8, first=16,
             last=1024, per_head=True),
        # one table and one length for all heads
        dict(name="evict shared fp8", op="evict", B=7, Hkv=2, D=64, fp8=True, n_lo=1, n_hi=5000, part=3, first=1,
             last=7, per_head=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    fp8, D, Hkv = rng.random() < 0.5, rng.choice([64, 128, 128]), rng.choice([1, 2, 4, 8])
    if rng.random() < 0.6:
        G, kq = rng.choice([1, 2, 4, 4, 8]), rng.choice([1, 1, 1, 2, 3, 4])
        p_hi = _log(rng, 16, 100000)
        NP = min(_log(rng, 1, 12), max(1, 130000 // p_hi))
        # members x tokens: what a pass computes
        B = min(_log(rng, 1, 200), max(1, 2 ** 23 // (p_hi * kq * G) + 1))
        B = max(B, min(NP, 4))
        n_hi = min(_log(rng, 1, 4000), max(1, 120000 // B))
        if rng.random() < 0.15:
            n_lo = n_hi = 0
        else:
            n_lo = rng.randint(min(kq, n_hi), n_hi)
        return dict(op="prefix", B=B, NP=NP, alone=rng.choice([0, 0, B // 5]), kq=kq, Hq=G * Hkv, Hkv=Hkv, D=D, fp8=fp8,
                    p_lo=rng.randint(1, p_hi), p_hi=p_hi, n_lo=n_lo, n_hi=n_hi,
                    per_head=n_hi > 0 and rng.random() < 0.4, mass=n_hi > 0 and kq == 1 and rng.random() < 0.3)
    n_hi = _log(rng, 20, 200000)
    B = min(_log(rng, 1, 48), max(1, 400000 // n_hi))
    part = rng.choice([2, 3, 4, 8, 16])
    return dict(op="evict", B=B, Hkv=Hkv, D=D, fp8=fp8, n_lo=rng.randint(1, n_hi), n_hi=n_hi, part=part,
                first=rng.choice([0, 1, 4, 16]), last=rng.choice([0, 1, 16, _log(rng, 1, 300)]),
                per_head=Hkv == 1 or rng.random() < 0.7)


def _lens(lo, hi, B, salt=0):
    """B lengths in [lo, hi], the same for every seed."""
    r = random.Random(lo * 1000003 + hi * 101 + B * 7 + salt)
    v = [r.randint(lo, hi) for _ in range(B)]
    v[0] = hi
    return v


def _head_lens(case):
    """Lengths of every (request, head): rows of Hkv equal or differing numbers."""
    B, H = case["B"], case["Hkv"]
    if not case["per_head"]:
        return [[n] * H for n in _lens(case["n_lo"], case["n_hi"], B, 1)]
    v = _lens(case["n_lo"], case["n_hi"], B * H, 1)
    return [v[b * H:(b + 1) * H] for b in range(B)]


def _members(case):
    """The prefix of every request, -1 for those without one; every prefix has a request where there are enough."""
    B, NP, alone = case["B"], case["NP"], case["alone"]
    r = random.Random(B * 31 + NP * 7 + alone)
    v = [-1] * alone + [i if i < NP else r.randrange(NP) for i in range(B - alone)]
    r.shuffle(v)
    return v


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
    """N(0, 1), one value in a hundred 20 times as large: the values of keys and values."""
    x = torch.randn(*shape, generator=g, device="cuda")
    if outliers:
        x = torch.where(torch.rand(*shape, generator=g, device="cuda") < 0.01, x * 20, x)
    return x.to(torch.bfloat16)


def _pool(s, g, pages, case):
    shape = (pages, case["Hkv"], PAGE, case["D"])
    for name in ("k", "v"):
        if case["fp8"]:  # N(0, 100^2) codes, as a page whose largest value is near 448 holds them
            x = torch.randn(*shape, generator=g, device="cuda") * 100
            s[name + "_pages"] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            s[name + "_scale"] = torch.exp(torch.randn(*shape[:2], generator=g, device="cuda") * 0.3 - 4.6)
        else:
            s[name + "_pages"], s[name + "_scale"] = _rows(g, *shape), None


def _tables(perm, at, counts):
    """Tables [rows][heads or 1][most] that take pages perm[at:] in turn; (table, next place)."""
    most = max(1, max(max(r) for r in counts))
    bt = torch.full((len(counts), len(counts[0]), most), -1, dtype=torch.int32)
    for b, r in enumerate(counts):
        for h, c in enumerate(r):
            bt[b, h, :c] = perm[at:at + c]
            at += c
    return bt.cuda(), at


def _page_counts(lens, per_head):
    return [[(n + PAGE - 1) // PAGE for n in (r if per_head else r[:1])] for r in lens]


def prepare(case, seed):
    g = _gen(seed)
    B, H, D = case["B"], case["Hkv"], case["D"]
    lens = _head_lens(case)
    counts = _page_counts(lens, case["per_head"])
    own_heads = H if case["per_head"] else 1  # lengths and tables a request
    s = dict(case=case, lens=_i32([r[:own_heads] for r in lens]), max_len=max(max(r) for r in lens),
             flags=torch.zeros((B + 3) // 4 * 4, dtype=torch.uint8, device="cuda"))
    if case["op"] == "evict":
        keep = [[min(n, max(1, n // case["part"] + case["first"])) for n in r] for r in lens]
        new = _page_counts(keep, case["per_head"])
        total = sum(map(sum, counts)) + sum(map(sum, new)) + 4
        perm = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        s["bt"], at = _tables(perm, 0, counts)
        s["new_bt"], at = _tables(perm, at, new)
        _pool(s, g, total, case)
        # totals over past steps: most tokens little, few much, some (new ones) nothing yet
        x = torch.exp(torch.randn(B, H, s["max_len"], generator=g, device="cuda") * 2 - 6)
        s["mass"] = torch.where(torch.rand(x.shape, generator=g, device="cuda") < 0.02, torch.zeros_like(x), x)
        s["keep"], s["max_keep"] = _i32([r[:own_heads] for r in keep]), max(max(r) for r in keep)
        s["room"] = s["max_keep"] + 64  # of the new totals: tokens that decoding will append
        s["new_lens"] = torch.zeros(B, own_heads, dtype=torch.int32, device="cuda")
        s["new_mass"] = torch.zeros(B, H, s["room"], device="cuda")
        s["kept"] = torch.zeros(B, H, s["max_keep"], dtype=torch.int32, device="cuda")
        return s
    plens = [[n] for n in _lens(case["p_lo"], case["p_hi"], case["NP"])]
    total = sum(map(sum, counts)) + sum((n + PAGE - 1) // PAGE for n, in plens) + 4
    perm = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    s["bt"], at = _tables(perm, 0, counts)
    s["p_bt"], at = _tables(perm, at, _page_counts(plens, False))
    s["p_lens"], s["p_max"] = _i32([n for n, in plens]), max(n for n, in plens)
    s["prefix_of"] = _i32(_members(case))
    _pool(s, g, total, case)
    s["q"] = _rows(g, B, case["kq"], case["Hq"], D, outliers=False)
    s["out"] = torch.zeros_like(s["q"])
    s["scale"] = 1.0 / math.sqrt(D)
    s["mass"] = torch.rand(B, H, s["max_len"], generator=g, device="cuda") * 0.01 if case["mass"] else None
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    evict = s["case"]["op"] == "evict"
    if own:
        return (_own_evict if evict else _own_prefix)(s)
    return (_plain_evict if evict else _plain_prefix)(s)


def _values(t):
    """A pool's bytes as the values they stand for."""
    return t.view(torch.float8_e4m3fn) if t.dtype == torch.uint8 else t


def _evict_result(s):
    out = [s["new_lens"], s["kept"], s["new_mass"], _values(s["k_pages"]), _values(s["v_pages"])]
    return out + ([s["k_scale"], s["v_scale"]] if s["k_scale"] is not None else [])


# --- the library's calls ---------------------------------------------------
def _cache_and_pages(s):
    from paged_fp8_kv_decode_gb300 import binding as B
    case = s["case"]
    heads = 1 if case["per_head"] else 0  # tables and lengths of each head's own, or one for all

    def pages(bt, lens):
        return B.Pages(bt.shape[0], bt.shape[2], bt, bt.stride(0), heads * bt.stride(1), lens, lens.stride(0), heads)
    return B.Cache(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"]), pages


def _own_prefix(s):
    from paged_fp8_kv_decode_gb300 import binding as B, prefix as P
    case = s["case"]
    cache, pages = _cache_and_pages(s)
    mine = pages(s["bt"], s["lens"]) if s["max_len"] > 0 else None
    shared = B.Pages(case["NP"], s["p_bt"].shape[2], s["p_bt"], s["p_bt"].stride(0), 0, s["p_lens"], 1, 0)
    if "workspace" not in s:  # a program allocates it once
        s["workspace"] = torch.empty(P.pfkv_prefix_decode_workspace_size(
            cache, mine, shared, case["B"], case["Hq"], case["kq"], s["max_len"], s["p_max"], mass=case["mass"]),
            dtype=torch.uint8, device="cuda")
    P.pfkv_prefix_decode_attn(cache, mine, shared, s["prefix_of"], s["q"], s["scale"], s["max_len"], s["p_max"],
                              s["workspace"], s["out"], attn_mass=s["mass"], flags=s["flags"])
    return [s["out"], s["mass"]] if case["mass"] else [s["out"]]


def _own_evict(s):
    from paged_fp8_kv_decode_gb300 import evict as E
    case = s["case"]
    cache, pages = _cache_and_pages(s)
    src, dst = pages(s["bt"], s["lens"]), pages(s["new_bt"], s["new_lens"])
    if "workspace" not in s:
        s["workspace"] = torch.empty(E.pfkv_kv_evict_workspace_size(cache, src, s["max_len"], s["max_keep"]),
                                     dtype=torch.uint8, device="cuda")
    E.pfkv_kv_evict(cache, src, dst, s["keep"], s["mass"], s["max_len"], s["max_keep"], s["workspace"], s["new_lens"],
                    new_mass=s["new_mass"], kept=s["kept"], keep_first=case["first"], keep_last=case["last"],
                    flags=s["flags"])
    return _evict_result(s)


# --- plain forms -----------------------------------------------------------
def _gathered(s, name, bt, n):
    """Values of the first n tokens of the tables' rows, in 32 bits: [rows, Hkv, n, D]."""
    H = s["case"]["Hkv"]
    page = bt[:, :, :(n + PAGE - 1) // PAGE].long().clamp(min=0).expand(-1, H, -1)
    h = torch.arange(H, device="cuda")[None, :, None]
    x = _values(s[name + "_pages"])[page, h] if s[name + "_scale"] is None else \
        s[name + "_pages"][page, h].view(torch.float8_e4m3fn)
    x = x.float()
    if s[name + "_scale"] is not None:
        x = x * s[name + "_scale"][page, h][..., None, None]
    return x.flatten(2, 3)[:, :, :n]


def _part(s, q, bt, n, sees):
    """Unnormalised attention of rows q [X, Hkv, R, D] over the tables' first n tokens, of which a row
    sees the first `sees` [X, Hkv or 1, R]: (weighted sums, sums, maxima, weights)."""
    x = q @ _gathered(s, "k", bt, n).transpose(2, 3)
    x = x.mul_(s["scale"]).masked_fill_(torch.arange(n, device="cuda") >= sees[..., None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp_(min=-1e30)
    w = x.sub_(top).exp_()
    live = (torch.arange(n, device="cuda") < sees.amax(-1, keepdim=True))[..., None]
    v = torch.where(live, _gathered(s, "v", bt, n), 0.0)
    return w @ v, w.sum(-1, keepdim=True), top, w


def _plain_prefix(s):
    case = s["case"]
    B, kq, H, D, NP = case["B"], case["kq"], case["Hkv"], case["D"], case["NP"]
    G = case["Hq"] // H
    q = s["q"].float().view(B, kq, H, G, D).permute(0, 2, 1, 3, 4)     # [B, H, kq, G, D]
    # the rows of each prefix's requests side by side
    of = torch.where(s["prefix_of"] < 0, NP, s["prefix_of"].long())
    same = (of[:, None] == of[None]) & (torch.arange(B, device="cuda")[:, None] > torch.arange(B, device="cuda")[None])
    place = same.sum(1)
    most = max(1, max(_members(case).count(p) for p in range(NP)))     # as a program knows its groups
    member = of < NP
    rows = torch.zeros(NP + 1, max(most, B), H, kq, G, D, device="cuda")
    rows[of, place] = q
    rows = rows[:NP, :most].permute(0, 2, 1, 3, 4, 5).reshape(NP, H, most * kq * G, D)
    sees = s["p_lens"][:, None, None].expand(-1, 1, rows.shape[2])
    part = _part(s, rows, s["p_bt"], s["p_max"], sees)[:3]
    at = of.clamp(max=NP - 1), place.clamp(max=most - 1)
    o, z, m = (t.view(NP, H, most, kq * G, -1).transpose(1, 2)[at] for t in part)
    none = ~member[:, None, None, None]
    o, z, m = o.masked_fill(none, 0.0), z.masked_fill(none, 0.0), m.masked_fill(none, -1e30)
    if s["max_len"] > 0:
        t = torch.arange(kq * G, device="cuda") // G
        sees = (s["lens"][..., None] - kq + 1 + t).clamp(min=0)        # [B, H or 1, kq * G]
        o2, z2, m2, w = _part(s, q.reshape(B, H, kq * G, D), s["bt"], s["max_len"], sees)
        top = torch.maximum(m, m2)
        a, b = (m - top).exp(), (m2 - top).exp()
        o, z = o * a + o2 * b, z * a + z2 * b
        if case["mass"]:
            s["mass"] += (w * (b / z.clamp(min=1e-30))).sum(2)
    o = torch.where(z > 0, o / z, 0.0)
    s["out"].copy_(o.view(B, H, kq, G, D).permute(0, 2, 1, 3, 4).reshape(s["out"].shape))
    return [s["out"], s["mass"]] if case["mass"] else [s["out"]]


def _plain_evict(s):
    case = s["case"]
    B, H, K = case["B"], case["Hkv"], s["max_keep"]
    n, k = (s[x].long().expand(B, H)[..., None] for x in ("lens", "keep"))
    first = k.clamp(max=case["first"])
    last = torch.minimum(k - first, torch.full_like(k, case["last"]))
    j = torch.arange(s["max_len"], device="cuda")
    middle = (j >= first) & (j < n - last)
    order = torch.sort(torch.where(middle, s["mass"], -math.inf), dim=-1, descending=True, stable=True)[1]
    rank = torch.zeros_like(order).scatter_(-1, order, j.expand_as(order))
    keeps = (j < n) & ((j < first) | (j >= n - last) | (middle & (rank < k - first - last)))
    to = torch.where(keeps, keeps.cumsum(-1) - 1, K)                    # K: a place that is cut off
    kept = torch.zeros(B, H, K + 1, dtype=torch.long, device="cuda").scatter_(-1, to, j.expand_as(to))[..., :K]
    i = torch.arange(K, device="cuda")
    there = i < k
    s["kept"].copy_(torch.where(there, kept, 0))
    s["new_lens"].copy_(s["keep"])
    s["new_mass"].zero_()
    s["new_mass"][..., :K] = torch.where(there, s["mass"].gather(-1, kept), 0.0)
    # rows in their new places, page by page
    places = (K + PAGE - 1) // PAGE
    pad = places * PAGE - K
    h = torch.arange(H, device="cuda")[None, :, None]
    page = s["bt"].long().clamp(min=0).expand(-1, H, -1).gather(-1, kept // PAGE)
    slot = kept % PAGE
    to_page = s["new_bt"].long().expand(-1, H, -1)[..., i // PAGE]
    b_, h_, i_ = there.nonzero(as_tuple=True)
    where = to_page[b_, h_, i_], h_, i_ % PAGE
    if case["fp8"]:
        def paged(x, fill):
            return torch.nn.functional.pad(x, (0, pad), value=fill).view(B, H, places, PAGE)
        live = paged(there, False)
        src = paged(page, -1)
        src = torch.where(live, src, src[..., :1])
        one = (src == src[..., :1]).all(-1)                             # every token from one page
        p_, q_, r_ = (torch.arange(places, device="cuda") * PAGE < k).nonzero(as_tuple=True)
    for name in ("k", "v"):
        pool = s[name + "_pages"]
        x = pool[page, h, slot]
        if case["fp8"]:
            scale = s[name + "_scale"]
            x = x.view(torch.float8_e4m3fn).float()
            from_ = scale[page, h]
            y = x * from_[..., None]
            top = paged(torch.where(there, y.abs().amax(-1), 0.0), 0.0).amax(-1)
            fresh = torch.where(top == 0, 1.0, top / 448)
            new = torch.where(one, paged(from_, 1.0)[..., 0], fresh)
            z = torch.where(one, 1.0, new)[..., None].expand(-1, -1, -1, PAGE).flatten(2)[..., :K]
            kept_as = one[..., None].expand(-1, -1, -1, PAGE).flatten(2)[..., :K]
            x = (torch.where(kept_as[..., None], x, y) / z[..., None]).clamp(-448, 448)
            x = x.to(torch.float8_e4m3fn).view(torch.uint8)
            scale[s["new_bt"].long().expand(-1, H, -1)[p_, q_, r_], q_] = new[p_, q_, r_]
        pool[where] = x[b_, h_, i_]
    return _evict_result(s)


# ---------------------------------------------------------------------------
# the definition in 64 bits, request by request
# ---------------------------------------------------------------------------
def _tokens(s, name, row, n):
    """The first n tokens of one head's table row, by head h = row[0]: [n, D] in 64 bits."""
    h, table = row
    pages = table[:(n + PAGE - 1) // PAGE].long()
    x = _values(s[name + "_pages"][pages, h]).double()
    if s[name + "_scale"] is not None:
        x = x * s[name + "_scale"][pages, h].double()[:, None, None]
    return x.reshape(-1, x.shape[-1])[:n]


def _exact_prefix(s):
    case = s["case"]
    G, kq = case["Hq"] // case["Hkv"], case["kq"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    mass = s["mass"].double() if case["mass"] else None
    lens, plens, of = _head_lens(case), s["p_lens"].tolist(), s["prefix_of"].tolist()
    for h in range(case["Hkv"]):
        shared = {p: [_tokens(s, x, (h, s["p_bt"][p, 0]), plens[p]) for x in "kv"] for p in set(of) if p >= 0}
        for b in range(case["B"]):
            n = lens[b][h]
            table = s["bt"][b, h if case["per_head"] else 0]
            k, v = (_tokens(s, x, (h, table), n) for x in "kv")
            P = plens[of[b]] if of[b] >= 0 else 0
            if P:
                k, v = torch.cat((shared[of[b]][0], k)), torch.cat((shared[of[b]][1], v))
            for t in range(kq):
                m = P + max(0, n - kq + 1 + t)
                if m == 0:
                    continue
                heads = slice(h * G, (h + 1) * G)
                w = torch.softmax(s["q"][b, t, heads].double() @ k[:m].T * s["scale"], -1)
                out[b, t, heads] = w @ v[:m]
                if mass is not None:
                    mass[b, h, :n] += w[:, P:].sum(0)
    return [out] if mass is None else [out, mass]


def _exact_evict(s):
    case = s["case"]
    pools = {x: _values(s[x + "_pages"]).double() for x in "kv"}
    scales = {x: s[x + "_scale"].double() if case["fp8"] else None for x in "kv"}
    values = {x: pools[x] * scales[x][..., None, None] if case["fp8"] else pools[x] for x in "kv"}
    pools, scales = {x: t.clone() for x, t in pools.items()}, {x: t.clone() if case["fp8"] else t for x, t in scales.items()}
    mass_out = torch.zeros(s["new_mass"].shape, dtype=torch.float64, device="cuda")
    lens, keep = (s[x].expand(case["B"], case["Hkv"]).tolist() for x in ("lens", "keep"))
    mass = s["mass"].double()
    bt, new_bt = s["bt"].long(), s["new_bt"].long()
    for b in range(case["B"]):
        for h in range(case["Hkv"]):
            t = h if case["per_head"] else 0
            n, k = lens[b][h], keep[b][h]
            f = min(case["first"], k)
            z = min(case["last"], k - f)
            rest = mass[b, h, f:n - z]
            best = torch.sort(-rest, stable=True)[1][:k - f - z] + f
            ids = torch.cat((torch.arange(f, device="cuda"), best.sort()[0], torch.arange(n - z, n, device="cuda")))
            mass_out[b, h, :k] = mass[b, h, ids]
            page, slot = bt[b, t][ids // PAGE], ids % PAGE
            places = (k + PAGE - 1) // PAGE
            to = new_bt[b, t][:places]
            fill = places * PAGE - k
            which = torch.cat((page, page[-1:].expand(fill))).view(-1, PAGE)
            # a last page that is not full takes its fill from its own last token: same page, same largest value
            one = (which == which[:, :1]).all(1)
            for x in "kv":
                rows = values[x][page, h, slot]
                if not case["fp8"]:
                    pools[x][to[torch.arange(k, device="cuda") // PAGE], h, torch.arange(k, device="cuda") % PAGE] = rows
                    continue
                top = torch.cat((rows, rows[-1:].expand(fill, -1))).view(places, -1).abs().amax(1) / 448
                top = torch.where(top == 0, torch.ones_like(top), top)
                scale = torch.where(one, scales[x][which[:, 0], h], top)
                at = torch.arange(k, device="cuda")
                pools[x][to[at // PAGE], h, at % PAGE] = (rows / scale[at // PAGE][:, None]).clamp(-448, 448)
                scales[x][to, h] = scale
    out = [None, None, mass_out, pools["k"], pools["v"]]
    return out + ([scales["k"], scales["v"]] if case["fp8"] else [])


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_evict(s) if case["op"] == "evict" else _exact_prefix(s)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    B, H, D, el = case["B"], case["Hkv"], case["D"], 1 if case["fp8"] else 2
    lens = _head_lens(case)
    token = 2 * D * el + (0.5 if case["fp8"] else 0)                    # K and V of one head, with its share of scales
    if case["op"] == "evict":
        keep = [[min(n, max(1, n // case["part"] + case["first"])) for n in r] for r in lens]
        most = max(max(r) for r in keep)
        k = sum(map(sum, keep))
        return {"bytes": 4 * sum(map(sum, lens)) + 2 * k * token + 4 * k + 4 * B * H * (most + 64),
                "flops": k * 2 * D * 3 if case["fp8"] else 0}
    plens, of, kq = _lens(case["p_lo"], case["p_hi"], case["NP"]), _members(case), case["kq"]
    used = sum(plens[p] for p in set(of) if p >= 0)
    mine = sum(map(sum, lens))
    rows = case["Hq"] // H
    pairs = sum(plens[p] for p in of if p >= 0) * kq * H
    pairs += sum(max(0, n - kq + 1 + t) for r in lens for n in r for t in range(kq))
    return {"bytes": (used * H + mine) * token + 4 * B * kq * case["Hq"] * D + (8 * mine if case["mass"] else 0),
            "flops": 4 * D * rows * pairs}
