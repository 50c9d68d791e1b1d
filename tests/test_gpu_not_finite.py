"""Scores that are not finite among a request's own tokens: what a row sees reaches it, in every
call that attends to own tokens; rows that do not see it have the bits that they have without it.

By the formula a score of NaN or +inf makes every weight of its row NaN, so the row and the totals
that it adds to are NaN; a score of -inf is a weight of zero."""
import math

import pytest
import torch

from prefix_cases import B, PAGE, Pool, call, close, no_prefixes, pages_of, rows

pytestmark = pytest.mark.gpu

NAN, INF = math.nan, math.inf


def plant(pool, pages, b, h, token, what):
    """Spoils a token's key (one element) or its unit's K scale."""
    page = pool.row(pages, b, h)[token // PAGE]
    if what == "scale":
        pool.cache.k_scale[page, h] = NAN
    elif pool.fp8:
        pool.cache.k_pages[page, h, token % PAGE, 7] = 0x7F
    else:
        pool.cache.k_pages[page, h, token % PAGE, 7] = NAN if what == "key" else INF


def whats(fp8):
    return ["key", "scale"] if fp8 else ["key", "inf"]


CASES = [(fp8, what) for fp8 in (False, True) for what in whats(fp8)]


@pytest.mark.parametrize("with_mass", [False, True])
@pytest.mark.parametrize("token", [0, 17, 299])
@pytest.mark.parametrize("fp8,what", CASES)
def test_own_token_behind_a_prefix(fp8, what, token, with_mass):
    """Own tokens behind a prefix, and of a request without one."""
    pool = Pool(200, 2, 128, fp8, seed=41)
    pre, own, of = pool.tables([300, 40]), pool.tables([300, 30, 300]), [0, 1, -1]
    q = rows(pool.g, 3, 1, 8, 128, outliers=0)
    q[..., 7] = q[..., 7].abs() + 0.5       # an infinite key's scores are +inf
    mass = [torch.zeros(3, 2, 300, device="cuda") if with_mass else None for _ in range(3)]
    want, _ = call(pool, own, pre, of, q, 0.1, mass=mass[0])
    for k, b in ((1, 0), (2, 2)):
        kept = [t.clone() for t in (pool.cache.k_pages, pool.cache.k_scale) if t is not None]
        plant(pool, own, b, 1, token, what)
        out, flags = call(pool, own, pre, of, q, 0.1, mass=mass[k])
        assert not flags[:3].any()
        assert out[b, 0, 4:].isnan().all()
        out[b, 0, 4:] = want[b, 0, 4:]
        assert torch.equal(out, want)
        if with_mass:
            assert mass[k][b, 1].isnan().all()
            mass[k][b, 1] = mass[0][b, 1]
            assert torch.equal(mass[k], mass[0])
        for t, old in zip((pool.cache.k_pages, pool.cache.k_scale), kept):
            t.copy_(old)


@pytest.mark.parametrize("fp8", [False, True])
def test_query(fp8):
    """A query that is NaN: its rows are, wherever they see a token."""
    pool = Pool(200, 2, 64, fp8, seed=42)
    pre, own, of = pool.tables([300]), pool.tables([20, 30, 0, 0]), [0, -1, -1, 0]
    q = rows(pool.g, 4, 1, 8, 64, outliers=0)
    q[:, 0, 5, 33] = NAN
    out, flags = call(pool, own, pre, of, q, 0.125)
    assert not flags[:4].any() and out[[0, 1, 3], 0, 5].isnan().all() and not out[2].any()


@pytest.mark.parametrize("what", [NAN, INF, -INF])
@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("fp8", [False, True])
def test_query_leaves_others(fp8, D, what):
    """A query head that is not finite leaves the other heads, those of its kv head among them, as they are."""
    pool = Pool(200, 2, D, fp8, seed=42)
    pre, own, of = pool.tables([300]), pool.tables([20, 30, 0, 0]), [0, -1, -1, 0]
    q = rows(pool.g, 4, 1, 8, D, outliers=0)
    # no element of the head that is spoiled is the largest of its kv head's queries
    q[:, 0, 5] = q[:, 0, 5].clamp(-1, 1)
    want, _ = call(pool, own, pre, of, q, 0.125)
    plain = _decode(pool, own, q[:, 0].contiguous(), 0, 30)
    q[:, 0, 5, 33] = what
    out, flags = call(pool, own, pre, of, q, 0.125)
    again = _decode(pool, own, q[:, 0].contiguous(), 0, 30)
    assert not flags[:4].any()
    if what != what:
        assert out[[0, 1, 3], 0, 5].isnan().all() and again[:2, 5].isnan().all()
    out[:, 0, 5], again[:, 5] = want[:, 0, 5], plain[:, 5]
    assert torch.equal(out, want) and torch.equal(again, plain)


@pytest.mark.parametrize("fp8", [False, True])
def test_candidates(fp8):
    """The last of three candidates has a key that is NaN: the rows of those before do not see it."""
    pool = Pool(200, 2, 128, fp8, seed=43)
    pre, own, of = pool.tables([130]), pool.tables([35, 3]), [0, -1]
    q = rows(pool.g, 2, 3, 4, 128, outliers=0)
    want, _ = call(pool, own, pre, of, q, 0.1)
    for b, n in enumerate((35, 3)):
        plant(pool, own, b, 0, n - 1, "key")
    out, flags = call(pool, own, pre, of, q, 0.1)
    assert not flags[:2].any() and out[:, 2, :2].isnan().all()
    out[:, 2, :2] = want[:, 2, :2]
    assert torch.equal(out, want)


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("fp8", [False, True])
def test_values(fp8, bad):
    """A value that is not finite, over a prefix and among own tokens: one element of the rows that see it."""
    pool = Pool(200, 2, 64, fp8, seed=47)
    pre, own, of = pool.tables([300, 140]), pool.tables([90, 60, 33]), [0, -1, 1]
    q = rows(pool.g, 3, 1, 8, 64, outliers=0)
    mass = [torch.zeros(3, 2, 90, device="cuda") for _ in range(2)]
    want, _ = call(pool, own, pre, of, q, 0.1, mass=mass[0])
    for pages, i, token, d in ((pre, 0, 210, 5), (own, 1, 17, 40)):
        page = pool.row(pages, i, 1)[token // PAGE]
        if fp8:
            pool.cache.v_pages[page, 1, token % PAGE, d] = 0x7F
        else:
            pool.cache.v_pages[page, 1, token % PAGE, d] = bad
    out, flags = call(pool, own, pre, of, q, 0.1, mass=mass[1])
    assert not flags[:3].any() and torch.equal(*mass)
    for b, d in ((0, 5), (1, 40)):
        assert not out[b, 0, 4:, d].isfinite().any()
        out[b, 0, 4:, d] = want[b, 0, 4:, d]
    assert torch.equal(out, want)


@pytest.mark.parametrize("first,last", [(21, 22), (0, 16), (0, 48), (3, 50)])
def test_minus_infinity(first, last):
    """A score of -inf is a weight of zero, for the row and for the totals, whole units of them too."""
    pool = Pool(200, 2, 128, False, seed=44)
    pre, own, of = pool.tables([300]), pool.tables([90, 60]), [0, -1]
    q = rows(pool.g, 2, 1, 8, 128, outliers=0)
    q[..., 7] = q[..., 7].abs() + 0.5
    got = []
    for x in (-INF, -1e30):  # and the same with keys whose weights underflow
        for b in range(2):
            ids = pool.row(own, b, 1)
            j = torch.arange(first, last, device="cuda")
            pool.cache.k_pages[ids[j // PAGE], 1, j % PAGE, 7] = x
        mass = torch.zeros(2, 2, 90, device="cuda")
        out, flags = call(pool, own, pre, of, q, 0.1, mass=mass)
        other = torch.zeros_like(mass)
        plain = _decode(pool, own, q[:, 0].contiguous(), 0, 90, mass=other)
        cores = _decode(pool, own, q[:, 0].contiguous(), 64, 90, options=B.PFKV_STAGE_CUDA_CORES)
        assert not flags[:2].any()
        got.append((out, mass, plain, other, cores))
    for x, y in zip(*got):
        assert x.isfinite().all() and torch.equal(x, y)
    assert not got[0][1][:, 1, first:last].any() and not got[0][3][:, 1, first:last].any()
    # the weights of the request without a prefix sum to one a query head
    close(got[0][1][1].sum(-1), torch.full((2,), 4.0, dtype=torch.float64, device="cuda"), 1e-3, "weights of a row")


def _decode(pool, own, q, split, n, stages=None, mass=None, options=0):
    """pfkv_paged_decode_attn and its relatives; returns (out, flags)."""
    hq = q.shape[-2]
    out, flags = torch.zeros_like(q), torch.full((4,), 0xAA, dtype=torch.uint8, device="cuda")
    ws = torch.full((8 << 20,), 0xFF, dtype=torch.uint8, device="cuda")
    if q.dim() == 4:
        assert ws.numel() >= B.pfkv_decode_multi_workspace_size(pool.cache, own, hq, q.shape[1], split, n)
        B.pfkv_paged_decode_attn_multi(pool.cache, own, q, 0.1, split, n, ws, out, flags)
    elif mass is not None:
        assert ws.numel() >= B.pfkv_decode_mass_workspace_size(pool.cache, own, hq, split, n)
        B.pfkv_paged_decode_attn_mass(pool.cache, own, q, 0.1, split, n, ws, out, flags, mass)
    else:
        B.pfkv_paged_decode_attn_stages(pool.cache, own, q, 0.1, split, n, ws, out, flags, B.PFKV_STAGE_ALL | options)
    assert not flags[:q.shape[0]].any()
    return out


@pytest.mark.parametrize("kind", ["plain", "split", "cuda cores", "cuda cores, one chunk", "mass", "mass, split", "candidates"])
@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("fp8,what", CASES)
def test_decode(fp8, what, D, kind):
    """The calls without prefixes, by the persistent kernel and by the one of a chunk a CTA."""
    pool = Pool(200, 2, D, fp8, seed=45)
    own = pool.tables([700, 40])
    kq = 3 if kind == "candidates" else 1
    q = rows(pool.g, 2, kq, 8, D, outliers=0)
    q[..., 7] = q[..., 7].abs() + 0.5
    q = q if kq > 1 else q[:, 0].contiguous()
    split = {"split": 48, "mass, split": 256, "cuda cores": 64, "cuda cores, one chunk": 1024}.get(kind, 0)
    options = B.PFKV_STAGE_CUDA_CORES if "cuda" in kind else 0
    mass = [torch.zeros(2, 2, 700, device="cuda") if "mass" in kind else None for _ in range(2)]
    want = _decode(pool, own, q, split, 700, mass=mass[0], options=options)
    plant(pool, own, 0, 1, 300, what)
    out = _decode(pool, own, q, split, 700, mass=mass[1], options=options)
    hit = out[0, ..., 4:, :]
    assert hit.isnan().all()
    hit.copy_(want[0, ..., 4:, :])
    assert torch.equal(out, want)
    if mass[0] is not None:
        assert mass[1][0, 1].isnan().all()
        mass[1][0, 1] = mass[0][0, 1]
        assert torch.equal(*mass)


@pytest.mark.parametrize("fp8", [False, True])
def test_many_parts(fp8):
    """A long request whose parts many workers hold, of which one meets the NaN; no prefixes."""
    n = 20000
    pool = Pool(pages_of(n) + 20, 1, 128, fp8, seed=46)
    own = pool.tables([n, 70])
    q = rows(pool.g, 2, 1, 4, 128, outliers=0)
    want, _ = call(pool, own, no_prefixes(1), [-1, -1], q, 0.1)
    plant(pool, own, 0, 0, 12345, "key")
    out, flags = call(pool, own, no_prefixes(1), [-1, -1], q, 0.1)
    assert not flags[:2].any() and out[0].isnan().all() and torch.equal(out[1], want[1])
    assert _decode(pool, own, q[:, 0].contiguous(), 0, n)[0].isnan().all()

