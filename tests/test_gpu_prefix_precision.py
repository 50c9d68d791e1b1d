"""Attention over a prefix where a rounding of its weights shows most: a few dominant tokens whose large
values nearly cancel, and queries whose elements are far apart.

The library's bound for attention, |got - ref| <= 1e-2 + 1e-2 |ref|, holds for requests that have the
tokens as their own (a weight rounded once to 16 bits would be off by up to 2^-8 or 2^-11 of w |v|, which
a sum near zero does not shrink).  It has to hold for the same tokens behind a prefix."""
import pytest
import torch

from prefix_cases import Pool, call, no_prefixes, rows

pytestmark = pytest.mark.gpu


def exact(pool, pages, q, scale, n):
    """Attention of q [B, 1, Hq, D] to the n tokens of the tables' first row, in 64 bits; and sum w |v|."""
    G = q.shape[2] // pool.H
    out, size = (torch.zeros(q.shape, dtype=torch.float64, device="cuda") for _ in range(2))
    for h in range(pool.H):
        k, v = (pool.values(pages, 0, h, n, x) for x in "kv")
        w = torch.softmax(q[:, 0, h * G:(h + 1) * G].double() @ k.T * scale, -1)
        out[:, 0, h * G:(h + 1) * G], size[:, 0, h * G:(h + 1) * G] = w @ v, w @ v.abs()
    return out, size


def within(got, want):
    bad = (got.double() - want).abs() > 1e-2 + 1e-2 * want.abs()
    assert not bad.any(), (int(bad.sum()), float(((got.double() - want).abs() / (1e-2 + 1e-2 * want.abs())).max()))


def cancelling(pool, pages, q, n, tokens, seed):
    """Three tokens with scores near 24, their values such that each dimension's sum nearly cancels."""
    scale = q.shape[-1] ** -0.5
    g = torch.Generator().manual_seed(seed)
    G, D = q.shape[2] // pool.H, q.shape[3]
    for h in range(pool.H):
        qv = q[0, 0, h * G].double()
        ids = pool.row(pages, 0, h)
        at = [(ids[t // 16], h, t % 16) for t in tokens]
        for (page, _, slot), score in zip(at, (24.0, 24.6, 25.0)):
            row = qv * (score / (scale * (qv @ qv)))
            if pool.fp8:
                pool.cache.k_scale[page, h] = 2.0 ** -6
                pool.cache.k_pages[page, h, slot] = (row * 64).clamp(-448, 448).float().to(torch.float8_e4m3fn).view(torch.uint8)
            else:
                pool.cache.k_pages[page, h, slot] = row.to(torch.bfloat16)
        if pool.fp8:  # the other tokens of those units, and values on a grid
            for page in {int(p) for p, _, _ in at}:
                pool.cache.v_scale[page, h] = 0.25
        k = pool.values(pages, 0, h, n, "k")
        w = torch.softmax(q[0, 0, h * G].double() @ k.T * scale, -1)[list(tokens)].cpu()
        codes = torch.arange(0x68, 0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn).double() * 0.25  # 16 .. 112
        grid = torch.cat((codes, -codes))
        v2 = grid[torch.randint(0, len(grid), (D,), generator=g)]
        total = (w[0] * grid[:, None] + w[1] * grid).flatten()[None] + w[2] * v2[:, None]
        best = total.abs().argmin(-1)
        values = torch.stack((grid[best // len(grid)], grid[best % len(grid)], v2)).cuda()
        for (page, _, slot), v in zip(at, values):
            if pool.fp8:
                pool.cache.v_pages[page, h, slot] = (v * 4).float().to(torch.float8_e4m3fn).view(torch.uint8)
            else:
                pool.cache.v_pages[page, h, slot] = v.to(torch.bfloat16)
    return scale


@pytest.mark.parametrize("requests", [1, 40])
@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("fp8", [False, True])
def test_values_that_cancel(fp8, D, requests):
    for seed in range(4):
        n = 700
        pool = Pool(200, 2, D, fp8, seed=seed)
        pre = pool.tables([n])
        # keys that leave the other scores near 0
        ids = pool.row(pre, 0, 0)[:44]
        if fp8:
            pool.cache.k_scale[ids] = 2.0 ** -14
        else:
            pool.cache.k_pages[ids] = (pool.cache.k_pages[ids].float() * 0.01).to(torch.bfloat16)
        q = rows(pool.g, 1, 1, 2, D, outliers=0).repeat_interleave(8, 2).expand(requests, -1, -1, -1).contiguous()
        tokens = [(5, 9, 14), (130, 133, 250), (17, 300, 699), (255, 256, 511)][seed]
        scale = cancelling(pool, pre, q, n, tokens, seed)
        want, size = exact(pool, pre, q, scale, n)
        assert want.abs().mean() < 2 and size.mean() > 20
        # as own tokens, by the split kernel
        within(call(pool, pre, no_prefixes(2), [-1], q[:1], scale)[0], want[:1])
        out, flags = call(pool, None, pre, [0] * requests, q, scale)
        assert not flags[:requests].any()
        within(out, want)


@pytest.mark.parametrize("D", [128, 64])
def test_queries_far_apart(D):
    """FP8 pools: one element of a query 2,000 to 8,000 times as large as the others, whose products with the
    keys decide all the same (the key's elements there are zero): queries are exact for such elements."""
    for k, far in enumerate((2.0 ** 9, 2.0 ** 10, 2.0 ** 11)):
        pool = Pool(200, 2, D, True, seed=50 + k)
        pre = pool.tables([500])
        live = pool.row(pre, 0, 0)[:32]
        pool.cache.k_pages[live, :, :, 11] = 0
        pool.cache.k_scale[live] = 0.05
        q = rows(pool.g, 3, 1, 16, D, outliers=0)
        q = q.sign() * (q.abs().clamp(0.5, 4))
        q[..., 11] = 4 * far
        want, _ = exact(pool, pre, q, D ** -0.5, 500)
        out, flags = call(pool, None, pre, [0, 0, 0], q, D ** -0.5)
        assert not flags[:3].any()
        within(out, want)
