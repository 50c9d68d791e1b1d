"""Values of a prefix that are very large or small, and V scales that are far apart."""
import pytest
import torch

from prefix_cases import B, F16, Pool, call, close, rows
from latent_cases import score_error, softmax_attend
from test_gpu_prefix_many import attend_alone

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("requests", [1, 40])
@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("size", [2.0 ** 100, 2.0 ** -90])
def test_large_values_bf16(size, D, requests):
    """Scores that grow from tile to tile, so that weights lie above the reference of the tiles before,
    with values near 2^100: what is summed stays finite.  Two hundred prefixes that name the same pages,
    so that a CTA has several tiles of one."""
    NP, n = 200, 1000
    pool = Pool(200, 1, D, False, seed=81)
    pre = pool.tables([n])
    ids = pool.row(pre, 0, 0)
    for t in range(0, n, 128):  # scores of a tile lie about 12 above those of the one before
        pool.cache.k_pages[ids[t // 16:(t + 128) // 16], 0, :, 0] = 15.0 * (t // 128)
    pool.cache.v_pages[ids] = (pool.cache.v_pages[ids].double() * size).to(torch.bfloat16)
    bt, lens = pre.block_tables.repeat(NP, 1, 1), pre.seq_lens.repeat(NP, 1)
    pre = B.Pages(NP, pre.max_pages, bt, bt.stride(0), 0, lens, 1, 0)
    pre.lens = [[n]] * NP
    of = [p for p in range(NP) for _ in range(requests)]
    q = rows(pool.g, len(of), 1, 8, D, outliers=0)
    q[..., 0] = 8.0
    want, tol = attend_alone(pool, pre, of, q, 0.1)
    out, flags = call(pool, None, pre, of, q, 0.1)
    assert not flags[:len(of)].any()
    close(out, want, tol, "out")


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("apart", [12, 20, 24])
@pytest.mark.parametrize("D", [128, 64])
def test_scales_apart_fp8(D, apart, zeros):
    """A V scale 2^apart above the others, of a page that gets no weight, or that holds zeros: a weight
    times its V scale is within 2^-11 of itself, or 2^-31 of the largest weight times that scale."""
    pool = Pool(200, 2, D, True, seed=82)
    pre, of, scale = pool.tables([700, 300]), [0, 1, 0], 0.125
    q = rows(pool.g, 3, 1, 8, D, outliers=0).abs()
    far = pool.row(pre, 0, 0)[9]
    pool.cache.v_scale[far] = pool.cache.v_scale[pool.row(pre, 0, 0)[:44]].amax(0) * 2.0 ** apart
    if zeros:
        pool.cache.v_pages[far] = 0
    else:  # scores far below all others
        pool.cache.k_pages[far], pool.cache.k_scale[far] = 0xFE, 1.0
    out, flags = call(pool, None, pre, of, q, scale)
    assert not flags[:3].any()
    for b, n in enumerate((700, 300, 700)):
        ids = pool.row(pre, of[b], 0)[:(n + 15) // 16]
        for h in range(2):
            heads = slice(4 * h, 4 * h + 4)
            k, v = (pool.values(pre, of[b], h, n, x) for x in "kv")
            qq = q[b, 0, heads].double()
            s = qq @ k.T * scale
            seen = s > s.amax() - 200  # (the far page's weights are zero in any number of bits)
            err = score_error(qq, k[seen.any(0)], scale) + 2.0 ** -17 * qq.abs().amax(-1) * k[seen.any(0)].abs().sum(-1).amax() * scale
            want, tol = softmax_attend(s, v, F16, err)
            p = torch.softmax(s, -1)
            vs = pool.cache.v_scale[ids, h].double()
            codes = v / vs.repeat_interleave(16)[:n, None]
            tol = tol + 2.0 ** -31 * p.amax(-1, keepdim=True) * vs.amax() * codes.abs().sum(0)
            close(out[b, 0, heads], want, tol, (b, h))
