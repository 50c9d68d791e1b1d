"""Values of a prefix that are very large or small."""
import pytest
import torch

from prefix_cases import B, Pool, call, close, rows
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
