"""Page scales below 2^-100, zero and negative ones among them, are taken for 2^-100 by the
attention over an FP8 pool."""
import pytest
import torch

import test_gpu_latent_decode as D
from latent_cases import PAGE, gen, latent_pool, rows, tables
from paged_fp8_kv_decode_gb300 import latent as L

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("small", [-1.0, -1e-20, -0.0, 0.0, 1e-38, 2.0 ** -101])
def test_small_scales(small):
    g = gen(97)
    lens = [400, 37]
    bt, num = tables([(n + PAGE - 1) // PAGE for n in lens], seed=3)
    cache = latent_pool(g, num, True)
    qc, qr = rows(g, 2, 1, 24, 512, outliers=0), rows(g, 2, 1, 24, 64, outliers=0)
    at = [int(bt[0, 3]), int(bt[0, 24]), int(bt[1, 0])]
    outs = []
    for z in (small, 2.0 ** -100):
        scale = cache.c_scale.clone()
        scale[at] = z
        out, fl = D.run(L.LatentCache(cache.c_pages, cache.r_pages, scale), bt, lens, qc, qr)
        assert not any(fl)
        outs.append(out)
    assert torch.equal(*outs)
    D.check(L.LatentCache(cache.c_pages, cache.r_pages, scale), bt, lens, qc, qr, outs[1])
