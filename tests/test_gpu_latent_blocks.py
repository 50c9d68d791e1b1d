"""pfkv_latent_decode_attn with three and more blocks of 128 rows a request (heads times
query tokens): their parts, flags and merge."""
import pytest
import torch

import test_gpu_latent_decode as D
from latent_cases import PAGE, gen, i32, latent_pool, rows, tables

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,kq,lens", [
    (128, 4, [300, 5, 129, 4000]),                   # 512 rows
    (128, 3, [2, 0, 64]),
    (100, 7, [900, 6]),                              # 700 rows
    (160, 3, [257] * 50),                            # 480
    (1, 400, [500, 399, 1]),
    (600, 1, [1000, 77]),
])
def test_rows(H, kq, lens, fp8):
    g = gen(H + kq)
    bt, num = tables([(n + PAGE - 1) // PAGE for n in lens], seed=5)
    cache = latent_pool(g, num, fp8)
    qc, qr = rows(g, len(lens), kq, H, 512, outliers=0), rows(g, len(lens), kq, H, 64, outliers=0)
    out, fl = D.run(cache, bt, lens, qc, qr)
    assert not any(fl)
    few = list(range(len(lens)))[:6]
    D.check(cache, bt[few], lens[:6], qc[few], qr[few], out[few])
    again, _ = D.run(cache, bt, lens, qc, qr)
    assert torch.equal(out, again)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_refused_page_of_one_block_zeroes_them_all(fp8):
    """Pages that only the last tiles of a request name: each block's parts look them up,
    in whichever cluster they lie."""
    g = gen(105)
    lens = [1500, 4000, 200, 1600, 128]
    bt, num = tables([(n + PAGE - 1) // PAGE for n in lens], seed=6)
    cache = latent_pool(g, num, fp8, tags=True)
    expected = cache.page_tags[bt.long().clamp(min=0)].contiguous()
    good = bt.clone()
    bt[1, 249] = num + 3                             # the last page
    expected[3, 0] ^= 4                              # the first one
    qc, qr = rows(g, 5, 4, 128, 512, outliers=0), rows(g, 5, 4, 128, 64, outliers=0)
    out, fl = D.run(cache, bt, i32(lens), qc, qr, max_len=4000, expected=expected)
    assert fl == [0, 2, 0, 1, 0]
    D.check(cache, good, lens, qc, qr, out, skip=(1, 3))
