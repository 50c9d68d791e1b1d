"""pfkv_latent_decode_attn on batches of short requests: tiles of 64 tokens or fewer,
of which the second CTA of a pair brings no keys, many of them in a row in every
cluster; and tiles whose pages are all refused."""
import pytest
import torch

import test_gpu_latent_decode as D
from latent_cases import PAGE, gen, latent_pool, rows, tables

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,kq", [(16, 1), (128, 2)])
def test_many_tiles_of_few_tokens(H, kq, fp8):
    g = gen(81)
    lens = [(7 * i) % 64 + 1 for i in range(1500)]   # some twenty tiles a cluster
    bt, num = tables([(n + PAGE - 1) // PAGE for n in lens], seed=2)
    cache = latent_pool(g, num, fp8)
    qc, qr = rows(g, len(lens), kq, H, 512, outliers=0), rows(g, len(lens), kq, H, 64, outliers=0)
    out, fl = D.run(cache, bt, lens, qc, qr)
    assert not any(fl)
    few = list(range(0, len(lens), 41))
    D.check(cache, bt[few], [lens[b] for b in few], qc[few], qr[few], out[few])
    for _ in range(20):
        again, fl = D.run(cache, bt, lens, qc, qr)
        assert not any(fl) and torch.equal(out, again)


@pytest.mark.parametrize("fp8", [False, True])
def test_tiles_whose_pages_are_all_refused(fp8):
    """Requests of a few whole tiles without one page of the pool, between sound ones:
    their tiles bring no bytes at all."""
    g = gen(82)
    lens = [(384, 40, 512, 128)[i % 4] for i in range(400)]
    bt, num = tables([(n + PAGE - 1) // PAGE for n in lens], seed=3)
    cache = latent_pool(g, num, fp8)
    good = bt.clone()
    refused = [b for b in range(len(lens)) if b % 3 == 1]
    bt[refused] = num + 9
    qc, qr = rows(g, len(lens), 1, 32, 512, outliers=0), rows(g, len(lens), 1, 32, 64, outliers=0)
    for _ in range(10):
        out, fl = D.run(cache, bt, lens, qc, qr)
        assert fl == [2 if b % 3 == 1 else 0 for b in range(len(lens))]
        assert not out[refused].any()
    few = [b for b in range(0, len(lens), 7) if b % 3 != 1]
    D.check(cache, good[few], [lens[b] for b in few], qc[few], qr[few], out[few])
