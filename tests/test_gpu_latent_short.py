"""pfkv_latent_decode_attn on batches of short requests: tiles of 64 tokens or fewer,
of which the second CTA of a pair brings no keys, many of them in a row in every
cluster."""
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
