"""Pools and arrays whose offsets pass 32 bits: pages beyond 4 GB, rows beyond 2^31
elements."""
import pytest
import torch

import test_gpu_latent_decode as D
import test_gpu_latent_prefill as P
from latent_cases import BF16, PAGE, SCALE, close, flags_for, gen, i32, latent_values, pages, rows
from paged_fp8_kv_decode_gb300 import latent as L
from paged_fp8_kv_decode_gb300 import rope as R

pytestmark = pytest.mark.gpu

PAGES = 600_000                                      # 4.9 GB of codes, 9.8 GB of bf16


@pytest.mark.parametrize("fp8", [False, True])
def test_far_pages(fp8):
    g = gen(121)
    lens = [300, 40]
    num = [(n + PAGE) // PAGE for n in lens]
    bt = torch.zeros(2, max(num), dtype=torch.int32, device="cuda")
    bt[0, :num[0]] = PAGES - 1 - torch.arange(num[0], device="cuda")   # from the far end
    bt[1, :num[1]] = torch.arange(num[1], device="cuda") * 7 + (PAGES // 2 + 1)
    c = torch.empty(PAGES, PAGE, 512, dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    r = torch.empty(PAGES, PAGE, 64, dtype=torch.bfloat16, device="cuda")
    cache = L.LatentCache(c, r, torch.ones(PAGES, device="cuda") if fp8 else None)
    new_c, new_r = rows(g, sum(lens), 512), rows(g, sum(lens), 64)
    starts, fl = i32(P.starts_of(lens)), flags_for(2)
    L.pfkv_latent_append(cache, pages(bt, i32(lens)), R.Rope(torch.zeros(32, device="cuda")), i32([0, 0]), new_c, new_r,
                         row_starts=starts, max_new_tokens=max(lens), flags=fl)
    c_out, r_out = torch.empty_like(new_c), torch.empty_like(new_r)
    L.pfkv_latent_gather(cache, pages(bt, i32(lens)), starts, max(lens), c_out, r_out, flags=fl)
    assert not fl.any()
    assert torch.equal(r_out, new_r)                 # turned by nothing
    for b, (lo, hi) in enumerate(zip(P.starts_of(lens), P.starts_of(lens)[1:])):
        held, _ = latent_values(cache, bt[b], hi - lo)
        close(c_out[lo:hi], held, BF16 * held.abs() if fp8 else 0.0, "gathered")
        if not fp8:
            assert torch.equal(c_out[lo:hi], new_c[lo:hi])
    qc, qr = rows(g, 2, 2, 20, 512, outliers=0), rows(g, 2, 2, 20, 64, outliers=0)
    out, fl = D.run(cache, bt, lens, qc, qr)
    assert not any(fl)
    D.check(cache, bt, lens, qc, qr, out)


def test_far_rows_of_prompts():
    """Head and row strides that put the last rows beyond 2^31 elements."""
    g = gen(122)
    n, H, gap = 300, 3, 1 << 30
    big = torch.empty(2 * gap + n * 512, dtype=torch.bfloat16, device="cuda")
    view = lambda at, width: big[at:].as_strided((n, H, width), (512, gap, 1))  # noqa: E731
    x = dict(qn=view(0, 128), kn=view(128, 128), v=view(256, 128), qr=rows(g, n, H, 64, outliers=0),
             kr=rows(g, n, 64, outliers=0))
    for k in ("qn", "kn", "v"):
        x[k].copy_(rows(g, n, H, 128, outliers=0))
    out = view(384, 128)
    out.zero_()
    _, fl = P.run(x, [0, 100, n], [0, 100, n], 200, out=out)
    assert not any(fl)
    P.check(x, (0, 100), (0, 100), out)
    P.check(x, (100, n), (100, n), out)
