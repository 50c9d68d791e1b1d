"""The latent calls as a serving program uses them: prompts are appended to the
cache and attended in the expanded form, their prefix read back by the gather;
then tokens are decoded in the absorbed form.  The two forms of the same tokens
agree, and both agree with attention in 64 bits on what the cache holds."""
import pytest
import torch

from latent_cases import (BF16, F16, SCALE, close, flags_for, gen, i32, latent_pool, latent_values, pages, rows,
                          score_error, softmax_attend, tables)
from paged_fp8_kv_decode_gb300 import latent as L
from paged_fp8_kv_decode_gb300 import rope as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
def test_prompt_then_decode(fp8):
    g = gen(71)
    H, Bn, pre, new = 16, 3, [48, 0, 100], [70, 33, 1]
    n = [a + b for a, b in zip(pre, new)]
    bt, num = tables([(x + 1 + 15) // 16 for x in n], seed=1)
    cache = latent_pool(g, num, fp8)
    rope = R.Rope((10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)).float().cuda(), True)
    # up-projections of keys and values
    up = (torch.randn(H, 512, 256, generator=g, device="cuda") / 512 ** 0.5).to(torch.bfloat16)

    def starts(v):
        s = [0]
        for x in v:
            s.append(s[-1] + x)
        return s

    c, r = rows(g, sum(n), 512, outliers=0), rows(g, sum(n), 64, outliers=0)
    q = rows(g, sum(n), H, 192, outliers=0)
    ns = starts(n)
    fl = flags_for(Bn)
    # two rounds of appends: the prefixes, then the rest of the prompts
    for lo, hi in (([0] * Bn, pre), (pre, n)):
        take = torch.cat([torch.arange(ns[b] + lo[b], ns[b] + hi[b]) for b in range(Bn)]).cuda()
        cnt = [h - a for a, h in zip(lo, hi)]
        qq = q[take][..., 128:].contiguous()
        L.pfkv_latent_append(cache, pages(bt, i32(hi)), rope, i32(lo), c[take], r[take], qq, qq,
                             row_starts=i32(starts(cnt)), max_new_tokens=max(cnt), flags=fl)
    # `qq` now holds the turned queries of the second round; read back everything and expand it
    c_all, r_all = torch.empty_like(c), torch.empty_like(r)
    L.pfkv_latent_gather(cache, pages(bt, i32(n)), i32(ns), max(n), c_all, r_all, flags=fl)
    kv = torch.einsum("td,hde->the", c_all.float(), up.float()).to(torch.bfloat16)
    out = torch.empty(sum(new), H, 128, dtype=torch.bfloat16, device="cuda")
    qn = q[take][..., :128]
    L.pfkv_latent_prefill_attn(qn, qq, kv[..., :128], r_all, kv[..., 128:], i32(starts(new)), i32(ns), max(new), SCALE,
                               True, out, flags=fl)
    # the same queries in the absorbed form, one request at a time; each form against
    # 64 bits on the operands that it was given, and the two against each other
    both = []
    for b in range(Bn):
        s, k = slice(starts(new)[b], starts(new)[b + 1]), slice(ns[b], ns[b + 1])
        qc = torch.einsum("the,hde->thd", qn[s].float(), up[..., :128].float()).to(torch.bfloat16)[None]
        o = torch.empty_like(qc)
        pg = pages(bt[b:b + 1], i32(n[b:b + 1]))
        ws = torch.empty(L.pfkv_latent_decode_workspace_size(cache, pg, H, new[b], n[b]), dtype=torch.uint8, device="cuda")
        L.pfkv_latent_decode_attn(cache, pg, qc, qq[s][None], SCALE, n[b], ws, o, flags=fl)
        c64, r64 = latent_values(cache, bt[b], n[b])
        seen = torch.ones(new[b], n[b], dtype=torch.bool, device="cuda").tril(n[b] - new[b])
        for h in range(H):
            for got, q64, k64, v64, step in (
                    (out[s, h], torch.cat((qn[s, h], qq[s, h]), 1), torch.cat((kv[k, h, :128], r_all[k]), 1),
                     kv[k, h, 128:], BF16),
                    (o[0, :, h], torch.cat((qc[0, :, h], qq[s, h]), 1), torch.cat((c64, r64), 1), c64,
                     F16 if fp8 else BF16)):
                q64, k64 = q64.double(), k64.double()
                x = torch.where(seen, q64 @ k64.T * SCALE, -torch.inf)
                ref, tol = softmax_attend(x, v64.double(), step, score_error(q64, k64, SCALE))
                close(got, ref, tol, (b, h))
        both.append((out[s].double(), torch.einsum("thd,hde->the", o[0].double(), up[..., 128:].double())))
    assert not fl.any()
    # The forms round different operands to bf16 (expanded keys and values; absorbed
    # queries and results), independently: the scores' errors have a deviation of
    # SCALE 2^-8 sqrt(sum (q k)^2 / 3) < 0.01, results one of about 2^-9 of their
    # size a rounding.  2^-5 of the norm is several times all of them together.
    x, y = (torch.cat([p[i] for p in both]) for i in (0, 1))
    assert float((x - y).norm() / x.norm()) < 2.0 ** -5
