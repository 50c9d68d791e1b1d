"""No kernel of the rotary append or the latent cache writes outside the buffers that a
call is given: pools, scales, results, flags and workspace lie between guards of random
bytes, which are unchanged after the call, and the guarded call's results are those of an
unguarded one."""
import pytest
import torch

import test_gpu_latent_prefill as P
from latent_cases import PAGE, SCALE, flags_for, gen, i32, latent_pool, pages, rows, tables
from paged_fp8_kv_decode_gb300 import binding as B
from paged_fp8_kv_decode_gb300 import latent as L
from paged_fp8_kv_decode_gb300 import rope as R
from test_gpu_canary import Guarded

pytestmark = pytest.mark.gpu


def both(call, **buffers):
    """Runs call(buffers) on copies of the buffers and on guarded ones."""
    plain = {k: t.clone() for k, t in buffers.items() if t is not None}
    guarded = {k: Guarded(t, 100 + i) for i, (k, t) in enumerate(buffers.items()) if t is not None}
    call(**{k: plain.get(k) for k in buffers})
    call(**{k: guarded[k].t if k in guarded else None for k in buffers})
    torch.cuda.synchronize()
    for k, g in guarded.items():
        assert g.intact(), k
        if k not in ("ws", "flags"):
            assert torch.equal(g.t.view(torch.uint8), plain[k].view(torch.uint8)), k
    return plain


def freq(n):
    return R.Rope((10000.0 ** (-torch.arange(n, dtype=torch.float64) / n)).float().cuda(), True)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,Hkv,Hq", [(128, 3, 7), (64, 1, 5)])
def test_rope_append(D, Hkv, Hq, fp8):
    g = gen(101)
    at, new = [0, 5, 33, 160], [1, 40, 3, 17]
    starts = P.starts_of(new)
    n = [a + b for a, b in zip(at, new)]
    bt, num = tables([(x + PAGE - 1) // PAGE for x in n], seed=1, spare=0)
    pool = rows(g, num, Hkv, PAGE, D).view(torch.uint8)[..., :D].contiguous() if fp8 else rows(g, num, Hkv, PAGE, D)
    scale = torch.rand(num, Hkv, generator=g, device="cuda") if fp8 else None
    k, v, q = (rows(g, sum(new), h, D) for h in (Hkv, Hkv, Hq))

    def call(k_pages, v_pages, k_scale, v_scale, q_out, flags):
        R.pfkv_rope_append(B.Cache(k_pages, v_pages, k_scale, v_scale), pages(bt, i32(n)), freq(D // 4), i32(at), k, v, q, q_out,
                           row_starts=i32(starts), max_new_tokens=max(new), flags=flags)
    both(call, k_pages=pool, v_pages=pool, k_scale=scale, v_scale=scale, q_out=torch.zeros_like(q),
         flags=torch.zeros(4, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H", [1, 19])
def test_latent_append_and_gather(H, fp8):
    g = gen(102)
    at, new = [0, 5, 33, 160, 15], [1, 40, 3, 17, 2]
    n = [a + b for a, b in zip(at, new)]
    bt, num = tables([(x + PAGE - 1) // PAGE for x in n], seed=2, spare=0)
    pool = latent_pool(g, num, fp8)
    c, r, q = rows(g, sum(new), 512), rows(g, sum(new), 64), rows(g, sum(new), H, 64)

    def append(c_pages, r_pages, c_scale, q_out, flags):
        L.pfkv_latent_append(L.LatentCache(c_pages, r_pages, c_scale), pages(bt, i32(n)), freq(32), i32(at), c, r, q, q_out,
                             row_starts=i32(P.starts_of(new)), max_new_tokens=max(new), flags=flags)
    got = both(append, c_pages=pool.c_pages, r_pages=pool.r_pages, c_scale=pool.c_scale, q_out=torch.zeros_like(q),
               flags=torch.zeros(8, dtype=torch.uint8, device="cuda"))
    cache = L.LatentCache(got["c_pages"], got["r_pages"], got.get("c_scale"))

    def gather(c_out, r_out, flags):
        L.pfkv_latent_gather(cache, pages(bt, i32(n)), i32(P.starts_of(n)), max(n), c_out, r_out, flags=flags)
    both(gather, c_out=rows(g, sum(n), 512), r_out=rows(g, sum(n), 64), flags=torch.zeros(8, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,kq,lens", [
    (33, 4, [1, 700, 130]),                          # 132 rows, parts merged by four warps
    (33, 4, [1, 700, 130, 0, 63, 2000, 5, 9, 400, 77]),  # and by one
    (1, 1, [9000]),
    (5, 1, [3000] * 70),                             # more requests than pairs of CTAs
    (128, 3, [500, 129]),
])
def test_decode(H, kq, lens, fp8):
    g = gen(103)
    bt, num = tables([(n + PAGE - 1) // PAGE for n in lens], seed=3, spare=0)
    cache = latent_pool(g, num, fp8)
    qc, qr = rows(g, len(lens), kq, H, 512, outliers=0), rows(g, len(lens), kq, H, 64, outliers=0)
    pg = pages(bt, i32(lens))
    size = L.pfkv_latent_decode_workspace_size(cache, pg, H, kq, max(lens))

    def call(ws, out, flags):
        L.pfkv_latent_decode_attn(cache, pg, qc, qr, SCALE, max(lens), ws, out, flags=flags)
    got = both(call, ws=torch.empty(size, dtype=torch.uint8, device="cuda"), out=torch.zeros_like(qc),
               flags=flags_for(len(lens)))
    assert not got["flags"].any()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,nq,pre", [(1, [1], [0]), (3, [127, 1, 300], [0, 200, 5]), (20, [129] * 33, [3] * 33)])
def test_prefill(H, nq, pre, causal):
    g = gen(104)
    nk = [a + b for a, b in zip(nq, pre)]
    x = P.inputs(g, sum(nq), sum(nk), H)

    def call(out, flags):
        L.pfkv_latent_prefill_attn(x["qn"], x["qr"], x["kn"], x["kr"], x["v"], i32(P.starts_of(nq)), i32(P.starts_of(nk)),
                                   max(nq), SCALE, causal, out, flags=flags)
    got = both(call, out=torch.zeros_like(x["qn"]), flags=flags_for(len(nq)))
    assert not got["flags"].any()
