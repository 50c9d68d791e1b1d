"""Per-step inputs and outputs in pinned host memory (new rows, queries, positions,
lengths, tables, results, flags): the calls read and write them there, with the results
that they have on device memory."""
import pytest
import torch

import test_gpu_latent_prefill as P
from latent_cases import PAGE, SCALE, flags_for, gen, i32, latent_pool, pages, rows, tables
from paged_fp8_kv_decode_gb300 import binding as B
from paged_fp8_kv_decode_gb300 import latent as L
from paged_fp8_kv_decode_gb300 import rope as R

pytestmark = pytest.mark.gpu


def there(t):
    return t.cpu().pin_memory()


def same(call, pools, inputs, outputs):
    """call(pools, inputs, outputs) with everything on the device and with inputs and outputs
    in host memory."""
    done = []
    for place in (lambda t: t.clone(), there):
        p, i, o = [t.clone() for t in pools], {k: place(t) for k, t in inputs.items()}, {k: place(t) for k, t in outputs.items()}
        call(p, i, o)
        torch.cuda.synchronize()
        done.append([t.cpu() for t in p] + [t.cpu() for t in o.values()])
    for a, b in zip(*done):
        assert torch.equal(a, b)
    return done[0]


def freq(n):
    return R.Rope((10000.0 ** (-torch.arange(n, dtype=torch.float64) / n)).float().cuda())


@pytest.mark.parametrize("fp8", [False, True])
def test_appends_and_gather(fp8):
    g = gen(111)
    at, new = [0, 5, 33], [20, 1, 40]
    n = [a + b for a, b in zip(at, new)]
    bt, num = tables([(x + PAGE - 1) // PAGE for x in n], seed=1)
    lat = latent_pool(g, num, fp8)
    pools = [t for t in (lat.c_pages, lat.r_pages, lat.c_scale) if t is not None]
    ins = dict(bt=bt, n=i32(n), at=i32(at), starts=i32(P.starts_of(new)), c=rows(g, 61, 512), r=rows(g, 61, 64), q=rows(g, 61, 3, 64))
    outs = dict(q=torch.zeros(61, 3, 64, dtype=torch.bfloat16, device="cuda"), flags=flags_for(3))

    def append(p, i, o):
        L.pfkv_latent_append(L.LatentCache(*p), pages(i["bt"], i["n"]), freq(32), i["at"], i["c"], i["r"], i["q"], o["q"],
                             row_starts=i["starts"], max_new_tokens=40, flags=o["flags"])
    same(append, pools, ins, outs)
    kv = rows(g, num, 2, PAGE, 64).view(torch.uint8)[..., :64].contiguous() if fp8 else rows(g, num, 2, PAGE, 64)
    kvs = [kv, kv] + ([torch.ones(num, 2, device="cuda")] * 2 if fp8 else [])
    ins.update(k=rows(g, 61, 2, 64), v=rows(g, 61, 2, 64))

    def rope_append(p, i, o):
        R.pfkv_rope_append(B.Cache(*p), pages(i["bt"], i["n"]), freq(32), i["at"], i["k"], i["v"], i["q"], o["q"],
                           row_starts=i["starts"], max_new_tokens=40, flags=o["flags"])
    same(rope_append, kvs, ins, outs)
    ins = dict(bt=bt, n=i32(n), starts=i32(P.starts_of(n)))
    bad = bt.clone()
    bad[1, 0] = -1
    for table, want in ((bt, [0, 0, 0]), (bad, [0, 2, 0])):
        outs = dict(flags=flags_for(3), c=rows(g, sum(n), 512), r=rows(g, sum(n), 64))

        def gather(p, i, o):
            L.pfkv_latent_gather(L.LatentCache(*p), pages(i["bt"], i["n"]), i["starts"], max(n), o["c"], o["r"], flags=o["flags"])
        got = same(gather, pools, dict(ins, bt=table), outs)
        assert got[len(pools)][:3].tolist() == want


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,kq,lens", [(16, 1, [900, 3, 70]), (128, 2, [5000, 130])])
def test_decode(H, kq, lens, fp8):
    g = gen(112)
    bt, num = tables([(x + PAGE - 1) // PAGE for x in lens], seed=2)
    lat = latent_pool(g, num, fp8)
    pools = [t for t in (lat.c_pages, lat.r_pages, lat.c_scale) if t is not None]
    ins = dict(bt=bt, n=i32(lens), qc=rows(g, len(lens), kq, H, 512), qr=rows(g, len(lens), kq, H, 64))
    outs = dict(o=torch.zeros_like(ins["qc"]), flags=flags_for(len(lens)))

    def call(p, i, o):
        cache, pg = L.LatentCache(*p), pages(i["bt"], i["n"])
        ws = torch.empty(L.pfkv_latent_decode_workspace_size(cache, pg, H, kq, max(lens)), dtype=torch.uint8, device="cuda")
        L.pfkv_latent_decode_attn(cache, pg, i["qc"], i["qr"], SCALE, max(lens), ws, o["o"], flags=o["flags"])
    same(call, pools, ins, outs)


def test_prefill_results():
    """The rows that it reads are device memory; starts, results and flags may lie elsewhere."""
    g = gen(113)
    nq = [300, 1, 70]
    x = P.inputs(g, 371, 371, 5)

    def call(p, i, o):
        L.pfkv_latent_prefill_attn(x["qn"], x["qr"], x["kn"], x["kr"], x["v"], i["s"], i["s"], 300, SCALE, True, o["o"],
                                   flags=o["flags"])
    same(call, [], dict(s=i32(P.starts_of(nq))), dict(o=torch.zeros_like(x["qn"]), flags=flags_for(3)))
