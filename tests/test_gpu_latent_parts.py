"""How the latent kernels share out their work, at the edges: lists of requests of
very different lengths whose parts begin and end anywhere in a cluster's range,
NaN among many parts, and prompts with more tiles than the GPU has
multiprocessors."""
import pytest
import torch

import test_gpu_latent_decode as D
import test_gpu_latent_prefill as P
from latent_cases import PAGE, SCALE, gen, i32, latent_pool, pages, rows, tables
from paged_fp8_kv_decode_gb300 import binding as B
from paged_fp8_kv_decode_gb300 import latent as L

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,kq,lens", [
    (16, 1, [128] * 300),                            # more parts than clusters, a tile each
    (128, 1, [1, 0, 129, 2000, 1, 1, 640, 0, 127, 5000, 16]),
    (64, 3, [3, 300, 0, 1, 1500] * 9),               # two row blocks a request
    (8, 1, [9000] + [1] * 100),                      # one long among short ones
    (8, 1, [1] * 100 + [9000]),
    (128, 2, [257, 256, 255]),                       # fewer tiles than clusters
    (16, 1, [1]),
])
def test_parts_anywhere_in_a_range(H, kq, lens, fp8):
    g = gen(len(lens) + H)
    bt, num = tables([(n + PAGE - 1) // PAGE for n in lens], seed=3)
    cache = latent_pool(g, num, fp8)
    qc, qr = rows(g, len(lens), kq, H, 512, outliers=0), rows(g, len(lens), kq, H, 64, outliers=0)
    out, fl = D.run(cache, bt, lens, qc, qr)
    assert not any(fl)
    D.check(cache, bt, lens, qc, qr, out)
    again, _ = D.run(cache, bt, lens, qc, qr)
    assert torch.equal(out, again)                   # the split and the order of sums are the call's alone


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("many", [1, 40])
def test_a_nan_in_a_visible_token_reaches_its_request_alone(many, fp8):
    lens = [12000] + [300] * (many - 1)
    g = gen(7)
    bt, num = tables([(n + PAGE - 1) // PAGE for n in lens], seed=5)
    cache = latent_pool(g, num, fp8)
    qc, qr = rows(g, many, 1, 16, 512, outliers=0), rows(g, many, 1, 16, 64, outliers=0)
    page = int(bt[0, 700])                           # of one of the first request's many parts
    if fp8:
        cache.c_pages[page, 3, 5] = 0x7F
    else:
        cache.c_pages[page, 3, 5] = float("nan")
    out, fl = D.run(cache, bt, lens, qc, qr)
    assert not any(fl)
    assert out[0].isnan().all()
    assert not out[1:].isnan().any()


@pytest.mark.parametrize("H,nq,pre", [
    (64, [1, 130, 257, 0, 512, 300, 129], [0, 700, 3, 40, 0, 129, 1000]),
    (16, [64] * 40, [0, 5] * 20),                    # one tile of rows an item, many items a CTA
    (3, [2000], [0]),
])
def test_many_items_of_every_length(H, nq, pre):
    g = gen(H + len(nq))
    nk = [q + p for q, p in zip(nq, pre)]
    qs, ks = P.starts_of(nq), P.starts_of(nk)
    x = P.inputs(g, sum(nq), sum(nk), H)
    out, fl = P.run(x, qs, ks, max(nq))
    assert not any(fl)
    for b in range(len(nq)):
        P.check(x, (qs[b], qs[b + 1]), (ks[b], ks[b + 1]), out, heads=[0, H // 2, H - 1])


@pytest.mark.parametrize("causal", [True, False])
def test_a_negative_scale(causal):
    g = gen(11)
    nq, nk = [200, 77], [200, 300]
    qs, ks = P.starts_of(nq), P.starts_of(nk)
    x = P.inputs(g, sum(nq), sum(nk), 4)
    out, _ = P.run(x, qs, ks, max(nq), causal=causal, scale=-SCALE)
    for b in range(2):
        P.check(x, (qs[b], qs[b + 1]), (ks[b], ks[b + 1]), out, causal, -SCALE)


def test_a_nan_key_reaches_the_rows_that_see_it():
    g = gen(12)
    nq = [300, 140]
    qs = P.starts_of(nq)
    x = P.inputs(g, sum(nq), sum(nq), 2)
    x["kn"][150, 1, 7] = float("nan")                # of the first request
    out, fl = P.run(x, qs, qs, max(nq))
    assert not any(fl)
    assert out[150:300, 1].isnan().all()
    bad = out.isnan().any(-1)
    bad[150:300, 1] = False
    assert not bad.any()


@pytest.mark.parametrize("bound", [60, 4096, 1 << 30])
def test_a_loose_bound_of_the_queries(bound):
    g = gen(13)
    nq = [60, 1, 33, 0] * 16
    qs = P.starts_of(nq)
    x = P.inputs(g, sum(nq), sum(nq), 32)
    out, fl = P.run(x, qs, qs, bound)
    assert not any(fl)
    for b in range(len(nq)):
        P.check(x, (qs[b], qs[b + 1]), (qs[b], qs[b + 1]), out, heads=[0, 31])


def test_no_queries_at_all_and_a_bound_of_none():
    g = gen(14)
    x = P.inputs(g, 0, 20, 2)
    _, fl = P.run(x, [0, 0, 0], [0, 5, 20], 7)
    assert fl == [0, 0]
    x = P.inputs(g, 9, 9, 2)
    out, fl = P.run(x, [0, 0, 9], [0, 0, 9], 0)
    assert fl == [0, B.PFKV_FLAG_BAD_LENGTH] and (out == 7.0).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("scale", [0.0, -SCALE])
def test_scales_of_zero_and_below(scale, fp8):
    lens = [300, 5]
    g = gen(15)
    bt, num = tables([(n + PAGE - 1) // PAGE for n in lens], seed=9)
    cache = latent_pool(g, num, fp8)
    qc, qr = rows(g, 2, 1, 16, 512, outliers=0), rows(g, 2, 1, 16, 64, outliers=0)
    out, _ = D.run(cache, bt, lens, qc, qr, scale=scale)
    D.check(cache, bt, lens, qc, qr, out, scale=scale)
    x = P.inputs(g, 140, 140, 3)
    out, _ = P.run(x, [0, 140], [0, 140], 140, scale=scale)
    P.check(x, (0, 140), (0, 140), out, scale=scale)


def test_calls_on_two_streams_at_once():
    """Calls of both attentions in flight together, each with its own workspace and
    arrays, give what they give alone."""
    g = gen(16)
    lens = [3000, 40, 700]
    bt, num = tables([(n + PAGE - 1) // PAGE for n in lens], seed=11)
    cache = latent_pool(g, num, True)
    qc, qr = rows(g, 3, 1, 32, 512, outliers=0), rows(g, 3, 1, 32, 64, outliers=0)
    want, _ = D.run(cache, bt, lens, qc, qr)
    x = P.inputs(g, 900, 900, 8)
    alone, _ = P.run(x, [0, 900], [0, 900], 900)
    pg = pages(bt, i32(lens))
    size = L.pfkv_latent_decode_workspace_size(cache, pg, 32, 1, 3000)
    starts = i32([0, 900])
    streams = [torch.cuda.Stream() for _ in range(3)]
    spaces = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs, prompt = [torch.zeros_like(qc) for _ in range(2)], torch.zeros_like(alone)
    torch.cuda.synchronize()
    for _ in range(5):
        for s, ws, o in zip(streams, spaces, outs):
            L.pfkv_latent_decode_attn(cache, pg, qc, qr, SCALE, 3000, ws, o, stream=s)
        L.pfkv_latent_prefill_attn(x["qn"], x["qr"], x["kn"], x["kr"], x["v"], starts, starts, 900, SCALE, True, prompt,
                                   stream=streams[2])
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)
    assert torch.equal(prompt, alone)


def test_tensors_elsewhere_are_refused(monkeypatch):
    g = gen(17)
    x = P.inputs(g, 5, 5, 2)
    with pytest.raises(ValueError):
        P.run(dict(x, qn=x["qn"].cpu().pin_memory()), [0, 5], [0, 5], 5, out=torch.zeros_like(x["qn"]))
    bt, num = tables([1])
    cache = latent_pool(g, num, False)
    lens = i32([3])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)   # as if another device were current
    with pytest.raises(ValueError):
        L.pfkv_latent_prefill_attn(x["qn"], x["qr"], x["kn"], x["kr"], x["v"], lens, lens, 5, 1.0, True, x["qn"], stream=0)
    lens2 = torch.cat((lens, lens))
    with pytest.raises(ValueError):
        L.pfkv_latent_gather(cache, pages(bt, lens), lens2, 3, torch.zeros(3, 512, dtype=torch.bfloat16, device="cuda:0"),
                             torch.zeros(3, 64, dtype=torch.bfloat16, device="cuda:0"), stream=0)
