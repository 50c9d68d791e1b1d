"""The latent calls in their order, each with flags of its own: all zero for sound tables,
and the request with a refused page flagged by every call that meets it."""
import pytest
import torch

from latent_cases import SCALE, flags_for, gen, i32, latent_pool, pages, rows, tables
from paged_fp8_kv_decode_gb300 import latent as L
from paged_fp8_kv_decode_gb300 import rope as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("refused", [None, 1])
def test_flags_of_every_call(refused, fp8):
    g = gen(106)
    H, Bn, n = 16, 3, [70, 33, 101]
    bt, num = tables([(x + 16) // 16 for x in n], seed=7)
    if refused is not None:
        bt[refused, 1] = num + 1
    want = [2 if b == refused else 0 for b in range(Bn)]
    cache = latent_pool(g, num, fp8)
    rope = R.Rope((10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)).float().cuda(), True)
    starts = [0, 70, 103, 204]
    c, r, q = rows(g, 204, 512), rows(g, 204, 64), rows(g, 204, H, 64)

    def flags(call):
        fl = flags_for(Bn)
        call(fl)
        torch.cuda.synchronize()
        return fl[:Bn].tolist()

    tables_of = lambda lens: pages(bt, i32(lens))  # noqa: E731
    assert flags(lambda fl: L.pfkv_latent_append(cache, tables_of(n), rope, i32([0] * 3), c, r, q, q, row_starts=i32(starts),
                                                 max_new_tokens=101, flags=fl)) == want
    c_all, r_all = torch.empty_like(c), torch.empty_like(r)
    assert flags(lambda fl: L.pfkv_latent_gather(cache, tables_of(n), i32(starts), 101, c_all, r_all, flags=fl)) == want
    kv = rows(g, 204, H, 256, outliers=0)
    out = torch.empty(204, H, 128, dtype=torch.bfloat16, device="cuda")
    qn = rows(g, 204, H, 128, outliers=0)
    assert flags(lambda fl: L.pfkv_latent_prefill_attn(qn, q, kv[..., :128], r_all, kv[..., 128:], i32(starts), i32(starts), 101,
                                                       SCALE, True, out, flags=fl)) == [0] * Bn  # it reads no pages
    # a step: one token more, then attention over the cache
    one = [rows(g, Bn, 1, *s) for s in ((512,), (64,), (H, 64))]
    more = [x + 1 for x in n]
    assert flags(lambda fl: L.pfkv_latent_append(cache, tables_of(more), rope, i32(n), *one, one[2], flags=fl)) == [0] * Bn
    qc = rows(g, Bn, 1, H, 512, outliers=0)
    ws = torch.empty(L.pfkv_latent_decode_workspace_size(cache, tables_of(more), H, 1, 102), dtype=torch.uint8, device="cuda")
    o = torch.full_like(qc, 7.0)
    assert flags(lambda fl: L.pfkv_latent_decode_attn(cache, tables_of(more), qc, one[2], SCALE, 102, ws, o, flags=fl)) == want
    for b in range(Bn):
        assert o[b].any() == (b != refused)


def test_flags_of_a_replayed_graph():
    """A captured prompt call writes its flags at every replay, whatever they held."""
    g = gen(107)
    x = {k: rows(g, 60, *s, outliers=0) for k, s in dict(qn=(4, 128), qr=(4, 64), kn=(4, 128), kr=(64,), v=(4, 128)).items()}
    qs, out, fl = i32([0, 20, 60]), torch.zeros(60, 4, 128, dtype=torch.bfloat16, device="cuda"), flags_for(2)
    call = lambda: L.pfkv_latent_prefill_attn(x["qn"], x["qr"], x["kn"], x["kr"], x["v"], qs, qs, 50, SCALE, True, out, flags=fl)  # noqa: E731
    call()
    want = out.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call()
    for starts, flags in (([0, 20, 60], [0, 0]), ([0, 20, 61], [0, 4]), ([0, 51, 60], [4, 0]), ([0, 20, 60], [0, 0])):
        fl.fill_(0x55)
        out.fill_(7.0)
        qs.copy_(i32(starts))
        graph.replay()
        torch.cuda.synchronize()
        assert fl[:2].tolist() == flags and (fl[2:] == 0x55).all()
        if starts == [0, 20, 60]:
            assert torch.equal(out, want)
