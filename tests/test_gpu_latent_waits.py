"""Waits inside the attention kernels that give up: the call ends, every request of it
that may lack rows is flagged, and the next call is sound.  The limit is an argument of
the self-test entry points, so no wait has to last."""
import pytest
import torch

import test_gpu_latent_decode as D
import test_gpu_latent_prefill as P
from latent_cases import PAGE, SCALE, flags_for, gen, i32, latent_pool, pages, rows, tables
from paged_fp8_kv_decode_gb300 import binding as B
from paged_fp8_kv_decode_gb300 import latent as L

pytestmark = pytest.mark.gpu

NEVER = 1000                                         # 0.2 ms at least: not in sound calls of microseconds


def prefill(tries, x, qs, ks, max_q, causal=True):
    out = torch.full(x["qn"].shape, 7.0, dtype=torch.bfloat16, device="cuda")
    fl = flags_for(len(qs) - 1)
    fl.fill_(0x55)
    L.pfkv_selftest_latent_prefill(tries, x["qn"], x["qr"], x["kn"], x["kr"], x["v"], i32(qs), i32(ks), max_q, SCALE, causal,
                                   out, flags=fl)
    torch.cuda.synchronize()
    assert (fl[len(qs) - 1:] == 0x55).all()
    return out, fl[:len(qs) - 1].tolist()


def test_prefill_flags_all_that_a_wait_left_unwritten():
    g = gen(91)
    nq = [300, 1, 64, 0, 700] * 40                   # several items a CTA
    qs = P.starts_of(nq)
    x = P.inputs(g, sum(nq), sum(nq), 8)
    want, fl = P.run(x, qs, qs, max(nq))
    assert not any(fl)
    for tries in (0, NEVER):
        out, fl = prefill(tries, x, qs, qs, max(nq))
        assert fl == [0 if tries else B.PFKV_FLAG_DEVICE_TIMEOUT] * len(nq)
        assert torch.equal(out, want) if tries else (out == 7.0).all()
    bad = list(qs)
    bad[3] = -5                                      # two requests whose rows are refused besides
    _, fl = prefill(0, x, bad, qs, max(nq))
    assert fl[:5] == [8, 8, 12, 12, 8]
    out, fl = P.run(x, qs, qs, max(nq))              # the call after it
    assert not any(fl) and torch.equal(out, want)


def test_prefill_refuses_a_limit_beyond_its_own():
    g = gen(92)
    x = P.inputs(g, 5, 5, 1)
    for tries in (-1, 100001):
        with pytest.raises(B.PfkvError) as e:
            prefill(tries, x, [0, 5], [0, 5], 5)
        assert e.value.status == B.PFKV_ERR_INVALID_ARG


def test_prefill_waits_that_last_as_long_as_an_item():
    """128 queries over a million keys have no second tile: its warps wait for the next
    item's scores, and that item for its place, while the first tile works for
    milliseconds.  A limit of 300 tries (1.2 ms at most) does not count there."""
    g = gen(93)
    H, nq, nk = 160, [128, 200], [1 << 20, 300]      # more pairs than multiprocessors: both on one CTA
    qs, ks = P.starts_of(nq), P.starts_of(nk)
    x = P.inputs(g, sum(nq), sum(nk), 1)
    x = {n: t if n == "kr" else t.expand(-1, H, -1) for n, t in x.items()}
    want = torch.zeros(sum(nq), H, 128, dtype=torch.bfloat16, device="cuda")
    _, fl = P.run(x, qs, ks, max(nq), out=want)
    assert not any(fl)
    P.check(x, (128, 328), (1 << 20, (1 << 20) + 300), want, heads=(0, 159))
    out, fl = prefill(300, x, qs, ks, max(nq))
    assert fl == [0, 0]
    assert torch.equal(out, want)


def decode(tries, cache, bt, lens, qc, qr):
    Bn, kq, H, _ = qc.shape
    pg = pages(bt, i32(lens))
    ws = torch.empty(L.pfkv_latent_decode_workspace_size(cache, pg, H, kq, max(lens)), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)
    out, fl = torch.full_like(qc, 7.0), flags_for(Bn)
    fl.fill_(0x55)
    L.pfkv_selftest_latent_decode(tries, cache, pg, qc, qr, SCALE, max(lens), ws, out, flags=fl)
    torch.cuda.synchronize()
    return out, fl[:Bn].tolist()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,kq", [(16, 1), (128, 2)])
def test_decode_flags_and_zeroes_what_a_wait_left(H, kq, fp8):
    g = gen(99)
    lens = [300, 1, 0, 5000, 64, 129] * 6
    bt, num = tables([(n + PAGE - 1) // PAGE for n in lens], seed=6)
    cache = latent_pool(g, num, fp8)
    qc, qr = rows(g, len(lens), kq, H, 512, outliers=0), rows(g, len(lens), kq, H, 64, outliers=0)
    want, fl = D.run(cache, bt, lens, qc, qr)
    assert not any(fl)
    out, fl = decode(0, cache, bt, lens, qc, qr)
    assert fl == [B.PFKV_FLAG_DEVICE_TIMEOUT if n else 0 for n in lens]
    assert not out.any()
    out, fl = decode(NEVER, cache, bt, lens, qc, qr)
    assert not any(fl) and torch.equal(out, want)
    out, fl = D.run(cache, bt, lens, qc, qr)
    assert not any(fl) and torch.equal(out, want)
