"""Values that are not finite, in tokens that a query must not see: they reach the rows
that see them, as they are, and no other row."""
import pytest
import torch

import test_gpu_latent_decode as D
import test_gpu_latent_prefill as P
from latent_cases import (BF16, PAGE, SCALE, close, gen, latent_pool, rows, score_error, softmax_attend, tables)

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def expect(got, s, v, weight_step, err, what):
    """Rows of softmax(s) v (s is -inf where a row does not see a token) where every seen
    value is finite; elsewhere infinity, if all that are not are infinities of one sign,
    or NaN."""
    seen, odd = ~torch.isinf(s), ~v.isfinite()
    o, tol = softmax_attend(s, torch.where(odd, 0.0, v), weight_step, err)
    up, down, nan = ((seen.double() @ m.double()) > 0 for m in (v == INF, v == -INF, v.isnan()))
    nan = nan | up & down
    special = up | down | nan
    close(torch.where(special, 0.0, got.double()), torch.where(special, 0.0, o), tol, what)
    assert got[nan].isnan().all() and (got[up & ~nan] == INF).all() and (got[down & ~nan] == -INF).all(), what


@pytest.mark.parametrize("nq,nk,odd", [
    (300, 300, {150: NAN}),
    (300, 300, {0: INF, 5: -INF, 127: NAN, 128: INF, 255: -INF, 256: NAN, 299: INF}),
    (300, 300, {299: NAN}),
    (500, 570, {69: INF, 70: NAN, 200: INF, 201: -INF, 333: NAN, 569: INF}),     # steps and tiles out of step
    (64, 1000, {3: NAN, 937: INF, 960: NAN, 999: NAN}),
    (200, 90, {0: NAN, 40: INF, 89: -INF}),                                       # rows that see no key
    (700, 700, {j: (NAN, INF)[j % 2] for j in range(1, 700, 3)}),
    (1, 200, {199: NAN}),
])
def test_prefill(nq, nk, odd):
    g = gen(nq + nk)
    lens_q, lens_k = [40, nq, 33], [40, nk, 50]
    qs, ks = P.starts_of(lens_q), P.starts_of(lens_k)
    x = P.inputs(g, qs[-1], ks[-1], 3)
    for j, bad in odd.items():                       # of the second request's second head
        x["v"][ks[1] + j, 1, (5 * j) % 128] = bad
        x["v"][ks[1] + j, 1, 77] = bad
    out, fl = P.run(x, qs, ks, max(lens_q))
    assert not any(fl)
    for b in range(3):
        for h in range(3):
            if (b, h) != (1, 1):
                P.check(x, (qs[b], qs[b + 1]), (ks[b], ks[b + 1]), out, heads=[h])
    q, k = slice(qs[1], qs[2]), slice(ks[1], ks[2])
    qq = torch.cat((x["qn"][q, 1], x["qr"][q, 1]), 1).double()
    kk = torch.cat((x["kn"][k, 1], x["kr"][k]), 1).double()
    seen = torch.ones(nq, nk, dtype=torch.bool, device="cuda").tril(nk - nq)
    s = torch.where(seen, qq @ kk.T * SCALE, -torch.inf)
    expect(out[q, 1], s, x["v"][k, 1].double(), BF16, score_error(qq, kk, SCALE), (nq, nk))


def test_prefill_without_a_mask():
    """Every query sees every key: one NaN or infinity reaches its column of all rows."""
    g = gen(94)
    x = P.inputs(g, 150, 300, 2)
    x["v"][170, 0, 9], x["v"][299, 0, 100] = NAN, -INF
    out, _ = P.run(x, [0, 150], [0, 300], 150, causal=False)
    assert out[:, 0, 9].isnan().all() and (out[:, 0, 100] == -INF).all()
    assert out[:, 1].isfinite().all() and int(out.isfinite().logical_not().sum()) == 300


def test_prefill_of_many_prompts():
    """Several tiles of queries a multiprocessor, most of them with such a value, the last
    ones among them."""
    g = gen(95)
    H, nq = 64, [300, 130, 257, 70, 600] * 3
    qs = P.starts_of(nq)
    x = P.inputs(g, qs[-1], qs[-1], H)
    for b, n in enumerate(nq):
        for h in range(H):
            if (b + h) % 3:
                x["v"][qs[b] + n - 1 - (7 * h + b) % 60, h, h] = (NAN, INF, -INF)[h % 3]
    clean = dict(x, v=torch.where(x["v"].isfinite(), x["v"], 0.0))
    want, _ = P.run(clean, qs, qs, max(nq))
    out, fl = P.run(x, qs, qs, max(nq))
    assert not any(fl)
    for b, n in enumerate(nq):
        for h in range(H):
            if (b + h) % 3:
                at, bad = n - 1 - (7 * h + b) % 60, (NAN, INF, -INF)[h % 3]
                assert not out[qs[b]:qs[b] + at, h].isnan().any(), (b, h)
                got = out[qs[b] + at:qs[b + 1], h, h]
                assert got.isnan().all() if bad != bad else (got == bad).all(), (b, h)
                want[qs[b] + at:qs[b + 1], h, h] = 0.0
                out[qs[b] + at:qs[b + 1], h, h] = 0.0
    assert torch.equal(out, want)                    # all else has the same bits


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,kq", [(16, 3), (128, 2), (128, 4), (1, 7), (64, 2), (3, 40), (1, 200), (5, 130)])
@pytest.mark.parametrize("back", [0, 1])
def test_decode(H, kq, back, fp8):
    """A latent that is not finite in the last candidate, or the one before it: the rows of
    earlier candidates have the bits that they have without it, later ones are NaN."""
    if back >= kq:
        return
    g = gen(96)
    lens = [128, 129, 130, 200, 256, 16, 3, 2, 1, 700, 0, 384, 145] * 2
    bt, num = tables([(n + PAGE - 1) // PAGE for n in lens], seed=H + kq)
    cache = latent_pool(g, num, fp8)
    qc, qr = rows(g, len(lens), kq, H, 512, outliers=0), rows(g, len(lens), kq, H, 64, outliers=0)
    want, fl = D.run(cache, bt, lens, qc, qr)
    assert not any(fl)
    D.check(cache, bt, lens, qc, qr, want)
    for b, n in enumerate(lens):
        if n - 1 - back >= 0:
            j = n - 1 - back
            page = int(bt[b, j // PAGE])
            bad = (0x7F, 0xFF)[b % 2] if fp8 else (NAN, INF, -NAN)[b % 3]
            cache.c_pages[page, j % PAGE, (37 * b) % 512] = bad
            if not fp8:                              # a score of -inf would hide it: NaN beside it
                cache.c_pages[page, j % PAGE, (37 * b + 1) % 512] = NAN
    out, fl = D.run(cache, bt, lens, qc, qr)
    assert not any(fl)
    for b, n in enumerate(lens):
        for t in range(kq):
            if n - kq + 1 + t > n - 1 - back >= 0:
                assert out[b, t].isnan().all(), (b, t)
            else:
                assert torch.equal(out[b, t], want[b, t]), (b, t, n)
