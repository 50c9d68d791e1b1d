"""Batches whose prefixes make more segments (blocks of query rows a prefix and kv head) than the
plan keeps in shared memory, empty prefixes and unused ones among them."""
import pytest
import torch

from prefix_cases import BF16, F16, P, Pool, call, close, gen, pages_of, rows
from latent_cases import score_error, softmax_attend
from test_gpu_prefix import check

pytestmark = pytest.mark.gpu

KEPT = 1024  # segments that shared memory has room for


def attend_alone(pool, pre, of, q, scale):
    """`prefix_cases.attend` without own tokens, a prefix's requests at once."""
    Bn, kq, Hq, D = q.shape
    G = Hq // pool.H
    out, tol = (torch.zeros(q.shape, dtype=torch.float64, device="cuda") for _ in range(2))
    of = torch.tensor(of, device="cuda")
    for p in of[of >= 0].unique().tolist():
        members = (of == p).nonzero()[:, 0]
        for h in range(pool.H):
            n = pre.lens[p][h]
            if n == 0:
                continue
            k, v = (pool.values(pre, p, h, n, x) for x in "kv")
            heads = slice(h * G, (h + 1) * G)
            qq = q[members][:, :, heads].double().reshape(-1, D)
            err = score_error(qq, k, scale)
            if pool.fp8:  # a query's pair of e4m3 values: 2^-17 of the row's largest
                err = err + 2.0 ** -17 * qq.abs().amax(-1) * k.abs().sum(-1).amax() * abs(scale)
            o, e = softmax_attend(qq @ k.T * scale, v, F16 if pool.fp8 else BF16, err)
            at = torch.arange(Hq, device="cuda")[heads]
            out[members[:, None, None], torch.arange(kq, device="cuda")[:, None], at] = o.view(-1, kq, G, D)
            tol[members[:, None, None], torch.arange(kq, device="cuda")[:, None], at] = \
                (e + n * 2.0 ** -31 * v.abs().amax()).view(-1, kq, G, D)
    return out, tol


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B_,H,D,NP,kq,G,hi", [
    (2500, 4, 64, 700, 1, 2, 40),                   # requests in chunks
    (700, 4, 128, 300, 1, 2, 300),                  # requests at hand; lengths of several tiles
    (1700, 1, 64, P.PFKV_PREFIX_MAX, 1, 2, 20),     # as many prefixes as a call takes, most of them unused
    (600, 2, 64, 3, 130, 8, 200),                   # few prefixes of many blocks
])
def test_many_segments(B_, H, D, NP, kq, G, hi, fp8):
    g = gen(71)
    of = torch.randint(-1, NP, (B_,), generator=g, device="cuda").tolist()
    plens = torch.randint(0, hi, (NP,), generator=g, device="cuda")
    plens[torch.rand(NP, generator=g, device="cuda") < 0.2] = 0
    plens = plens.tolist()
    plens[1], plens[2] = 0, hi
    used = torch.bincount(torch.tensor(of) + 1, minlength=NP + 1)[1:]
    assert H * int(((used * kq * G + 255) // 256).sum()) > KEPT
    pool = Pool(sum(map(pages_of, plens)) + 8, H, D, fp8, seed=71)
    pre = pool.tables(plens)
    q = rows(pool.g, B_, kq, G * H, D, outliers=0)
    want, tol = attend_alone(pool, pre, of, q, D ** -0.5)
    out, flags = call(pool, None, pre, of, q, D ** -0.5)
    torch.cuda.synchronize()
    assert not flags[:B_].any()
    close(out, want, tol, "out")


@pytest.mark.parametrize("fp8", [False, True])
def test_with_own_tokens(fp8):
    g = gen(72)
    of = torch.randint(-1, 600, (900,), generator=g, device="cuda").tolist()
    plens, lens = (torch.randint(0, hi, (n,), generator=g, device="cuda").tolist() for hi, n in ((50, 600), (20, 900)))
    assert 4 * len(set(of) - {-1}) > KEPT
    pool = Pool(sum(map(pages_of, plens + lens)) + 8, 4, 64, fp8, seed=72)
    pre, own = pool.tables(plens), pool.tables(lens)
    check(pool, own, pre, of, rows(pool.g, 900, 1, 8, 64, outliers=0), 0.125)
