"""pfkv_prefix_decode_attn against its definition in 64 bits."""
import math

import pytest
import torch

from prefix_cases import Pool, attend, call, close, i32, no_prefixes, rows

pytestmark = pytest.mark.gpu


def check(pool, own, pre, of, q, scale, mass=None, **over):
    want, tol, m_want, m_tol = attend(pool, own, pre, of, q, scale, mass)
    out, flags = call(pool, own, pre, of, q, scale, mass=mass, **over)
    torch.cuda.synchronize()
    assert not flags[:q.shape[0]].any()
    close(out, want, tol, "out")
    if mass is not None:
        close(mass, m_want, m_tol, "mass")
    return out


# kv heads, group, query tokens, prefixes' lengths, each request's prefix, own lengths
CASES = {
    "one": (2, 4, 1, [300], [0, 0, 0], [5, 40, 1]),
    "lone request": (1, 1, 1, [1], [0], [1]),
    "no prefix": (2, 2, 1, [77], [-1, 0, -1], [20, 3, 170]),
    "empty prefix": (2, 8, 1, [0, 33], [0, 1, 0], [16, 17, 0]),
    "tile edges": (1, 4, 1, [127, 128, 129, 256, 255, 16], [0, 1, 2, 3, 4, 5], [15, 16, 17, 0, 1, 2]),
    "many rows": (1, 8, 2, [500, 40], [0] * 9 + [1] * 8 + [0] * 12, [3] * 29),
    "two blocks": (2, 8, 1, [700], [0] * 33, list(range(33))),
    "long": (2, 4, 1, [9001, 20], [0, 1, 0, 0], [0, 300, 1000, 129]),
    "verify": (2, 4, 3, [100, 259], [1, 0, -1, 1, 0], [3, 1, 2, 100, 0]),
    "unused prefixes": (4, 1, 1, [50, 60, 70], [2, 2, -1], [1, 2, 3]),
    "many prefixes": (2, 2, 1, [1 + 13 * i for i in range(40)], [(7 * i) % 41 - 1 for i in range(60)], [(5 * i) % 37 for i in range(60)]),
}


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name", list(CASES))
def test_matches(name, fp8, D):
    H, G, kq, plens, of, lens = CASES[name]
    pool = Pool(sum(map(lambda n: n // 16 + 1, plens + lens)) + 9, H, D, fp8, seed=len(name))
    pre, own = pool.tables(plens), pool.tables(lens, wide=2)
    check(pool, own, pre, of, rows(pool.g, len(of), kq, G * H, D, outliers=0), D ** -0.5)


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kq,G,plens", [(1, 8, [1500, 3]), (7, 1, [64, 448]), (33, 4, [700, 129])])
def test_prefix_alone(kq, G, plens, fp8, D):
    """Attention to the states of an encoder: no own tokens, every query token sees the whole prefix."""
    pool = Pool(400, 2, D, fp8, seed=3)
    pre, of = pool.tables(plens), [0, 1, -1]
    check(pool, None, pre, of, rows(pool.g, 3, kq, 2 * G, D, outliers=0), D ** -0.5)


@pytest.mark.parametrize("fp8", [False, True])
def test_no_prefixes_at_all(fp8):
    pool = Pool(40, 2, 128, fp8, seed=4)
    own = pool.tables([0, 1, 100])
    check(pool, own, no_prefixes(2), [-1, -1, -1], rows(pool.g, 3, 1, 8, 128, outliers=0), 0.1)


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("fp8", [False, True])
def test_tables_and_lengths_a_head(fp8, D):
    pool = Pool(400, 3, D, fp8, tags=True, seed=5)
    pre = pool.tables([[300, 0, 17], [5, 600, 128]], heads_apart=True)
    own = pool.tables([[0, 16, 33], [70, 1, 0], [5, 5, 5], [200, 0, 1]], heads_apart=True)
    check(pool, own, pre, [0, 1, -1, 1], rows(pool.g, 4, 2, 6, D, outliers=0), D ** -0.5)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads_apart", [False, True])
def test_mass(heads_apart, fp8):
    pool = Pool(600, 2, 128, fp8, tags=True, seed=6)
    pre = pool.tables([1000, 35])
    own = pool.tables([[40, 300], [0, 1], [17, 16], [2000, 31]] if heads_apart else [40, 1, 16, 2000], heads_apart=heads_apart)
    mass = torch.rand(4, 2, 2011, generator=pool.g, device="cuda")
    check(pool, own, pre, [0, 1, -1, 0], rows(pool.g, 4, 1, 8, 128, outliers=0), 128 ** -0.5, mass=mass)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_scales_of_scores(scale, fp8):
    """A scale of zero, below zero, and one that leaves a token alone."""
    pool = Pool(200, 2, 128, fp8, seed=7)
    pre, own = pool.tables([500, 130]), pool.tables([20, 30, 400])
    check(pool, own, pre, [0, 1, 0], rows(pool.g, 3, 1, 8, 128, outliers=0), scale)


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("fp8", [False, True])
def test_strides_and_in_place(fp8, D):
    """Queries as a slice of a wider row, results in the other order of axes, and results over the queries."""
    pool = Pool(200, 2, D, fp8, seed=8)
    pre, own, of = pool.tables([500, 130]), pool.tables([20, 30, 400]), [0, 1, 0]
    wide = rows(pool.g, 3, 2, 12, D, outliers=0)
    q = wide[:, :, 2:10]
    want = check(pool, own, pre, of, q.contiguous(), D ** -0.5)
    back = torch.full((8, 2, 3, D + 8), math.nan, dtype=torch.bfloat16, device="cuda")
    out = back[..., :D].permute(2, 1, 0, 3)
    call(pool, own, pre, of, q, D ** -0.5, out=out)
    assert torch.equal(out, want) and back[..., D:].isnan().all()
    call(pool, own, pre, of, q, D ** -0.5, out=q)
    assert torch.equal(q, want)
    assert not torch.equal(wide[:, :, 0], torch.zeros_like(wide[:, :, 0]))


def test_flags():
    """What fails a check flags its request, and every request of a prefix that fails; the others are as they were."""
    for fp8 in (False, True):
        pool = Pool(400, 2, 128, fp8, tags=True, seed=9)
        pre = pool.tables([200, 100, 50, 300, 77], heads_apart=True)
        own = pool.tables([30, 40, 50, 60, 70, 80, 90, 20, 10], heads_apart=True)
        of = [0, 1, 2, 3, 4, -1, 0, 0, 0]
        q = rows(pool.g, 9, 1, 8, 128, outliers=0)
        want = check(pool, own, pre, of, q, 0.1)
        pre.block_tables[1, 1, 3] = pool.cache.k_pages.shape[0]      # BAD_PAGE of request 1
        pre.expected_tags[2, 0, 1] ^= 4                              # TAG_MISMATCH of request 2
        pre.seq_lens[3] = 301                                        # BAD_LENGTH of request 3 (above the bound)
        of[4] = 5                                                    # no such prefix
        own.block_tables[5, 0, 0] = -1
        own.expected_tags[6, 1, 5] ^= 1
        own.seq_lens[7] = -1
        out, flags = call(pool, own, pre, of, q, 0.1, max_len=90, max_pre=300)
        assert flags[:9].tolist() == [0, 2, 1, 4, 2, 2, 1, 4, 0]
        assert torch.equal(out[0], want[0]) and torch.equal(out[8], want[8]) and not out[1:8].any()
        # an entry past the last live one is not looked at, and no mass comes of flagged requests
        mass = torch.zeros(9, 2, 90, device="cuda")
        call(pool, own, pre, of, q, 0.1, max_len=90, max_pre=300, mass=mass)
        assert not mass[1:8].any() and mass[0, :, :30].all() and mass[8, :, :10].all() and not mass[8, :, 10:].any()
