"""pfkv_kv_evict against its definition: the kept tokens exactly, the bytes and scales of the
new pages exactly too (fp32 products, divisions and encodings)."""
import math

import pytest
import torch

from prefix_cases import PAGE, Pool, evict_call, gen, i32, kept_ids, pages_of, per_head

pytestmark = pytest.mark.gpu


def totals(pool, B, n, kind):
    x = torch.exp(torch.randn(B, pool.H, n, generator=pool.g, device="cuda") * 2 - 6)
    if kind == "equal":
        x = torch.full_like(x, 0.25)
    elif kind == "few":          # many equal ones
        x = torch.randint(0, 3, x.shape, generator=pool.g, device="cuda").float() / 7
    elif kind == "strange":
        u = torch.rand(x.shape, generator=pool.g, device="cuda")
        for at, y in ((0.1, math.nan), (0.2, math.inf), (0.3, -math.inf), (0.4, -0.0), (0.5, 0.0), (0.6, -1.0), (0.7, 1e-42)):
            x = torch.where((u < at) & (u >= at - 0.1), torch.full_like(x, y), x)
        x = torch.where(u > 0.95, -torch.full_like(x, math.nan), x)
    elif kind == "close":        # all bits but the lowest eleven alike
        x = (torch.randint(0, 2048, x.shape, generator=pool.g, device="cuda", dtype=torch.int32) + 0x3F123000).view(torch.float32)
    return x


def expect(pool, src, dst, keep, mass, first, last):
    """The pool, lengths, totals and indices that the call has to give."""
    c = pool.cache
    k_pages, v_pages = c.k_pages.clone(), c.v_pages.clone()
    scales = [None if s is None else s.clone() for s in (c.k_scale, c.v_scale)]
    B, H = src.batch, pool.H
    kept = {}
    for b in range(B):
        for h in range(H):
            n = src.lens[b][h]
            ids = kept_ids(mass[b, h, :n], n, int(keep[b, h if keep.shape[1] > 1 else 0]), first, last)
            kept[b, h] = ids
            fr, to = pool.row(src, b, h), pool.row(dst, b, h)
            for p in range(pages_of(len(ids))):
                part = torch.tensor(ids[p * PAGE:(p + 1) * PAGE], device="cuda")
                at, slot, new = fr[part // PAGE], part % PAGE, to[p]
                for old, pool_, i in ((c.k_pages, k_pages, 0), (c.v_pages, v_pages, 1)):
                    x = old[at, h, slot]
                    if pool.fp8:
                        s = (c.k_scale, c.v_scale)[i][at, h]
                        if len(set(at.tolist())) == 1:
                            scales[i][new, h] = s[0]
                        else:
                            y = x.view(torch.float8_e4m3fn).float() * s[:, None]
                            top = y.abs().amax()
                            # by a tensor: a number's reciprocal would be multiplied by
                            z = torch.where(top == 0, torch.ones_like(top), top / torch.full_like(top, 448.0))
                            scales[i][new, h] = z
                            x = (y / z).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                    pool_[new, h, :len(part)] = x
    return k_pages, v_pages, scales, kept


def check(pool, src, dst, keep, mass, first, last, **over):
    k, v, (ks, vs), kept = expect(pool, src, dst, keep, mass, first, last)
    lens, new_mass, ids, flags = evict_call(pool, src, dst, keep, mass, first, last, **over)
    torch.cuda.synchronize()
    assert not flags[:src.batch].any()
    c = pool.cache
    for got, want, what in ((c.k_pages, k, "k"), (c.v_pages, v, "v")):
        assert torch.equal(got.view(torch.uint8), want.view(torch.uint8)), what
    if pool.fp8:
        assert torch.equal(c.k_scale.view(torch.int32), ks.view(torch.int32))
        assert torch.equal(c.v_scale.view(torch.int32), vs.view(torch.int32))
    for (b, h), want in kept.items():
        m = len(want)
        assert int(lens.reshape(src.batch, -1)[b, h if lens.shape[1] > 1 else 0]) == m
        if ids is not None:
            assert ids[b, h, :m].tolist() == want and (ids[b, h, m:] == -3).all()
        w = torch.tensor(want, dtype=torch.long, device="cuda")
        assert torch.equal(new_mass[b, h, :m].view(torch.int32), mass[b, h][w].view(torch.int32))
        assert (new_mass[b, h, m:] == 0).all()


# own lengths (a number, or one a head), what is kept, first, last
CASES = {
    "plain": ([100, 37, 260], [40, 20, 100], 4, 8),
    "one token": ([1, 1, 2], [1, 0, 1], 0, 0),
    "nothing": ([0, 40, 16], [5, 0, 0], 3, 3),
    "everything": ([33, 16, 64], [33, 100, 64], 2, 2),
    "ends alone": ([90, 50, 31], [12, 9, 5], 8, 100),
    "few kept": ([1000, 999], [2, 1], 0, 0),
    "unaligned": ([515, 1030], [129, 257], 1, 3),
    "long": ([20011, 3], [5000, 2], 16, 64),
    "last page": ([48, 47], [17, 16], 0, 1),
}


@pytest.mark.parametrize("D,H", [(128, 2), (64, 3)])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name", list(CASES))
def test_matches(name, fp8, D, H):
    lens, keep, first, last = CASES[name]
    pool = Pool(2 * sum(map(pages_of, lens)) + 12, H, D, fp8, seed=len(name))
    src = pool.tables(lens)
    dst = pool.tables([min(a, b) for a, b in zip(lens, keep)], fill=False)
    mass = totals(pool, len(lens), max(lens), "plain")
    check(pool, src, dst, i32(keep)[:, None], mass, first, last)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kind", ["equal", "few", "strange", "close"])
def test_totals(kind, fp8):
    pool = Pool(900, 2, 128, fp8, seed=12)
    lens, keep = [700, 5000], [111, 1999]
    src, dst = pool.tables(lens), pool.tables(keep, fill=False)
    check(pool, src, dst, i32(keep)[:, None], totals(pool, 2, 5000, kind), 3, 5)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [128, 64])
def test_heads_apart(D, fp8):
    """Tables, lengths and numbers of kept tokens a head; tags on both sides; totals with strides; no list of what is kept."""
    pool = Pool(900, 3, D, fp8, tags=True, seed=13)
    lens, keep = [[100, 0, 37], [500, 16, 1], [33, 2000, 64]], [[50, 4, 37], [16, 16, 0], [1, 700, 63]]
    src = pool.tables(lens, heads_apart=True)
    dst = pool.tables([[min(a, b) for a, b in zip(x, y)] for x, y in zip(lens, keep)], heads_apart=True, fill=False)
    mass = totals(pool, 3, 2005, "plain").transpose(0, 1).contiguous().transpose(0, 1)
    check(pool, src, dst, i32(keep), mass, 2, 6, kept=False, room=1234)


def test_new_lengths_over_old_ones():
    pool = Pool(100, 2, 128, True, seed=14)
    src, dst = pool.tables([100, 37]), pool.tables([40, 20], fill=False)
    check(pool, src, dst, i32([[40], [20]]), totals(pool, 2, 100, "plain"), 4, 4, new_lens=src.seq_lens)
    assert src.seq_lens.tolist() == [[40], [20]]


def test_shared_pages_stay():
    """Two requests that name the same pages keep tokens of their own, and the pages stay as they were."""
    pool = Pool(100, 2, 128, True, seed=15)
    src = pool.tables([160, 160])
    src.block_tables[1] = src.block_tables[0]
    dst = pool.tables([50, 70], fill=False)
    check(pool, src, dst, i32([[50], [70]]), totals(pool, 2, 160, "plain"), 0, 0)


@pytest.mark.parametrize("fp8", [False, True])
def test_flags(fp8):
    pool = Pool(300, 2, 64, fp8, tags=True, seed=16)
    lens, keep = [60] * 9, [30] * 9
    src, dst = pool.tables(lens, heads_apart=True, lens_apart=True), pool.tables(keep, heads_apart=True, fill=False)
    k = i32(per_head(keep, 2))
    src.block_tables[1, 1, 3] = -1
    src.expected_tags[2, 0, 3] ^= 1
    dst.block_tables[3, 0, 1] = pool.cache.k_pages.shape[0]
    dst.expected_tags[4, 1, 0] ^= 1
    src.seq_lens[5, 1] = 61
    k[6, 0] = -1
    src.seq_lens[7, 0] = -1
    before = [t.clone() for t in (pool.cache.k_pages.view(torch.uint8), pool.cache.v_pages.view(torch.uint8))]
    mass = totals(pool, 9, 60, "plain")
    lens_out, new_mass, ids, flags = evict_call(pool, src, dst, k, mass, 1, 1, max_len=60, max_keep=30)
    assert flags[:9].tolist() == [0, 2, 1, 2, 1, 4, 4, 4, 0]
    assert lens_out.tolist() == [[30, 30]] + [[0, 0]] * 7 + [[30, 30]]
    touched = torch.zeros(pool.cache.k_pages.shape[0], dtype=torch.bool, device="cuda")
    for b in (0, 8):
        touched[dst.block_tables[b, :, :2].long().flatten()] = True
    for old, now in zip(before, (pool.cache.k_pages, pool.cache.v_pages)):
        assert torch.equal(old[~touched], now.view(torch.uint8)[~touched])
    assert new_mass[1:8].isnan().all() and (new_mass[0, :, :30] > 0).all()
    # bounds: k above the caller's bound
    _, _, _, flags = evict_call(pool, src, dst, k, mass, 1, 1, max_len=60, max_keep=29)
    assert flags[0] == 4 and flags[8] == 4


@pytest.mark.parametrize("fp8", [False, True])
def test_nothing_of_a_flagged_request(fp8):
    """A request of which one head fails a check: no head's indices, totals or pages are written."""
    pool = Pool(300, 2, 64, fp8, seed=17)
    src, dst = pool.tables([60, 90], heads_apart=True), pool.tables([30, 40], heads_apart=True, fill=False)
    src.block_tables[0, 1, 2] = -1
    before = [t.clone() for t in (pool.cache.k_pages.view(torch.uint8), pool.cache.v_pages.view(torch.uint8))]
    lens, new_mass, ids, flags = evict_call(pool, src, dst, i32([[30], [40]]), totals(pool, 2, 90, "plain"), 2, 3)
    assert flags[:2].tolist() == [2, 0] and lens.tolist() == [[0], [40]]
    assert (ids[0] == -3).all() and (ids[1] >= 0).all() and new_mass[0].isnan().all()
    hers = dst.block_tables[0, :, :2].long().flatten()
    for old, now in zip(before, (pool.cache.k_pages, pool.cache.v_pages)):
        assert torch.equal(old[hers], now.view(torch.uint8)[hers])
