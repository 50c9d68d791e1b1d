"""pfkv_prefix_decode_attn and pfkv_kv_evict as programs call them: captured and replayed, on two
streams at once, with inputs and results in host memory, between guards, in batches that need
several launches, over pools past 32 bits, one after the other; and with waits that run out."""
import math

import pytest
import torch

from paged_fp8_kv_decode_gb300 import rope as R
from prefix_cases import (B, E, P, PAGE, Pool, attend, call, close, evict_call, gen, i32, kept_ids, no_prefixes, pages_of,
                          per_head, rows)
from test_gpu_canary import Guarded
from test_gpu_evict import check as check_evict
from test_gpu_evict import totals
from test_gpu_prefix import check

pytestmark = pytest.mark.gpu


def workspace(pool, own, pre, batch, hq, kq, n, p, mass=False):
    return torch.empty(P.pfkv_prefix_decode_workspace_size(pool.cache, own, pre, batch, hq, kq, n, p, mass=mass),
                       dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("fp8", [False, True])
def test_replayed_with_other_inputs(fp8):
    """Two captured graphs, whose inputs change between replays, give what calls give."""
    pool = Pool(300, 2, 128, fp8, seed=21)
    pre, own = pool.tables([500, 130, 0]), pool.tables([20, 30, 400, 7])
    of, q = i32([0, 1, -1, 0]), rows(pool.g, 4, 1, 8, 128, outliers=0)
    mass = torch.zeros(4, 2, 400, device="cuda")
    outs, graphs, flags, keep = [], [], [], []  # what a graph uses lives as long as it
    for k in range(2):
        ws = workspace(pool, own, pre, 4, 8, 1, 400, 500, mass=k == 0)
        out, fl = torch.empty_like(q), torch.zeros(4, dtype=torch.uint8, device="cuda")
        args = pool.cache, own, pre, of, q, 0.1, 400, 500, ws, out
        P.pfkv_prefix_decode_attn(*args, attn_mass=mass if k == 0 else None, flags=fl)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            P.pfkv_prefix_decode_attn(*args, attn_mass=mass if k == 0 else None, flags=fl)
        outs.append(out), graphs.append(g), flags.append(fl), keep.append(args)
    mass.zero_()
    total = torch.zeros_like(mass, dtype=torch.float64)
    for step, (new_of, lens, plens) in enumerate(([[0, 1, -1, 0], [20, 30, 400, 7], [500, 130, 0]], [[1, 1, 2, -1], [1, 0, 399, 6], [1, 129, 0]],
                                                  [[2, 0, 0, 0], [20, 16, 17, 0], [257, 3, 0]])):
        of.copy_(i32(new_of))
        own.seq_lens.copy_(i32(lens)[:, None])
        pre.seq_lens.copy_(i32(plens)[:, None])
        own.lens, pre.lens = per_head(lens, 2), per_head(plens, 2)
        q.copy_(rows(pool.g, 4, 1, 8, 128, outliers=0))
        want, tol, m, m_tol = attend(pool, own, pre, new_of, q, 0.1, torch.zeros_like(mass))
        before = mass.double().clone()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert not flags[0].any() and not flags[1].any()
        for out in outs:
            close(out, want, tol, f"out of replay {step}")
        close(mass.double() - before, m, m_tol + mass.double() * 2.0 ** -23, f"mass of replay {step}")


@pytest.mark.parametrize("fp8", [False, True])
def test_two_streams_at_once(fp8):
    pool = Pool(2000, 2, 128, fp8, seed=22)
    pre, own, of = pool.tables([9000, 77]), pool.tables([300, 3, 90]), i32([0, 1, 0])
    q = [rows(pool.g, 3, 1, 16, 128, outliers=0) for _ in range(2)]
    want = [call(pool, own, pre, of, x, 0.1)[0] for x in q]
    src, mass = pool.tables([5000, 200]), totals(pool, 2, 5000, "plain")
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [workspace(pool, own, pre, 3, 16, 1, 300, 9000) for _ in range(2)]
    outs = [torch.empty_like(q[0]) for _ in range(2)]
    dst = [pool.tables([700, 50], fill=False) for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for s, x, w, o, d in zip(streams, q, ws, outs, dst):
            P.pfkv_prefix_decode_attn(pool.cache, own, pre, of, x, 0.1, 300, 9000, w, o, stream=s)
            with torch.cuda.stream(s):
                got.append(evict_call(pool, src, d, i32([[700], [50]]), mass, 4, 8, stream=s))
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
    for lens, new_mass, ids, flags in got:
        assert not flags[:2].any() and lens.tolist() == [[700], [50]]
        assert torch.equal(ids, got[0][2]) and torch.equal(new_mass, got[0][1])


@pytest.mark.parametrize("fp8", [False, True])
def test_host_memory(fp8):
    """Queries, tables, lengths, numbers of kept tokens, results and flags in pinned host memory."""
    pool = Pool(400, 2, 64, fp8, tags=True, seed=23)
    pre, own = pool.tables([300, 20], heads_apart=True), pool.tables([50, 1, 130], heads_apart=True)
    q = rows(pool.g, 3, 2, 4, 64, outliers=0)
    want, _ = call(pool, own, pre, [0, -1, 1], q, 0.1)
    pin = lambda t: t.cpu().pin_memory()  # noqa: E731

    def host(p):
        h = B.Pages(p.batch, p.max_pages, pin(p.block_tables), p.bt_stride_b, p.bt_stride_h, pin(p.seq_lens), p.len_stride_b,
                    p.len_stride_h, pin(p.expected_tags))
        h.lens = p.lens
        return h
    out, flags = pin(torch.zeros_like(q)), pin(torch.full((4,), 0xAA, dtype=torch.uint8))
    call(pool, host(own), host(pre), pin(i32([0, -1, 1])), pin(q), 0.1, out=out, flags=flags)
    torch.cuda.synchronize()
    assert torch.equal(out, want.cpu()) and not flags[:3].any()
    dst, other = (pool.tables([[20, 9], [1, 0], [64, 65]], heads_apart=True, fill=False) for _ in range(2))
    keep, mass = i32([[20, 9], [1, 0], [64, 65]]), totals(pool, 3, 130, "plain")
    own = B.Pages(3, own.max_pages, own.block_tables, own.bt_stride_b, own.bt_stride_h, i32([[50, 50], [1, 1], [130, 130]]), 2, 1,
                  own.expected_tags)
    own.lens = [[50, 50], [1, 1], [130, 130]]
    a = evict_call(pool, own, dst, keep, mass, 2, 3)
    b = evict_call(pool, host(own), host(other), pin(keep), mass, 2, 3, max_keep=65, new_lens=pin(torch.zeros(3, 2, dtype=torch.int32)))
    torch.cuda.synchronize()
    assert all(torch.equal(x.cpu(), y.cpu()) for x, y in zip(a[:3], b[:3])) and not b[3][:3].any()
    for i, r in enumerate([[20, 9], [1, 0], [64, 65]]):
        for h, n in enumerate(r):
            for which in "kv":
                assert torch.equal(pool.values(dst, i, h, n, which), pool.values(other, i, h, n, which))


@pytest.mark.parametrize("kq", [1, 3])
@pytest.mark.parametrize("fp8", [False, True])
def test_guards(fp8, kq):
    """Nothing outside the buffers of a call is written."""
    pool = Pool(500, 3, 128, fp8, seed=24)
    pre, own, of = pool.tables([700, 129, 5]), pool.tables([20, 0, 333, 16, 1]), [0, 1, -1, 0, 2]
    q = rows(pool.g, 5, kq, 12, 128, outliers=0)
    mass = torch.zeros(5, 3, 333, device="cuda") if kq == 1 else None
    want, _ = call(pool, own, pre, of, q, 0.1, mass=None if mass is None else mass.clone())
    ws = workspace(pool, own, pre, 5, 12, kq, 333, 700, mass=kq == 1)
    g = {"out": Guarded(torch.zeros_like(q), 1), "flags": Guarded(torch.zeros(8, dtype=torch.uint8, device="cuda"), 2), "ws": Guarded(ws, 3)}
    if mass is not None:
        g["mass"] = Guarded(mass, 4)
    P.pfkv_prefix_decode_attn(pool.cache, own, pre, i32(of), q, 0.1, 333, 700, g["ws"].t, g["out"].t,
                              attn_mass=g["mass"].t if mass is not None else None, flags=g["flags"].t)
    torch.cuda.synchronize()
    assert all(x.intact() for x in g.values()) and torch.equal(g["out"].t, want)


@pytest.mark.parametrize("fp8", [False, True])
def test_guards_of_eviction(fp8):
    pool = Pool(300, 3, 128, fp8, seed=25)
    lens, keep = [[200, 16, 0], [1, 77, 500]], [[60, 16, 5], [1, 20, 111]]
    src = pool.tables(lens, heads_apart=True)
    dst = pool.tables([[min(a, b) for a, b in zip(x, y)] for x, y in zip(lens, keep)], heads_apart=True, fill=False)
    mass = totals(pool, 2, 500, "plain")
    c = pool.cache
    guarded = [None if t is None else Guarded(t, 10 + i) for i, t in enumerate((c.k_pages, c.v_pages, c.k_scale, c.v_scale))]
    pool.cache = B.Cache(*[None if x is None else x.t for x in guarded])
    n = E.pfkv_kv_evict_workspace_size(pool.cache, src, 500, 111)
    more = [Guarded(t, 20 + i) for i, t in enumerate((torch.zeros(n, dtype=torch.uint8, device="cuda"), torch.zeros(2, 3, dtype=torch.int32, device="cuda"),
                                                      torch.zeros(2, 3, 120, device="cuda"), torch.zeros(2, 3, 111, dtype=torch.int32, device="cuda"),
                                                      torch.zeros(4, dtype=torch.uint8, device="cuda")))]
    E.pfkv_kv_evict(pool.cache, src, dst, i32(keep), mass, 500, 111, more[0].t, more[1].t, new_mass=more[2].t, kept=more[3].t, keep_first=1,
                    keep_last=1, flags=more[4].t)
    torch.cuda.synchronize()
    assert all(x.intact() for x in guarded + more if x is not None) and not more[4].t.any()
    for b in range(2):
        for h in range(3):
            ids = kept_ids(mass[b, h, :lens[b][h]], lens[b][h], keep[b][h], 1, 1)
            assert more[3].t[b, h, :len(ids)].tolist() == ids


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B_,H,D,NP", [(1100, 4, 64, 3), (2500, 1, 128, 700)])
def test_large_batches(B_, H, D, NP, fp8):
    """More segments than a launch of the split kernel holds; more prefixes and requests than the plan keeps at hand."""
    g = gen(26)
    of = torch.randint(-1, NP, (B_,), generator=g, device="cuda").tolist()
    lens = torch.randint(0, 20, (B_,), generator=g, device="cuda").tolist()
    plens = torch.randint(0, 40, (NP,), generator=g, device="cuda").tolist()
    pool = Pool(sum(map(pages_of, lens + plens)) + 8, H, D, fp8, seed=26)
    pre, own = pool.tables(plens), pool.tables(lens)
    check(pool, own, pre, of, rows(pool.g, B_, 1, 2 * H, D, outliers=0), D ** -0.5)


def test_pools_past_32_bits():
    """Pages, rows of totals and lists whose offsets pass 32 bits."""
    num = (1 << 32) // (PAGE * 128 * 2) + 300  # bytes of a bf16 pool of one head
    pool = Pool(400, 1, 128, False, seed=27)
    k, v = (torch.zeros(num, 1, PAGE, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pool.cache, pool.free = B.Cache(k, v), [num - 1 - i for i in range(250)] + [(1 << 20) - 5 + i for i in range(10)]
    pre, own = pool.tables([700]), pool.tables([40, 300])
    check(pool, own, pre, [0, 0], rows(pool.g, 2, 1, 4, 128, outliers=0), 0.1)
    dst = pool.tables([30, 100], fill=False)
    far = torch.zeros((1 << 31) + 5000, device="cuda")  # the second request's totals lie past 2^31 elements
    mass = torch.as_strided(far, (2, 1, 300), ((1 << 31) + 100, 300, 1))
    mass.copy_(totals(pool, 2, 300, "plain"))
    want = [kept_ids(mass[b, 0, :n], n, m, 2, 5) for b, (n, m) in enumerate(((40, 30), (300, 100)))]
    x = [pool.values(own, b, 0, n, "v")[w] for b, (n, w) in enumerate(zip((40, 300), want))]
    lens, _, ids, flags = evict_call(pool, own, dst, i32([[30], [100]]), mass, 2, 5)
    assert not flags[:2].any() and lens.tolist() == [[30], [100]]
    for b, w in enumerate(want):
        assert ids[b, 0, :len(w)].tolist() == w and torch.equal(pool.values(dst, b, 0, len(w), "v"), x[b])


@pytest.mark.parametrize("n,k", [(70000, 300), (300001, 33333), (820000, 100)])
def test_long_contexts(n, k):
    """Slices of many CTAs, and totals that do not fit in shared memory."""
    pool = Pool(pages_of(n) + pages_of(k) + 4, 1, 64, True, seed=28)
    src, dst = pool.tables([n]), pool.tables([k], fill=False)
    mass = totals(pool, 1, n, "plain")
    mass[0, 0, ::7] = 0.25  # many equal ones, among which the border falls
    lens, new_mass, ids, flags = evict_call(pool, src, dst, i32([[k]]), mass, 16, 64)
    middle = mass[0, 0, 16:n - 64]
    order = torch.sort(middle, descending=True, stable=True)[1][:k - 80] + 16
    want = torch.cat((torch.arange(16, device="cuda"), order.sort()[0], torch.arange(n - 64, n, device="cuda")))
    assert not flags[:1].any() and torch.equal(ids[0, 0].long(), want) and torch.equal(new_mass[0, 0, :k], mass[0, 0][want])


def test_waits_that_run_out():
    """Every request with a prefix is flagged and zero, the others are as they were, and the next call is sound."""
    for fp8 in (False, True):
        pool = Pool(400, 2, 128, fp8, seed=29)
        pre, own, of = pool.tables([3000, 200]), pool.tables([30, 40, 50]), [0, -1, 1]
        q = rows(pool.g, 3, 1, 8, 128, outliers=0)
        want = check(pool, own, pre, of, q, 0.1)
        out, flags = torch.full_like(q, math.nan), torch.zeros(4, dtype=torch.uint8, device="cuda")
        ws = workspace(pool, own, pre, 3, 8, 1, 50, 3000)
        P.pfkv_selftest_prefix_decode(0, pool.cache, own, pre, i32(of), q, 0.1, 50, 3000, ws, out, flags=flags)
        torch.cuda.synchronize()
        assert flags[:3].tolist() == [8, 0, 8]
        assert not out[0].any() and not out[2].any() and torch.equal(out[1], want[1])
        again, flags = call(pool, own, pre, of, q, 0.1)
        assert torch.equal(again, want) and not flags[:3].any()


@pytest.mark.parametrize("fp8", [False, True])
def test_not_finite(fp8):
    """What a row sees reaches it; what it does not see does not."""
    pool = Pool(200, 2, 128, fp8, seed=30)
    pre, own, of = pool.tables([300, 40]), pool.tables([20, 30, 4]), [0, 1, 0]
    q = rows(pool.g, 3, 1, 8, 128, outliers=0)
    want = check(pool, own, pre, of, q, 0.1)
    page = pool.row(pre, 0, 0)[5]
    pool.cache.k_pages[page, 1, 3, 7] = 0x7F if fp8 else math.nan
    out, flags = call(pool, own, pre, of, q, 0.1)
    assert out[0, 0, 4:].isnan().all() and out[2, 0, 4:].isnan().all() and not flags[:3].any()
    assert torch.equal(out[:, :, :4], want[:, :, :4]) and torch.equal(out[1], want[1])


def test_scales_of_any_sign():
    """K and V scales of zero and below zero."""
    pool = Pool(200, 2, 64, True, seed=31)
    pre, own, of = pool.tables([500, 40]), pool.tables([20, 30, 4]), [0, 1, 0]
    ids = pool.row(pre, 0, 0)
    pool.cache.k_scale[ids[3], 0] *= -1
    pool.cache.k_scale[ids[4], 1] = 0
    pool.cache.v_scale[ids[5], 0] *= -3
    pool.cache.v_scale[ids[6], 1] = 0
    pool.cache.k_scale[ids[31], :] = 0   # the last page, which is not full
    check(pool, own, pre, of, rows(pool.g, 3, 1, 8, 64, outliers=0), 0.125)


@pytest.mark.parametrize("fp8", [False, True])
def test_one_after_the_other(fp8):
    """Append (turned), attend over prefix and own tokens with their weights, evict by those, append and attend again."""
    H, Hq, D, n = 2, 8, 128, [70, 33]
    pool = Pool(200, H, D, fp8, tags=True, seed=32)
    pre, of = pool.tables([300]), [0, 0]
    own = pool.tables(n, heads_apart=True, wide=1, lens_apart=True)
    freq = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().cuda()
    rope = R.Rope(freq)
    mass = torch.zeros(2, H, 80, device="cuda")
    position = [300 + x for x in n]

    def step(own, mass):
        """One decode step at the sequences' own positions; returns its output."""
        at = own.seq_lens.clone()
        k, v, q = (rows(pool.g, 2, 1, h, D, outliers=0) for h in (H, H, Hq))
        flags = torch.zeros(4, dtype=torch.uint8, device="cuda")
        R.pfkv_rope_append(pool.cache, own, rope, at, k, v, q, q, rope_positions=i32(position), flags=flags)
        own.seq_lens += 1
        own.lens = own.seq_lens.tolist()
        check(pool, own, pre, of, q, D ** -0.5, mass=mass, max_len=80)
        assert not flags.any()
        for b in range(2):
            position[b] += 1

    # heads whose tables have room for the new token
    for b in range(2):
        for h in range(H):
            own.block_tables[b, h, pages_of(n[b])] = pool.free.pop()
    own.expected_tags.copy_(pool.cache.page_tags[own.block_tables.long().clamp(min=0), torch.arange(H, device="cuda")[None, :, None]])
    for _ in range(3):
        step(own, mass)
    keep = i32([[20, 36], [9, 36]])
    dst = pool.tables([[20, 36], [9, 36]], heads_apart=True, fill=False, wide=1, lens_apart=True)
    for b, r in enumerate([[20, 36], [9, 36]]):
        for h, m in enumerate(r):
            dst.block_tables[b, h, pages_of(m)] = pool.free.pop()
    dst.expected_tags.copy_(pool.cache.page_tags[dst.block_tables.long().clamp(min=0), torch.arange(H, device="cuda")[None, :, None]])
    lens, new_mass, ids, flags = evict_call(pool, own, dst, keep, mass, 2, 4, room=90)
    assert not flags[:2].any() and lens.tolist() == keep.tolist()
    for b in range(2):
        for h in range(H):
            want = kept_ids(mass[b, h, :own.lens[b][h]], own.lens[b][h], int(keep[b, h]), 2, 4)
            assert ids[b, h, :len(want)].tolist() == want
    dst.seq_lens.copy_(lens)
    for _ in range(2):
        step(dst, new_mass)
