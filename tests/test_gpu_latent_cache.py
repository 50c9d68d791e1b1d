"""pfkv_latent_append and pfkv_latent_gather against the rotation and the
quantisation in 64 bits: padded and packed rows, both pool types, pages opened
and continued, tags and bad pages, rows that must stay as they were."""
import pytest
import torch

from latent_cases import (BF16, E4M3, PAGE, TURN, close, flags_for, gen, i32, latent_pool, latent_values, pages, rows,
                          tables, turned)
from paged_fp8_kv_decode_gb300 import binding as B
from paged_fp8_kv_decode_gb300 import latent as L
from paged_fp8_kv_decode_gb300 import rope as R

pytestmark = pytest.mark.gpu


def inv_freq(rot=64):
    return (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()


def clone(c):
    return L.LatentCache(*[None if t is None else t.clone() for t in (c.c_pages, c.r_pages, c.c_scale, c.page_tags)])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B_,T,H,rot,inter,ctx,packed", [
    (3, 1, 128, 64, True, [0, 15, 4000], False),
    (2, 6, 5, 32, False, [12, 0], False),
    (4, 100, 16, 64, True, [0, 3, 16, 700000], True),
    (1, 257, 1, 64, False, [31], True),
])
def test_append(B_, T, H, rot, inter, ctx, packed, fp8):
    g = gen(21 + T)
    n = [T] * B_ if not packed else [max(1, T * (b + 1) // B_) for b in range(B_)]
    if packed and B_ > 2:
        n[2] = 0
    bt, num = tables([(c + max(k, 1) - 1) // PAGE + 1 for c, k in zip(ctx, n)], seed=T, first=[c // PAGE for c in ctx])
    cache = latent_pool(g, num, fp8)
    before = clone(cache)
    starts = [0]
    for x in n:
        starts.append(starts[-1] + x)
    lead = (starts[-1] + 2,) if packed else (B_, T)
    c, r, q = rows(g, *lead, 512), rows(g, *lead, 64), rows(g, *lead, H, 64)
    q_out, fl, f = torch.zeros_like(q), flags_for(B_), inv_freq(rot)
    L.pfkv_latent_append(cache, pages(bt, i32(ctx)), R.Rope(f, inter), i32(ctx), c, r, q, q_out,
                         row_starts=i32(starts) if packed else None, max_new_tokens=T, flags=fl)
    torch.cuda.synchronize()
    assert not fl.any()
    touched = torch.zeros(num, PAGE, dtype=torch.bool)
    for b in range(B_):
        rw = (slice(starts[b], starts[b + 1]),) if packed else (b,)
        pos = ctx[b] + torch.arange(n[b], device="cuda")
        want, size = turned(q[rw], pos, f, inter)
        close(q_out[rw], want, BF16 * want.abs() + TURN * size, "queries")
        key, size = turned(r[rw][:, None], pos, f, inter)
        for at in range(-(ctx[b] % PAGE), n[b], PAGE):
            t0, t1 = max(0, at), min(n[b], at + PAGE)
            slot, pg = (ctx[b] + t0) % PAGE, int(bt[b, (ctx[b] + t0) // PAGE])
            touched[pg, slot:slot + t1 - t0] = True
            sl = slice(slot, slot + t1 - t0)
            close(cache.r_pages[pg, sl], key[t0:t1, 0], BF16 * key[t0:t1, 0].abs() + TURN * size[t0:t1, 0], "keys")
            x = c[rw][t0:t1]
            if not fp8:
                assert torch.equal(cache.c_pages[pg, sl], x)
                continue
            if slot == 0:
                z = x.float().abs().max() / torch.tensor(448.0, device="cuda")  # by a tensor: IEEE division
                z = torch.ones_like(z) if float(z) == 0 else z
                assert torch.equal(cache.c_scale[pg], z)
            else:
                assert torch.equal(cache.c_scale[pg], before.c_scale[pg])
            y = (x.float() / cache.c_scale[pg]).clamp(-448, 448)
            assert torch.equal(cache.c_pages[pg, sl], y.to(torch.float8_e4m3fn).view(torch.uint8))
    rest = ~touched.cuda()
    assert torch.equal(cache.c_pages[rest], before.c_pages[rest])
    assert torch.equal(cache.r_pages[rest], before.r_pages[rest])
    if packed:
        assert not q_out[starts[-1]:].any()


@pytest.mark.parametrize("fp8", [False, True])
def test_append_without_queries_strided_and_flagged(fp8):
    g = gen(30)
    ctx = [0, 20, 63, -5]
    bt, num = tables([4] * 4, seed=2)
    cache = latent_pool(g, num, fp8, tags=True)
    expected = cache.page_tags[bt.long()].contiguous()
    expected[1, 1] ^= 4
    before = clone(cache)
    both = rows(g, 4, 3, 576)                        # latent and key side by side, as one projection gives them
    fl = flags_for(4)
    L.pfkv_latent_append(cache, pages(bt, i32(ctx), expected=expected), R.Rope(inv_freq()), i32(ctx), both[..., :512],
                         both[..., 512:], flags=fl)
    torch.cuda.synchronize()
    assert fl[:4].tolist() == [0, 1, 4, 4]           # request 2 runs off its table at its second token
    changed = (cache.r_pages != before.r_pages).flatten(1).any(1).nonzero().flatten().tolist()
    assert set(changed) == {int(bt[0, 0]), int(bt[2, 3])}
    key, size = turned(both[0, :, None, 512:], torch.arange(3, device="cuda"), inv_freq(), False)
    close(cache.r_pages[int(bt[0, 0]), :3], key[:, 0], BF16 * key[:, 0].abs() + TURN * size[:, 0], "keys")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens", [[1], [16, 0, 33], [15, 17, 1, 500, 64]])
def test_gather(lens, fp8):
    g = gen(31)
    bt, num = tables([(n + PAGE - 1) // PAGE for n in lens], seed=9)
    cache = latent_pool(g, num, fp8)
    starts, gap = [2], 3                             # rows before, between and behind the requests
    for n in lens:
        starts.append(starts[-1] + n + gap)
    total = starts[-1] + 4
    wide = rows(g, total, 600)
    c_out, r_out = wide[:, :512], rows(g, total, 64)
    c_old, r_old = wide.clone(), r_out.clone()
    fl = flags_for(len(lens))
    L.pfkv_latent_gather(cache, pages(bt, i32(lens)), i32(starts), max(lens), c_out, r_out, flags=fl)
    torch.cuda.synchronize()
    assert not fl.any()
    keep = torch.ones(total, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        c, r = latent_values(cache, bt[b], n)
        s = slice(starts[b], starts[b] + n)
        keep[s] = False
        assert torch.equal(c_out[s], c.to(torch.bfloat16) if not fp8 else c.float().to(torch.bfloat16))
        assert torch.equal(r_out[s], r.to(torch.bfloat16))
    assert torch.equal(wide[keep], c_old[keep]) and torch.equal(wide[:, 512:], c_old[:, 512:])
    assert torch.equal(r_out[keep], r_old[keep])


def test_gather_flags():
    g = gen(32)
    lens = [40, 20, 33, 17, 10]
    bt, num = tables([3, 2, 3, 2, 1], seed=10)
    cache = latent_pool(g, num, True, tags=True)
    expected = cache.page_tags[bt.long().clamp(min=0)].contiguous()
    expected[1, 1] ^= 2
    bt[2, 0] = -1
    starts = [0, 40, 60, 93, 109, 119]               # request 3 has room for 16 rows of its 17
    c_out, r_out = rows(g, 118, 512), rows(g, 118, 64)   # and request 4 runs past the arrays
    old = c_out.clone()
    fl = flags_for(5)
    L.pfkv_latent_gather(cache, pages(bt, i32(lens), expected=expected), i32(starts), 40, c_out, r_out, flags=fl)
    torch.cuda.synchronize()
    assert fl[:5].tolist() == [0, 1, 2, 4, 4]
    assert torch.equal(c_out[93:], old[93:])
    assert c_out[40:56].flatten().any() and not c_out[56:60].any()     # the stale page's rows are zero
    assert not c_out[60:76].any() and not r_out[60:76].any() and c_out[76:93].any()
    fl.zero_()
    L.pfkv_latent_gather(cache, pages(bt, i32(lens), expected=expected), i32(starts), 39, c_out, r_out, flags=fl)
    torch.cuda.synchronize()
    assert fl[:5].tolist() == [4, 1, 2, 4, 4]        # longer than the caller's bound


def test_an_empty_batch_is_a_no_op():
    g = gen(33)
    cache = latent_pool(g, 4, False)
    empty = B.Pages(0, 1, i32([0]), 1, 0, i32([0]), 1, 0, None)
    x = torch.zeros(0, 1, 512, dtype=torch.bfloat16, device="cuda")
    L.pfkv_latent_append(cache, empty, R.Rope(inv_freq()), i32([0]), x, x[..., :64])
    L.pfkv_latent_gather(cache, empty, i32([0]), 5, rows(g, 1, 512), rows(g, 1, 64))
