"""pfkv_rope_append against the rotation and the quantisation in 64 bits, and
against pfkv_kv_append: padded and packed rows, strides, one length a request or
a length a head, partial rotations, far and negative positions, pages that the
call opens or continues, tags, and what it must leave alone."""
import pytest
import torch

from latent_cases import (BF16, E4M3, PAGE, TURN, close, flags_for, gen, i32, pages, rows, tables, turned)
from paged_fp8_kv_decode_gb300 import binding as B
from paged_fp8_kv_decode_gb300 import rope as R

pytestmark = pytest.mark.gpu


def inv_freq(rot):
    return (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()


def pool(g, num_pages, Hkv, D, fp8, tags=False):
    shape = (num_pages, Hkv, PAGE, D)
    t = torch.randint(-2 ** 31, 2 ** 31 - 1, (num_pages, Hkv), generator=g, device="cuda", dtype=torch.int32) if tags else None
    if not fp8:
        return B.Cache(rows(g, *shape), rows(g, *shape), None, None, t)
    code = lambda: torch.randint(0, 127, shape, generator=g, device="cuda").to(torch.uint8)  # noqa: E731
    scale = lambda: torch.rand(shape[:2], generator=g, device="cuda") * 0.1 + 0.05  # noqa: E731
    return B.Cache(code(), code(), scale(), scale(), t)


def clone(c):
    return B.Cache(*[None if t is None else t.clone() for t in
                     (c.k_pages, c.v_pages, c.k_scale, c.v_scale, c.page_tags)])


def check_keys(got, before, bt, ctx, n, k, size, fp8, head=None):
    """One request's turned keys k [n, Hkv, D] in 64 bits (size: |a| + |b|)
    against the pool: values, scales, and that scales of continued pages stayed."""
    for at in range(-(ctx % PAGE), n, PAGE):
        t0, t1 = max(0, at), min(n, at + PAGE)
        slot, pg = (ctx + t0) % PAGE, int(bt[(ctx + t0) // PAGE])
        hs = slice(None) if head is None else slice(head, head + 1)
        want, sz = k[t0:t1].transpose(0, 1), size[t0:t1].transpose(0, 1)     # [H, tokens, D]
        stored = got.k_pages[pg, hs, slot:slot + t1 - t0]
        if not fp8:
            close(stored, want, BF16 * want.abs() + TURN * sz, "bf16 keys")
            continue
        z = got.k_scale[pg, hs].double()
        if slot == 0:
            top = want.abs().amax((1, 2))
            close(z, torch.where(top == 0, 1.0, top / 448), 2 * TURN * sz.amax((1, 2)) / 448 + 1e-12, "scale")
        else:
            assert torch.equal(got.k_scale[pg, hs], before.k_scale[pg, hs])
        y = want / z[:, None, None]
        yc = y.clamp(-448, 448)
        v = stored.view(torch.float8_e4m3fn).double()
        # half a step, or half of the subnormal step 2^-9, of a quotient that the
        # rotation's error moves (a move of the scale moves both alike)
        close(v, yc, E4M3 * yc.abs() + 2.0 ** -10 + 4 * TURN * sz / z[:, None, None] * (1 + E4M3), "codes")


CASES = [
    # B, T, Hq, Hkv, D, rot, inter, fp8, ctx, packed
    (3, 1, 32, 8, 128, 128, False, True, [0, 15, 8191], False),
    (2, 1, 1, 1, 64, 64, True, False, [16, 100], False),
    (4, 5, 8, 2, 64, 32, True, True, [3, 14, 0, 700000], False),
    (2, 37, 6, 3, 128, 64, False, True, [0, 7], False),
    (3, 50, 4, 4, 128, 16, True, False, [5, 0, 31], True),
    (5, 200, 16, 2, 128, 128, False, True, [0, 1, 15, 16, 33], True),
    (1, 333, 8, 8, 64, 64, False, True, [250], True),
    (2, 16, 2, 1, 128, 96, False, False, [0, 8], False),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_against_the_definition_and_the_plain_append(case):
    Bn, T, Hq, Hkv, D, rot, inter, fp8, ctx, packed = case
    g = gen(11 + T + D)
    n = [T] * Bn if not packed else [max(1, (T * (b + 1)) // Bn - b) for b in range(Bn)]
    if packed and Bn > 2:
        n[1] = 0
    first, last = [c // PAGE for c in ctx], [(c + max(k, 1) - 1) // PAGE + 1 for c, k in zip(ctx, n)]
    bt, num = tables(last, seed=T, first=first)
    cache = pool(g, num, Hkv, D, fp8)
    before = clone(cache)
    lead = (sum(n) + 3,) if packed else (Bn, T)            # three rows behind the last sequence
    q, k, v = rows(g, *lead, Hq, D), rows(g, *lead, Hkv, D), rows(g, *lead, Hkv, D)
    q_out = rows(g, *lead, Hq, D)
    q_before = q_out.clone()
    starts = [0]
    for x in n:
        starts.append(starts[-1] + x)
    fl = flags_for(Bn)
    f = inv_freq(rot)
    pg = pages(bt, i32(ctx))
    R.pfkv_rope_append(cache, pg, R.Rope(f, inter, 1.25), i32(ctx), k, v, q, q_out,
                       row_starts=i32(starts) if packed else None, max_new_tokens=T, flags=fl)
    torch.cuda.synchronize()
    assert not fl.any()
    touched = torch.zeros(num, PAGE, dtype=torch.bool)
    for b in range(Bn):
        rw = (slice(starts[b], starts[b + 1]),) if packed else (b,)
        pos = ctx[b] + torch.arange(n[b], device="cuda")
        want, size = turned(q[rw], pos, f, inter, 1.25)
        close(q_out[rw], want, BF16 * want.abs() + TURN * size, "queries")
        want, size = turned(k[rw], pos, f, inter, 1.25)
        check_keys(cache, before, bt[b].cpu(), ctx[b], n[b], want, size, fp8)
        for t in range(n[b]):
            touched[int(bt[b, (ctx[b] + t) // PAGE]), (ctx[b] + t) % PAGE] = True
    # values: the plain append's bytes; slots that no token goes to: as they were
    same = clone(before)
    if packed:
        pad = torch.zeros(Bn, Hkv, T, D, dtype=torch.bfloat16, device="cuda")
        for b in range(Bn):
            pad[b, :, :n[b]] = v[starts[b]:starts[b + 1]].transpose(0, 1)
    else:
        pad = v.transpose(1, 2).contiguous()
    B.pfkv_kv_append(same, pg, i32(ctx), pad, pad, new_lens=i32(n))
    assert torch.equal(cache.v_pages, same.v_pages)
    if fp8:
        assert torch.equal(cache.v_scale, same.v_scale)
    rest = ~touched.cuda()
    for a, z in ((cache.k_pages, before.k_pages), (cache.v_pages, before.v_pages)):
        assert torch.equal(a.transpose(1, 2)[rest], z.transpose(1, 2)[rest])
    if packed:
        assert torch.equal(q_out[starts[-1]:], q_before[starts[-1]:])


def test_strided_rows_in_place_and_a_broadcast_key():
    """q, k and v as slices of one projection's rows, q turned in place, and one
    key row for all heads (stride 0)."""
    g = gen(5)
    Bn, T, Hq, Hkv, D = 2, 3, 4, 2, 128
    ctx = [9, 30]
    bt, num = tables([1 + (c + T - 1) // PAGE for c in ctx], seed=1)
    qkv = rows(g, Bn, T, Hq + 2 * Hkv, D)
    q, v = qkv[:, :, :Hq], qkv[:, :, Hq + Hkv:]
    k = qkv[:, :, Hq:Hq + 1].expand(-1, -1, Hkv, -1)
    old, f = qkv.clone(), inv_freq(D)
    cache = pool(g, num, Hkv, D, True)
    before = clone(cache)
    R.pfkv_rope_append(cache, pages(bt, i32(ctx)), R.Rope(f), i32(ctx), k, v, q, q)
    torch.cuda.synchronize()
    for b in range(Bn):
        pos = ctx[b] + torch.arange(T, device="cuda")
        want, size = turned(old[b, :, :Hq], pos, f, False)
        close(qkv[b, :, :Hq], want, BF16 * want.abs() + TURN * size, "in place")
        want, size = turned(old[b, :, Hq:Hq + 1].expand(-1, Hkv, -1), pos, f, False)
        check_keys(cache, before, bt[b].cpu(), ctx[b], T, want, size, True)
    assert torch.equal(qkv[:, :, Hq:], old[:, :, Hq:])


def test_a_length_a_head_and_a_position_of_its_own():
    """Evicted heads: every head appends at its own slot, all turn by the token's
    true position."""
    g = gen(6)
    Bn, T, Hkv, D = 2, 21, 3, 128
    ctx = [[0, 5, 47], [16, 31, 2]]
    true = [100000, -40]
    mp, num = 6, 40
    perm = torch.stack([torch.randperm(num, generator=torch.Generator().manual_seed(h))[:Bn * mp] for h in range(Hkv)])
    bt = perm.view(Hkv, Bn, mp).transpose(0, 1).contiguous().to(torch.int32).cuda()
    pos = i32(ctx)
    pg = B.Pages(Bn, mp, bt, Hkv * mp, mp, pos, Hkv, 1, None)
    k, v = rows(g, Bn, T, Hkv, D), rows(g, Bn, T, Hkv, D)
    q = rows(g, Bn, T, 2, D)
    q_out = torch.zeros_like(q)
    cache, f, fl = pool(g, num, Hkv, D, True), inv_freq(D), flags_for(Bn)
    before = clone(cache)
    with pytest.raises(B.PfkvError):  # whose position would it be?
        R.pfkv_rope_append(cache, pg, R.Rope(f), pos, k, v)
    R.pfkv_rope_append(cache, pg, R.Rope(f), pos, k, v, q, q_out, rope_positions=i32(true), flags=fl)
    torch.cuda.synchronize()
    assert not fl.any()
    for b in range(Bn):
        p = true[b] + torch.arange(T, device="cuda")
        want, size = turned(q[b], p, f, False)
        close(q_out[b], want, BF16 * want.abs() + TURN * size, "queries")
        want, size = turned(k[b], p, f, False)
        for h in range(Hkv):
            check_keys(cache, before, bt[b, h].cpu(), ctx[b][h], T, want[:, h:h + 1], size[:, h:h + 1], True, head=h)


def test_bad_destinations_are_flagged_and_not_written():
    g = gen(7)
    Bn, T, Hkv, D = 6, 4, 2, 64
    ctx = [0, 16, -1, 62, 0, 20]
    bt, num = tables([4] * Bn, seed=3)
    cache = pool(g, num, Hkv, D, True, tags=True)
    expected = cache.page_tags[bt.long().clamp(min=0), 0].contiguous()
    cache.page_tags[:, 1] = cache.page_tags[:, 0]
    bt[1, 1] = num                                   # outside the pool
    expected[4, 0] ^= 1                              # reallocated since
    before = clone(cache)
    k, v = rows(g, Bn, T, Hkv, D), rows(g, Bn, T, Hkv, D)
    q, q_out = rows(g, Bn, T, 1, D), torch.zeros(Bn, T, 1, D, dtype=torch.bfloat16, device="cuda")
    fl = flags_for(Bn)
    fl[5] = 0x40                                     # bits are OR-ed in
    R.pfkv_rope_append(cache, pages(bt, i32(ctx), expected=expected), R.Rope(inv_freq(D)), i32(ctx), k, v, q, q_out,
                       flags=fl)
    torch.cuda.synchronize()
    assert fl[:6].tolist() == [0, 2, 4, 4, 1, 0x40]  # request 3 runs off its table
    changed = (cache.k_pages != before.k_pages).flatten(1).any(1).nonzero().flatten().tolist()
    assert set(changed) == {int(bt[0, 0]), int(bt[3, 3]), int(bt[5, 1])}
    assert q_out.flatten(1).any(1).all()             # queries are turned all the same


def test_bad_packed_rows_are_flagged():
    g = gen(8)
    ctx = [0, 0, 0]
    bt, num = tables([2] * 3, seed=4)
    cache = pool(g, num, 1, 64, False)
    before = clone(cache)
    k = rows(g, 20, 1, 64)
    q_out = torch.zeros_like(k)
    for starts, want in (([0, 12, 11, 15], [0, 4, 0]), ([0, 4, 25, 26], [0, 4, 4]), ([-1, 3, 3, 5], [4, 0, 0])):
        fl = flags_for(3)
        R.pfkv_rope_append(cache, pages(bt, i32(ctx)), R.Rope(inv_freq(64)), i32(ctx), k, k, k, q_out,
                           row_starts=i32(starts), max_new_tokens=12, flags=fl)
        torch.cuda.synchronize()
        assert fl[:3].tolist() == want, starts
    fl = flags_for(3)                                # longer than max_new_tokens
    R.pfkv_rope_append(clone(before), pages(bt, i32(ctx)), R.Rope(inv_freq(64)), i32(ctx), k, k,
                       row_starts=i32([0, 13, 14, 15]), max_new_tokens=12, flags=fl)
    torch.cuda.synchronize()
    assert fl[:3].tolist() == [4, 0, 0]


def test_new_lens_bound_what_is_written():
    g = gen(9)
    T, ctx, n = 9, [10, 3, 0], [9, 0, 4]
    bt, num = tables([2] * 3, seed=5)
    cache = pool(g, num, 2, 128, True)
    k, q = rows(g, 3, T, 2, 128), rows(g, 3, T, 4, 128)
    q_out = torch.zeros_like(q)
    before = clone(cache)
    f = inv_freq(128)
    R.pfkv_rope_append(cache, pages(bt, i32(ctx)), R.Rope(f), i32(ctx), k, k, q, q_out, new_lens=i32(n))
    torch.cuda.synchronize()
    for b in range(3):
        want, size = turned(k[b, :n[b]], ctx[b] + torch.arange(n[b], device="cuda"), f, False)
        check_keys(cache, before, bt[b].cpu(), ctx[b], n[b], want, size, True)
        assert not q_out[b, n[b]:].any()
        assert q_out[b, :n[b]].flatten(1).any(1).all()
    assert torch.equal(cache.k_pages[bt[1].long()], before.k_pages[bt[1].long()])


def test_zero_rows_and_extreme_values():
    """A unit of zeros takes scale 1 (its zeros may be negative: a zero times a
    negative cosine); a value near the largest bf16 reaches the codes as 448."""
    g = gen(10)
    bt, num = tables([1, 1], seed=6)
    cache = pool(g, num, 1, 128, True)
    k = torch.zeros(2, 3, 1, 128, dtype=torch.bfloat16, device="cuda")
    k[1, 0, 0, 127] = 3.0e38
    R.pfkv_rope_append(cache, pages(bt, i32([0, 0])), R.Rope(inv_freq(32)), i32([0, 0]), k, k)
    torch.cuda.synchronize()
    p0, p1 = int(bt[0, 0]), int(bt[1, 0])
    assert float(cache.k_scale[p0, 0]) == 1.0 and not (cache.k_pages[p0, 0, :3] & 0x7F).any()
    assert int(cache.k_pages[p1, 0, 0, 127]) == 0x7E and float(cache.k_scale[p1, 0]) > 1e35


def test_another_stream_and_a_captured_graph():
    g = gen(12)
    ctx = [5, 40]
    bt, num = tables([4, 4], seed=7)
    k, q = rows(g, 2, 1, 2, 128), rows(g, 2, 1, 8, 128)
    f = R.Rope(inv_freq(128))
    ref = pool(g, num, 2, 128, True)
    cache, want = clone(ref), torch.empty_like(q)
    pos = i32(ctx)
    R.pfkv_rope_append(ref, pages(bt, pos), f, pos, k, k, q, want)
    torch.cuda.synchronize()
    got = torch.zeros_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        R.pfkv_rope_append(cache, pages(bt, pos), f, pos, k, k, q, got)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(cache.k_pages, ref.k_pages)
    pos.add_(1)                                      # a replay reads the current contents
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(got, want)


def test_many_requests_and_the_empty_batch():
    """More CTAs than one wave; then no request at all."""
    g = gen(13)
    Bn = 700
    ctx = [(37 * b) % 90 for b in range(Bn)]
    bt, num = tables([c // PAGE + 1 for c in ctx], seed=8, first=[c // PAGE for c in ctx])
    cache, f = pool(g, num, 2, 64, True), inv_freq(64)
    k, q = rows(g, Bn, 1, 2, 64), rows(g, Bn, 1, 5, 64)
    q_out = torch.empty_like(q)
    R.pfkv_rope_append(cache, pages(bt, i32(ctx)), R.Rope(f), i32(ctx), k, k, q, q_out)
    torch.cuda.synchronize()
    want, size = turned(q[:, 0], i32(ctx), f, False)
    close(q_out[:, 0], want, BF16 * want.abs() + TURN * size, "queries")
    none = torch.zeros(0, 1, 2, 64, dtype=torch.bfloat16, device="cuda")
    R.pfkv_rope_append(cache, B.Pages(0, 1, bt, 1, 0, i32([0]), 1, 0, None), R.Rope(f), i32([0]), none, none)
