"""pfkv_latent_decode_attn against attention in 64 bits: head counts from one to
more than a tile holds, several query tokens, lengths from none to many pages,
both pool types, strides, stale slots that hold NaN, page scales far apart,
scores far apart, flags, graphs and repeated calls."""
import pytest
import torch

from latent_cases import (BF16, F16, PAGE, SCALE, close, flags_for, gen, i32, latent_pool, latent_values, pages, rows,
                          score_error, softmax_attend, tables)
from paged_fp8_kv_decode_gb300 import binding as B
from paged_fp8_kv_decode_gb300 import latent as L

pytestmark = pytest.mark.gpu


def run(cache, bt, lens, qc, qr, scale=SCALE, max_len=None, expected=None, out=None):
    Bn, kq, H, _ = qc.shape
    pg = pages(bt, lens if torch.is_tensor(lens) else i32(lens), expected=expected)
    top = max_len if max_len is not None else max(1, max(lens))
    ws = torch.empty(L.pfkv_latent_decode_workspace_size(cache, pg, H, kq, top), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)                                   # its contents on entry are ignored
    out = torch.full_like(qc, 7.0) if out is None else out
    fl = flags_for(Bn)
    fl.fill_(0x55)
    L.pfkv_latent_decode_attn(cache, pg, qc, qr, scale, top, ws, out, flags=fl)
    torch.cuda.synchronize()
    assert (fl[Bn:] == 0x55).all()
    return out, fl[:Bn].tolist()


def check(cache, bt, lens, qc, qr, out, scale=SCALE, skip=()):
    """Every row against the definition; the tolerance counts one rounding of a
    weight (bf16, or f16 for an FP8 pool), of q (FP8: f16 after scaling, exact
    here but for elements far below the row's largest) and of the output."""
    Bn, kq, H, _ = qc.shape
    fp8 = cache.c_pages.dtype == torch.uint8
    for b in range(Bn):
        if b in skip:
            assert not out[b].any()
            continue
        n = lens[b]
        c, r = latent_values(cache, bt[b], max(n, 0))
        for t in range(kq):
            m = n - kq + 1 + t
            if m <= 0:
                assert not out[b, t].any(), (b, t)
                continue
            k = torch.cat((c[:m], r[:m]), 1)
            q = torch.cat((qc[b, t], qr[b, t]), 1).double()
            err = score_error(q, k, scale)
            s = q @ k.T * scale
            o, tol = softmax_attend(s, c[:m], F16 if fp8 else BF16, err)
            if fp8:
                # f16 weights p_j z_j (z_j: the page's scale) over a reference that leaves
                # the largest at 2^7 or more: below 2^-14 they have an absolute step of
                # 2^-24, half of it is 2^-25 = 2^-32 of the largest.  In p_j that is 2^-32
                # max(p z) / z_j, which meets c_j in the product and o in the sum.
                z = cache.c_scale[bt[b, :(m + PAGE - 1) // PAGE].long()].double().repeat_interleave(PAGE)[:m]
                pz = (torch.softmax(s, -1) * z).amax(-1, keepdim=True)
                tol = tol + 2.0 ** -32 * pz * ((c[:m].abs() / z[:, None]).sum(0) + o.abs() * (1 / z).sum())
            close(out[b, t], o, tol, (b, t, n))


SHAPES = [
    # H, kq, lens
    (1, 1, [1, 2, 17]),
    (16, 1, [1000]),
    (16, 1, [64, 65, 63, 128, 1, 0, 500]),
    (128, 1, [300, 5, 129]),
    (128, 2, [200, 1, 77]),
    (20, 3, [90, 2, 16]),
    (64, 1, [63, 64, 65]),
    (5, 7, [400, 33]),
    (160, 1, [70, 200]),
    (33, 4, [1, 3, 4, 130]),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,kq,lens", SHAPES)
def test_shapes(H, kq, lens, fp8):
    g = gen(41 + H)
    bt, num = tables([(n + PAGE - 1) // PAGE for n in lens], seed=H)
    cache = latent_pool(g, num, fp8)
    qc, qr = rows(g, len(lens), kq, H, 512, outliers=0), rows(g, len(lens), kq, H, 64, outliers=0)
    out, fl = run(cache, bt, lens, qc, qr)
    assert not any(fl)
    check(cache, bt, lens, qc, qr, out)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,lens", [(16, [20000]), (128, [9001, 4100]), (64, [3001] * 40)])
def test_long_contexts_are_split_and_merged(H, lens, fp8):
    g = gen(43)
    bt, num = tables([(n + PAGE - 1) // PAGE for n in lens], seed=H)
    cache = latent_pool(g, num, fp8)
    qc, qr = rows(g, len(lens), 1, H, 512, outliers=0), rows(g, len(lens), 1, H, 64, outliers=0)
    out, _ = run(cache, bt, lens, qc, qr)
    check(cache, bt, lens, qc, qr, out)
    again, _ = run(cache, bt, lens, qc, qr)
    assert torch.equal(out, again)                   # the same bits every time


@pytest.mark.parametrize("fp8", [False, True])
def test_stale_slots_hold_nan(fp8):
    """Slots past the last token, and pages that no table names, hold NaN bytes."""
    g = gen(44)
    lens = [1, 15, 16, 17, 63, 64, 65, 200]
    bt, num = tables([(n + PAGE - 1) // PAGE for n in lens], seed=4)
    fill = latent_pool(g, num, fp8, fill=0xFF)       # NaN in e4m3 and in bf16
    good = latent_pool(g, num, fp8)
    cache = L.LatentCache(fill.c_pages, fill.r_pages, good.c_scale)
    for b, n in enumerate(lens):
        for j in range(n):
            p, s = int(bt[b, j // PAGE]), j % PAGE
            cache.c_pages[p, s], cache.r_pages[p, s] = good.c_pages[p, s], good.r_pages[p, s]
    for H, kq in ((16, 1), (128, 2)):
        qc, qr = rows(g, len(lens), kq, H, 512, outliers=0), rows(g, len(lens), kq, H, 64, outliers=0)
        out, _ = run(cache, bt, lens, qc, qr)
        check(cache, bt, lens, qc, qr, out)


@pytest.mark.parametrize("spread", [4.0, 40.0])
def test_page_scales_far_apart(spread):
    """FP8 pages whose scales differ by up to 2^40: large pages that carry no
    weight must not cost the small ones their precision."""
    g = gen(45)
    n = 400
    bt, num = tables([n // PAGE], seed=5)
    cache = latent_pool(g, num, True)
    e = (torch.rand(num, generator=g, device="cuda") - 1.0) * spread
    cache.c_scale.copy_(torch.exp2(e.round()) * 0.01)
    qc, qr = rows(g, 1, 1, 32, 512, outliers=0), rows(g, 1, 1, 32, 64, outliers=0) * 8
    out, _ = run(cache, bt, [n], qc, qr, scale=0.05)
    check(cache, bt, [n], qc, qr, out, scale=0.05)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("grow", [1, -1])
def test_scores_far_apart(fp8, grow):
    """Scores that climb (or fall) by hundreds along the tokens: the running
    maximum moves at every tile, and old sums vanish."""
    g = gen(46)
    n, H = 700, 24
    bt, num = tables([(n + PAGE - 1) // PAGE], seed=6)
    cache = latent_pool(g, num, fp8)
    for j in range(n):
        cache.r_pages[int(bt[0, j // PAGE]), j % PAGE] = grow * (j - n / 2) / 8.0
    qc = rows(g, 1, 1, H, 512, outliers=0)
    qr = torch.ones(1, 1, H, 64, device="cuda").to(torch.bfloat16)
    qr[:, :, ::2] = -1                               # half of the rows see them the other way round
    out, _ = run(cache, bt, [n], qc, qr, scale=0.1)
    check(cache, bt, [n], qc, qr, out, scale=0.1)


def test_a_query_row_with_small_elements():
    """FP8 pools take q as f16 after a power-of-two scaling: rows of very large
    and of very small values keep their precision."""
    g = gen(47)
    lens = [150]
    bt, num = tables([10], seed=7)
    cache = latent_pool(g, num, True)
    qc, qr = rows(g, 1, 1, 8, 512, outliers=0), rows(g, 1, 1, 8, 64, outliers=0)
    for h in range(8):
        f = 2.0 ** (40 * (h - 4))
        qc[0, 0, h] = (qc[0, 0, h].float() * f).to(torch.bfloat16)
        qr[0, 0, h] = (qr[0, 0, h].float() * f).to(torch.bfloat16)
    for h in (2, 3, 4):                              # one scale suits one magnitude at a time
        s = SCALE / 2.0 ** (40 * (h - 4))
        out, _ = run(cache, bt, lens, qc[:, :, h:h + 1].contiguous(), qr[:, :, h:h + 1].contiguous(), scale=s)
        check(cache, bt, lens, qc[:, :, h:h + 1], qr[:, :, h:h + 1], out, scale=s)


@pytest.mark.parametrize("fp8", [False, True])
def test_strides_and_neighbours(fp8):
    """q and out as parts of wider rows, heads before tokens; what lies between
    stays as it was."""
    g = gen(48)
    Bn, kq, H = 2, 3, 10
    lens = [100, 47]
    bt, num = tables([7, 3], seed=8)
    cache = latent_pool(g, num, fp8)
    q = rows(g, Bn, H, kq, 640, outliers=0)
    qc, qr = q[..., :512].transpose(1, 2), q[..., 512:576].transpose(1, 2)
    wide = rows(g, Bn, H, kq, 528)
    old = wide.clone()
    out, fl = run(cache, bt, lens, qc, qr, out=wide[..., :512].transpose(1, 2))
    assert not any(fl)
    check(cache, bt, lens, qc, qr, out)
    assert torch.equal(wide[..., 512:], old[..., 512:])


def test_one_query_for_all_heads():
    """Broadcast queries (stride 0): every head gives the same row."""
    g = gen(49)
    bt, num = tables([20], seed=9)
    cache = latent_pool(g, num, False)
    qc, qr = rows(g, 1, 1, 1, 512, outliers=0).expand(1, 1, 70, 512), rows(g, 1, 1, 1, 64, outliers=0).expand(1, 1, 70, 64)
    out, _ = run(cache, bt, [310], qc, qr, out=torch.empty(1, 1, 70, 512, dtype=torch.bfloat16, device="cuda"))
    check(cache, bt, [310], qc, qr, out)
    assert torch.equal(out[0, 0, :1].expand(70, 512), out[0, 0])


@pytest.mark.parametrize("fp8", [False, True])
def test_flags_zero_the_request_alone(fp8):
    g = gen(50)
    lens = [700, 300, 2000, 40, -3, 81, 100]
    n_pages = [(max(n, 1) + PAGE - 1) // PAGE for n in lens]
    bt, num = tables(n_pages, seed=10)
    cache = latent_pool(g, num, fp8, tags=True)
    expected = cache.page_tags[bt.long().clamp(min=0)].contiguous()
    expected[0, 40] ^= 1                             # a stale page
    bt[1, 18] = num + 5                              # its last page is outside the pool
    bt[3, 0] = -1
    qc, qr = rows(g, 7, 1, 48, 512, outliers=0), rows(g, 7, 1, 48, 64, outliers=0)
    good = bt.clone()
    out, fl = run(cache, bt, i32(lens), qc, qr, max_len=2000, expected=expected)
    assert fl == [1, 2, 0, 2, 4, 0, 0]
    check(cache, good, lens, qc, qr, out, skip=(0, 1, 3, 4))
    out, fl = run(cache, bt, i32(lens), qc, qr, max_len=1999, expected=expected)
    assert fl == [1, 2, 4, 2, 4, 0, 0]
    check(cache, good, lens, qc, qr, out, skip=(0, 1, 2, 3, 4))


def test_a_graph_replayed_with_new_lengths_and_two_streams():
    g = gen(51)
    lens = [500, 900]
    bt, num = tables([125, 125], seed=11)
    cache = latent_pool(g, num, True)
    qc, qr = rows(g, 2, 1, 128, 512, outliers=0), rows(g, 2, 1, 128, 64, outliers=0)
    n = i32(lens)
    pg = pages(bt, n)
    size = L.pfkv_latent_decode_workspace_size(cache, pg, 128, 1, 2000)
    ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.zeros_like(qc) for _ in range(2)]
    L.pfkv_latent_decode_attn(cache, pg, qc, qr, SCALE, 2000, ws[0], outs[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        L.pfkv_latent_decode_attn(cache, pg, qc, qr, SCALE, 2000, ws[0], outs[0])
    for new in ([500, 900], [1, 2000], [1777, 16]):
        n.copy_(i32(new))
        graph.replay()
        torch.cuda.synchronize()
        check(cache, bt, new, qc, qr, outs[0])
    a, b = torch.cuda.Stream(), torch.cuda.Stream()  # two calls at once, each with its own workspace
    torch.cuda.synchronize()
    for i, st in enumerate((a, b)):
        outs[i].zero_()
    torch.cuda.synchronize()
    for i, st in enumerate((a, b)):
        L.pfkv_latent_decode_attn(cache, pg, qc, qr, SCALE, 2000, ws[i], outs[i], stream=st)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1])


def test_workspace_too_small():
    g = gen(52)
    bt, num = tables([4], seed=12)
    cache = latent_pool(g, num, False)
    qc, qr = rows(g, 1, 1, 16, 512), rows(g, 1, 1, 16, 64)
    pg = pages(bt, i32([60]))
    size = L.pfkv_latent_decode_workspace_size(cache, pg, 16, 1, 64)
    ws = torch.empty(size - 1, dtype=torch.uint8, device="cuda")
    with pytest.raises(B.PfkvError) as e:
        L.pfkv_latent_decode_attn(cache, pg, qc, qr, SCALE, 64, ws, torch.empty_like(qc))
    assert e.value.status == B.PFKV_ERR_WORKSPACE
