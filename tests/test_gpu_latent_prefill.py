"""pfkv_latent_prefill_attn against attention in 64 bits: ragged packed prompts
from one token to many tiles, prefixes, queries that see no key, strides, NaN
behind the last sequence and in hidden keys' neighbours, flags and graphs."""
import pytest
import torch

from latent_cases import BF16, SCALE, close, flags_for, gen, i32, rows, score_error, softmax_attend
from paged_fp8_kv_decode_gb300 import latent as L

pytestmark = pytest.mark.gpu


def starts_of(n, gap=0):
    s = [0]
    for x in n:
        s.append(s[-1] + x + gap)
    return s


def inputs(g, Tq, Tk, H):
    kv = rows(g, Tk, H, 256, outliers=0)
    return dict(qn=rows(g, Tq, H, 128, outliers=0), qr=rows(g, Tq, H, 64, outliers=0), kn=kv[..., :128], v=kv[..., 128:],
                kr=rows(g, Tk, 64, outliers=0))


def run(x, qs, ks, max_q, causal=True, scale=SCALE, out=None):
    out = torch.full(x["qn"].shape, 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    fl = flags_for(len(qs) - 1)
    fl.fill_(0x55)
    L.pfkv_latent_prefill_attn(x["qn"], x["qr"], x["kn"], x["kr"], x["v"], i32(qs), i32(ks), max_q, scale, causal, out,
                               flags=fl)
    torch.cuda.synchronize()
    return out, fl[:len(qs) - 1].tolist()


def check(x, q, k, out, causal=True, scale=SCALE, heads=None):
    """Query rows q = (start, end), key rows k, of one request."""
    nq, nk = q[1] - q[0], k[1] - k[0]
    if nq == 0:
        return
    seen = torch.ones(nq, nk, dtype=torch.bool, device="cuda")
    if causal:
        seen = seen.tril(nk - nq)
    for h in range(x["qn"].shape[1]) if heads is None else heads:
        qq = torch.cat((x["qn"][q[0]:q[1], h], x["qr"][q[0]:q[1], h]), 1).double()
        kk = torch.cat((x["kn"][k[0]:k[1], h], x["kr"][k[0]:k[1]]), 1).double()
        if nk == 0:
            assert not out[q[0]:q[1], h].any()
            continue
        s = torch.where(seen, qq @ kk.T * scale, -torch.inf)
        o, tol = softmax_attend(s, x["v"][k[0]:k[1], h].double(), BF16, score_error(qq, kk, scale))
        close(out[q[0]:q[1], h], o, tol, (q, k, h))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,nq,pre", [
    (1, [1], [0]),
    (3, [127, 128, 129], [0, 0, 0]),
    (2, [255, 256, 257, 1, 3], [0, 1, 127, 300, 5]),
    (5, [64, 0, 31], [0, 40, 100]),
    (16, [700, 33], [0, 513]),
    (128, [5, 140], [0, 0]),
])
def test_ragged(H, nq, pre, causal):
    g = gen(61 + H)
    nk = [a + p for a, p in zip(nq, pre)]
    qs, ks = starts_of(nq), starts_of(nk)
    x = inputs(g, qs[-1] + 2, ks[-1] + 3, H)
    for t in ("qn", "qr", "kn", "v"):                # rows behind the last sequence
        x[t][qs[-1] if t[0] == "q" else ks[-1]:] = float("nan")
    x["kr"][ks[-1]:] = float("nan")
    out, fl = run(x, qs, ks, max(nq) + 9, causal)
    assert not any(fl)
    for b in range(len(nq)):
        check(x, (qs[b], qs[b + 1]), (ks[b], ks[b + 1]), out, causal)
    assert (out[qs[-1]:] == 7.0).all()


def test_a_neighbours_keys_do_not_leak():
    """The request behind holds NaN and infinity: rows of a tile that are not the
    request's own must not reach its sums."""
    g = gen(62)
    nq = [100, 60, 130]
    qs = starts_of(nq)
    x = inputs(g, qs[-1], qs[-1], 2)
    for t in ("kn", "v", "qn"):
        x[t][qs[1]:qs[2]] = float("nan")
    x["kr"][qs[1]:qs[2]] = float("inf")
    out, _ = run(x, qs, qs, 130)
    check(x, (qs[0], qs[1]), (qs[0], qs[1]), out)
    check(x, (qs[2], qs[3]), (qs[2], qs[3]), out)


def test_queries_before_every_key_are_zero():
    """More queries than keys: the first of them see nothing."""
    g = gen(63)
    x = inputs(g, 300 + 40, 170 + 0, 3)
    qs, ks = [0, 300, 340], [0, 170, 170]
    out, fl = run(x, qs, ks, 300)
    assert not any(fl)
    assert not out[:130].any() and not out[300:].any()
    check(x, (130, 300), (0, 170), out)


@pytest.mark.parametrize("grow", [1, -1])
def test_scores_far_apart(grow):
    g = gen(64)
    n = 600
    x = inputs(g, n, n, 2)
    x["kr"][:] = (grow * torch.arange(n, device="cuda")[:, None] / 4.0).to(torch.bfloat16)
    x["qr"][:] = 1.0
    x["qr"][:, 1] = -1.0
    out, _ = run(x, [0, n], [0, n], n, scale=0.1)
    check(x, (0, n), (0, n), out, scale=0.1)


def test_strides_and_gaps_between_requests():
    """Queries as slices of one row of 192, heads in reversed storage order, key
    rows shared by two requests, gaps between the requests' output rows."""
    g = gen(65)
    H, nq = 4, [90, 200]
    Tq = 400
    q = rows(g, H, Tq, 192, outliers=0).transpose(0, 1)
    kv = rows(g, H, 260, 256, outliers=0).transpose(0, 1)
    x = dict(qn=q[..., :128], qr=q[..., 128:], kn=kv[..., :128], v=kv[..., 128:], kr=rows(g, 260, 72, outliers=0)[:, :64])
    wide = torch.full((Tq, H, 136), 7.0, dtype=torch.bfloat16, device="cuda")
    out, fl = run(x, [10, 100, 300], [0, 260, 260], 200, out=wide[..., :128])
    assert not any(fl)
    check(x, (10, 100), (0, 260), out)
    assert not out[100:300].any()                    # the second request has no key
    assert (wide[:10] == 7.0).all() and (wide[300:] == 7.0).all() and (wide[..., 128:] == 7.0).all()


def test_flags():
    g = gen(66)
    x = inputs(g, 100, 100, 2)
    for qs, ks, want in (([0, 50, 40, 100], [0, 50, 60, 100], [0, 4, 0]),
                         ([0, 50, 101, 101], [0, 50, 60, 70], [0, 4, 4]),
                         ([0, 10, 20, 30], [-1, 10, 20, 101], [4, 0, 4]),
                         ([0, 61, 70, 80], [0, 61, 70, 80], [4, 0, 0])):
        out, fl = run(x, qs, ks, 60)
        assert fl == want, (qs, ks)
        for b, f in enumerate(fl):
            # two requests that claim the same rows (40 to 49 of the first list) race on them
            shared = any(i != b and not fl[i] and qs[i] < qs[b + 1] and qs[b] < qs[i + 1] for i in range(3))
            if not f and not shared:
                check(x, (qs[b], qs[b + 1]), (ks[b], ks[b + 1]), out)
        if want[0]:
            assert (out[:qs[1]] == 7.0).all()


def test_one_long_prompt():
    g = gen(67)
    n = 2500
    x = inputs(g, n, n, 8)
    out, _ = run(x, [0, n], [0, n], n)
    check(x, (0, n), (0, n), out, heads=(0, 3, 7))
    again, _ = run(x, [0, n], [0, n], n)
    assert torch.equal(out, again)


def test_a_graph_replayed_with_new_starts():
    g = gen(68)
    x = inputs(g, 400, 400, 4)
    qs = i32([0, 100, 400])
    out = torch.zeros(400, 4, 128, dtype=torch.bfloat16, device="cuda")
    call = lambda: L.pfkv_latent_prefill_attn(x["qn"], x["qr"], x["kn"], x["kr"], x["v"], qs, qs, 400, SCALE, True, out)  # noqa: E731
    call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call()
    for new in ([0, 100, 400], [0, 399, 400], [0, 0, 400]):
        qs.copy_(i32(new))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(new, new[1:]):
            check(x, (a, b), (a, b), out)
