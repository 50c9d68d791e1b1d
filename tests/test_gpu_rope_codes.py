"""Codes of the FP8 appends, byte by byte: the encoding of the fp32 quotient whatever
the elements' size, ties, both zeros, infinities and NaN included."""
import pytest
import torch

from latent_cases import PAGE, flags_for, gen, i32, pages, tables
from paged_fp8_kv_decode_gb300 import binding as B
from paged_fp8_kv_decode_gb300 import latent as L
from paged_fp8_kv_decode_gb300 import rope as R

pytestmark = pytest.mark.gpu


def patterns(g, kind, *shape):
    """bf16 elements, 128 in a row."""
    x = torch.randn(*shape, generator=g, device="cuda")
    if kind == "wide":                               # exponents over the whole range of the type, row by row
        x = x * torch.exp2(torch.randint(-120, 120, shape[:-1] + (1,), generator=g, device="cuda").float())
    elif kind == "outliers":                         # most quotients far below the codes' normal range
        x = torch.where(torch.rand(*shape, generator=g, device="cuda") < 0.002, x * 3e4, x)
    elif kind == "ties":                             # few significant bits: quotients on the middle between codes
        x = torch.randint(-64, 65, shape, generator=g, device="cuda").float() / 8
    elif kind == "zeros":                            # of both signs, and subnormals
        x = torch.where(torch.rand(*shape, generator=g, device="cuda") < 0.5, x.sign() * 0.0, x * 1e-39)
    x = x.to(torch.bfloat16)
    if kind == "special":
        x[..., 3] = float("nan")
        x[0, 0, 1, 5], x[0, 1, 0, 7] = float("inf"), -float("inf")
    return x


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["plain", "wide", "outliers", "ties", "zeros", "special"])
def test_values_get_the_bytes_of_the_plain_append(kind, D):
    g = gen(21)
    Bn, T, H, ctx = 2, 90, 3, [0, 7]
    bt, num = tables([(c + T + PAGE - 1) // PAGE for c in ctx], seed=2)
    def pool():
        return B.Cache(*[torch.zeros(num, H, PAGE, D, dtype=torch.uint8, device="cuda") for _ in range(2)],
                       *[torch.full((num, H), 0.02, device="cuda") for _ in range(2)])
    v = patterns(g, kind, Bn, T, H, D)
    pos = i32(ctx)
    pg = pages(bt, pos)
    got, want = pool(), pool()
    R.pfkv_rope_append(got, pg, R.Rope(torch.ones(D // 2, device="cuda")), pos, v, v, flags=flags_for(Bn))
    t = v.transpose(1, 2).contiguous()
    B.pfkv_kv_append(want, pg, pos, t, t, flags=flags_for(Bn))
    torch.cuda.synchronize()
    assert torch.equal(got.v_pages, want.v_pages)
    assert torch.equal(got.v_scale.view(torch.int32), want.v_scale.view(torch.int32))


@pytest.mark.parametrize("kind", ["plain", "wide", "outliers", "ties", "zeros"])
def test_latents_are_the_encoded_quotients(kind):
    g = gen(22)
    T = 96
    bt, num = tables([T // PAGE], seed=4)
    cache = L.LatentCache(torch.zeros(num, PAGE, 512, dtype=torch.uint8, device="cuda"),
                          torch.zeros(num, PAGE, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(num, device="cuda"))
    c = patterns(g, kind, 1, T, 4, 128).reshape(1, T, 512)
    r = torch.zeros(1, T, 64, dtype=torch.bfloat16, device="cuda")
    zero = i32([0])
    L.pfkv_latent_append(cache, pages(bt, zero), R.Rope(torch.ones(32, device="cuda")), zero, c, r)
    torch.cuda.synchronize()
    page = bt[0, :T // PAGE].long()
    x = c.float().view(-1, PAGE * 512)
    top = x.abs().amax(1, keepdim=True)
    scale = torch.where(top == 0, torch.ones_like(top), top / torch.full_like(top, 448.0))
    assert torch.equal(cache.c_scale[page], scale[:, 0])
    want = (x / scale).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(cache.c_pages[page].view(-1, PAGE * 512), want)
