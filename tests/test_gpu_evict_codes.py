"""The codes and scales that pfkv_kv_evict gives FP8 tokens that move from several units into one,
bit for bit against the definition: the new scale is absmax / 448 (fp32 division; 1 where absmax is 0,
and a NaN is no maximum), a code the e4m3 encoding of fl(fl(c s) / scale), NaN as 0x7F.

Every token kept lies in a unit of its own, so each row of a destination unit has its own old scale,
and what is decided row by row is met at the ratios of scales where it could go wrong."""
import math

import pytest
import torch

from prefix_cases import PAGE, B, gen, evict_call, i32

pytestmark = pytest.mark.gpu


class OneAPage:
    """A pool of one request: token 16 i + 3 of page i has codes[h][i] and scale[h][i], and is kept."""

    def __init__(self, codes, scale):
        H, n, D = codes.shape
        self.H, self.D, self.n = H, D, n
        new = (n + PAGE - 1) // PAGE
        k = torch.randint(0, 256, (n + new, H, PAGE, D), generator=gen(5), device="cuda", dtype=torch.int32).to(torch.uint8)
        k[:n, :, 3] = codes.transpose(0, 1)
        s = torch.full((n + new, H), 7.0, device="cuda")
        s[:n] = scale.t()
        self.cache = B.Cache(k, k.clone(), s, s.clone())
        self.src = B.Pages(1, n, torch.arange(n, dtype=torch.int32, device="cuda")[None], n, 0, i32([[n * PAGE]]), 1, 0)
        self.dst = B.Pages(1, new, torch.arange(n, n + new, dtype=torch.int32, device="cuda")[None], new, 0, i32([[0]]), 1, 0)
        self.src.lens = [[n * PAGE] * H]
        self.mass = torch.zeros(1, H, n * PAGE, device="cuda")
        self.mass[..., 3::PAGE] = 1.0


def by_definition(codes, scale):
    """Codes [H, n, D] and scales [H, n] -> codes of the units' rows, units' scales [H, units]."""
    H, n, D = codes.shape
    units = (n + PAGE - 1) // PAGE
    pad = units * PAGE - n
    y = codes.view(torch.float8_e4m3fn).float() * scale[..., None]
    top = torch.nn.functional.pad(y.abs().nan_to_num(nan=0.0, posinf=math.inf).amax(-1), (0, pad)).view(H, units, PAGE).amax(-1)
    # (by a tensor: a number's reciprocal would be multiplied by)
    z = torch.where(top == 0, torch.ones_like(top), top / torch.full_like(top, 448.0))
    x = y / z.repeat_interleave(PAGE, 1)[:, :n, None]
    out = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    out = torch.where(x.isnan(), torch.full_like(out, 0x7F), out)
    if n % PAGE == 1:  # a last unit of one token: of one old unit, so as it was
        out[:, -1], z[:, -1] = codes[:, -1], scale[:, -1]
    return out, z


def check(codes, scale):
    H, n, D = codes.shape
    pool = OneAPage(codes, scale)
    want, z = by_definition(codes, scale)
    lens, _, ids, flags = evict_call(pool, pool.src, pool.dst, i32([[n]]), pool.mass, 0, 0)
    torch.cuda.synchronize()
    assert not flags[:1].any() and lens.tolist() == [[n]]
    assert torch.equal(ids[0], torch.arange(n, device="cuda", dtype=torch.int32).mul(PAGE).add(3).expand(H, -1))
    for pages, scales in ((pool.cache.k_pages, pool.cache.k_scale), (pool.cache.v_pages, pool.cache.v_scale)):
        assert torch.equal(scales[n:].t().contiguous().view(torch.int32), z.view(torch.int32))
        got = pages[n:].transpose(0, 1).reshape(H, -1, D)[:, :n]
        bad = (got != want).nonzero()
        assert not len(bad), (len(bad), [(i, hex(int(codes[tuple(i)])), float(scale[i[0], i[1]]), float(z[i[0], i[1] // PAGE]),
                                          hex(int(got[tuple(i)])), hex(int(want[tuple(i)]))) for i in bad[:4].tolist()])


def magnitudes(g, n, D):
    """Rows of codes: D of the 127 finite magnitudes of e4m3 each (all of them where D is 128), signs at random."""
    m = torch.rand(n, 127, generator=g, device="cuda").argsort(-1)
    m = torch.cat((m, m[:, :1]), 1)[:, :D]
    return (m + 128 * torch.randint(0, 2, m.shape, generator=g, device="cuda")).to(torch.uint8)


@pytest.mark.parametrize("nan", [False, True])
@pytest.mark.parametrize("D", [128, 64])
def test_all_codes(D, nan):
    """Every code in rows whose scales lie 2^12 apart, so that new codes are subnormal and zero too."""
    g = gen(51)
    codes = torch.stack([magnitudes(g, 6001, D) for _ in range(2)])
    if nan:
        at = torch.rand(codes.shape, generator=g, device="cuda") < 0.002
        codes = torch.where(at, codes | 0x7F, codes)
    check(codes, torch.exp2(-12 * torch.rand(2, 6001, generator=g, device="cuda")))


@pytest.mark.parametrize("power", [True, False])
@pytest.mark.parametrize("D", [128, 64])
def test_borders(D, power):
    """Ratios of an old scale to the new one at which a product of a significand, 8 to 15 (and 1 to 7 of
    subnormal codes), is a border between two codes, normal or subnormal, or a few steps beside one.

    A row of 448s fixes a unit's new scale: exactly its own scale where that is a power of two,
    else within a rounding of it."""
    g = gen(52)
    m = torch.arange(1, 16, dtype=torch.float64)
    odd = torch.arange(1, 32, 2, dtype=torch.float64)
    ratio = (odd[:, None] / m)[..., None] * torch.exp2(torch.arange(-14, 7, dtype=torch.float64))
    ratio = ratio.flatten().unique()
    ratio = ratio[(ratio >= 2.0 ** -15) & (ratio <= 300)]
    rows = ratio.repeat_interleave(7).cuda()                      # each with offsets of -3 .. 3 steps
    steps = torch.arange(-3, 4, device="cuda").repeat(len(ratio))
    rows, steps = (torch.nn.functional.pad(t, (0, -len(t) % 15), value=v) for t, v in ((rows, 1.0), (steps, 0)))
    units = len(rows) // 15
    base = torch.full((units,), 2.0 ** -6, device="cuda")
    if not power:
        base = torch.exp2(torch.rand(units, generator=g, device="cuda") * 8 - 7)
    z = (base * 448) / torch.full_like(base, 448.0)               # the new scale, in fp32
    s = (rows * z.double().repeat_interleave(15)).float()
    s = (s.view(torch.int32) + steps.to(torch.int32)).view(torch.float32)
    codes = magnitudes(g, len(rows), D)
    # what would be larger than the row of 448s is left out (a zero)
    size = codes.view(torch.float8_e4m3fn).double().abs() * s[:, None].double()
    codes = torch.where(size > 447.9 * base.double().repeat_interleave(15)[:, None], codes & 0x80, codes)
    anchor = torch.full((units, 1, D), 0x7E, dtype=torch.uint8, device="cuda")
    codes = torch.cat((anchor, codes.view(units, 15, D)), 1).view(1, -1, D)
    scale = torch.cat((base[:, None], s.view(units, 15)), 1).view(1, -1)
    check(codes, scale)


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("kind", ["small", "large", "signs", "zero", "not finite", "all"])
def test_scales(kind, D):
    """Old scales that are very small, very large, below zero, zero, infinite and NaN."""
    g = gen(53)
    some = {"small": [1e-30, 3e-30, 1e-24, 1.5e-24, 1e-38, 1e-41], "large": [1e31, 2e30, 1e30, 9e29, 5e35], "signs": [-0.01, 0.02, -3.0, 0.5],
            "zero": [0.0, 0.01, -0.0, 0.3], "not finite": [math.inf, math.nan, 0.01, -math.inf, 1.0],
            "all": [1e-30, 1e31, -0.01, 0.0, 0.02, math.inf, math.nan, 1.0, 1e-12, 1e12, 1e-41]}[kind]
    pick = torch.randint(0, len(some), (2, 999), generator=g, device="cuda")
    codes = torch.stack([magnitudes(g, 999, D) for _ in range(2)])
    check(codes, torch.tensor(some, device="cuda")[pick])


@pytest.mark.parametrize("D", [128, 64])
def test_units_of_zeros(D):
    """A unit of zeros of either sign gets the scale 1, whatever its tokens' old scales; and one token that is not zero."""
    g = gen(54)
    codes = (128 * torch.randint(0, 2, (2, 50, D), generator=g, device="cuda")).to(torch.uint8)
    codes[0, 20, 5] = 0x01
    codes[1, 40, 9] = 0xFE
    scale = torch.rand(2, 50, generator=g, device="cuda")
    scale[:, 7], scale[:, 23] = 1e-30, -2.0
    check(codes, scale)
