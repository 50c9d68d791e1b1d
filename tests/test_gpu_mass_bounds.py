"""Totals of tokens behind a bound, or a length, of more than 65,535 blocks of 256 tokens: the
bound sizes a launch, in the call with prefixes and in the one without."""
import pytest
import torch

from prefix_cases import B, PAGE, Pool, attend, call, close, i32, rows

pytestmark = pytest.mark.gpu

FAR = 65535 * 256  # tokens that one launch of a block a 256 tokens reaches


@pytest.mark.parametrize("fp8", [False, True])
def test_loose_bound(fp8):
    pool = Pool(60, 1, 64, fp8, seed=61)
    pre, own, of = pool.tables([100]), pool.tables([40, 300]), [0, -1]
    q = rows(pool.g, 2, 1, 2, 64, outliers=0)
    mass = torch.zeros(2, 1, FAR + 700, device="cuda")
    want, tol, m, m_tol = attend(pool, own, pre, of, q, 0.125, torch.zeros(2, 1, 300, device="cuda"))
    out, flags = call(pool, own, pre, of, q, 0.125, mass=mass, max_len=FAR + 700)
    torch.cuda.synchronize()
    assert not flags[:2].any()
    close(out, want, tol, "out")
    close(mass[..., :300], m, m_tol, "mass")
    assert not mass[..., 300:].any()


@pytest.mark.parametrize("prefix", [False, True])
def test_long_sequence(prefix):
    """One request of more tokens than that, whose table names the same 64 pages again and again."""
    n, pages = FAR + 1000, 64
    need = (n + PAGE - 1) // PAGE
    pool = Pool(80, 1, 64, True, seed=62)
    pre, few = pool.tables([130]), pool.tables([pages * PAGE])
    bt = few.block_tables[0, 0].repeat(need // pages + 1)[:need][None].contiguous()
    own = B.Pages(1, need, bt, need, 0, i32([[n]]), 1, 0)
    own.lens = [[n]]
    q = rows(pool.g, 1, 1, 2, 64, outliers=0)
    mass = torch.zeros(1, 1, n, device="cuda")
    if prefix:
        _, flags = call(pool, own, pre, [0], q, 0.125, mass=mass)
    else:
        flags, out = torch.full((4,), 0xAA, dtype=torch.uint8, device="cuda"), torch.empty_like(q[:, 0])
        ws = torch.empty(B.pfkv_decode_mass_workspace_size(pool.cache, own, 2, 0, n), dtype=torch.uint8, device="cuda")
        B.pfkv_paged_decode_attn_mass(pool.cache, own, q[:, 0].contiguous(), 0.125, 0, n, ws, out, flags, mass)
    torch.cuda.synchronize()
    assert not flags[:1].any()
    # the weights of the 64 pages' tokens, by how often each is seen
    k = pool.values(few, 0, 0, pages * PAGE, "k")
    s = q[0, 0].double() @ k.T * 0.125
    times = torch.full((pages * PAGE,), n // (pages * PAGE), dtype=torch.float64, device="cuda")
    times[:n % (pages * PAGE)] += 1
    total = (times * s.exp()).sum(-1)
    if prefix:
        total = total + (q[0, 0].double() @ pool.values(pre, 0, 0, 130, "k").T * 0.125).exp().sum(-1)
    want = (s.exp() / total[:, None]).sum(0)
    # as in `attend`: scores (a query's f16 or e4m3 values: 2^-17 of its largest), exponential and logarithm; and the
    # fp32 sums: 9,200 tokens a worker, an eighth of them a lane, one after the other
    qq = q[0, 0].double()
    err = (qq.abs() @ k.abs().T).amax(-1) * 0.125 * 40 * 2.0 ** -24 + 2.0 ** -17 * qq.abs().amax(-1) * k.abs().sum(-1).amax() * 0.125
    tol = want * (2 * err.max() + 40 * 2.0 ** -20 + 1200 * 2.0 ** -24)
    got = mass[0, 0].double()
    at = torch.arange(n, device="cuda") % (pages * PAGE)
    close(got, want[at], tol[at], "weights")
