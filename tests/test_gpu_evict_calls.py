"""Calls of the eviction and of the attention over prefixes that programs make and the definitions
allow: captured and replayed, behind bounds far above the lengths, with nothing to attend to, with
flags in host memory."""
import math

import pytest
import torch

from prefix_cases import B, E, PAGE, Pool, attend, call, close, i32, kept_ids, no_prefixes, pages_of, rows
from test_gpu_evict import check as check_evict
from test_gpu_evict import totals
from test_gpu_prefix import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("most", [700, 40000])
def test_replayed(most, fp8):
    """A captured eviction, by one CTA a head and by clusters, whose inputs change between replays."""
    pool = Pool(2 * pages_of(most) + 2 * pages_of(2000) + 9, 1, 64, fp8, seed=91)
    src, dst = pool.tables([most, most // 3]), pool.tables([600, 200], fill=False)
    keep, mass = i32([[600], [200]]), totals(pool, 2, most, "plain")
    ws = torch.empty(E.pfkv_kv_evict_workspace_size(pool.cache, src, most, 600), dtype=torch.uint8, device="cuda")
    new_lens, flags = torch.zeros_like(keep), torch.zeros(4, dtype=torch.uint8, device="cuda")
    new_mass, kept = torch.zeros(2, 1, 700, device="cuda"), torch.zeros(2, 1, 600, dtype=torch.int32, device="cuda")

    def run():
        E.pfkv_kv_evict(pool.cache, src, dst, keep, mass, most, 600, ws, new_lens, new_mass=new_mass, kept=kept, keep_first=3,
                        keep_last=5, flags=flags)
    run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for k, (lens, many) in enumerate((([most, most // 3], [600, 200]), ([most // 2, 17], [101, 17]), ([30, most // 3], [0, 199]))):
        src.seq_lens.copy_(i32(lens)[:, None])
        keep.copy_(i32(many)[:, None])
        mass.copy_(totals(pool, 2, most, ("plain", "few", "close")[k]))
        new_mass.fill_(math.nan)
        g.replay()
        torch.cuda.synchronize()
        assert not flags[:2].any() and new_lens.tolist() == [[m] for m in many]
        for b, (n, m) in enumerate(zip(lens, many)):
            want = kept_ids(mass[b, 0, :n], n, m, 3, 5)
            assert kept[b, 0, :m].tolist() == want
            assert torch.equal(new_mass[b, 0, :m], mass[b, 0, torch.tensor(want, dtype=torch.long, device="cuda")])
            assert not new_mass[b, 0, m:].any()
            if not fp8:
                at = torch.tensor(want, dtype=torch.long)
                assert torch.equal(pool.values(dst, b, 0, m, "k"), pool.values(src, b, 0, n, "k")[at])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("max_len,max_keep", [(100, 50), (9000, 4000), (300000, 200000)])
def test_loose_bounds(max_len, max_keep, fp8):
    """Bounds that choose clusters and long grids, over short lengths."""
    pool = Pool(200, 3, 128, fp8, seed=92)
    lens, keep = [100, 37, 1, 0], [50, 20, 1, 5]
    src, dst = pool.tables(lens, wide=max_len // PAGE), pool.tables([min(a, b) for a, b in zip(lens, keep)], fill=False, wide=max_keep // PAGE)
    mass = torch.zeros(4, 3, max_len, device="cuda")
    mass[..., :100] = totals(pool, 4, 100, "few")
    check_evict(pool, src, dst, i32(keep)[:, None], mass, 2, 4, max_len=max_len, max_keep=max_keep)


@pytest.mark.parametrize("fp8", [False, True])
def test_loose_bounds_of_prefixes(fp8):
    pool = Pool(200, 2, 128, fp8, seed=93)
    pre, own = pool.tables([300, 0, 17], wide=3000), pool.tables([40, 0, 7, 129], wide=2000)
    q = rows(pool.g, 4, 1, 8, 128, outliers=0)
    mass = torch.rand(4, 2, 32000, generator=pool.g, device="cuda")
    check(pool, own, pre, [0, 1, -1, 2], q, 0.1, mass=mass, max_len=32000, max_pre=48000)
    tight, _ = call(pool, own, pre, [0, 1, -1, 2], q, 0.1)
    loose, _ = call(pool, own, pre, [0, 1, -1, 2], q, 0.1, max_len=129, max_pre=1 << 30)
    assert torch.equal(tight, loose)


@pytest.mark.parametrize("fp8", [False, True])
def test_nothing_to_attend_to(fp8):
    """Lengths and bounds of zero, for own tokens, prefixes and both."""
    pool = Pool(60, 2, 64, fp8, seed=94)
    pre, none, own = pool.tables([100]), pool.tables([0]), pool.tables([0, 0, 0])
    q = rows(pool.g, 3, 2, 4, 64, outliers=0)
    check(pool, own, pre, [0, -1, 0], q, 0.1, max_len=0)
    for tables in (own, None):
        for p, of in ((none, [0, 0, -1]), (no_prefixes(2), [-1, -1, -1])):
            out, flags = call(pool, tables, p, of, q, 0.1, max_len=0, max_pre=0)
            assert not out.any() and not flags[:3].any()


@pytest.mark.parametrize("fp8", [False, True])
def test_totals_without_prefixes(fp8):
    """The same output and totals as the call that knows no prefixes, within both calls' roundings."""
    pool = Pool(100, 2, 128, fp8, seed=95)
    own = pool.tables([300, 1, 90])
    q = rows(pool.g, 3, 1, 8, 128, outliers=0)
    mass, other = torch.zeros(2, 3, 2, 300, device="cuda")
    check(pool, own, no_prefixes(2), [-1, -1, -1], q, 0.1, mass=mass)
    ws = torch.empty(B.pfkv_decode_mass_workspace_size(pool.cache, own, 8, 0, 300), dtype=torch.uint8, device="cuda")
    out, flags = torch.empty_like(q[:, 0]), torch.zeros(4, dtype=torch.uint8, device="cuda")
    B.pfkv_paged_decode_attn_mass(pool.cache, own, q[:, 0].contiguous(), 0.1, 0, 300, ws, out, flags, other)
    # two sums of weights, each within 2^-18 of the exact ones (exponentials and logarithms of 40 at most)
    close(mass, other.double(), other.double() * 2.0 ** -14 + 1e-9, "totals")


@pytest.mark.parametrize("fp8", [False, True])
def test_flags_in_host_memory(fp8):
    pool = Pool(200, 2, 128, fp8, seed=96)
    pre, own, of = pool.tables([200, 100]), pool.tables([30, 40, 50, 60, 7]), [0, 1, -1, 9, 0]
    q = rows(pool.g, 5, 1, 8, 128, outliers=0)
    want, tol, _, _ = attend(pool, own, pre, [0, 1, -1, -1, 0], q, 0.1)
    pre.block_tables[1, 0, 2] = -1
    own.seq_lens[4] = -3
    flags = torch.full((8,), 0xAA, dtype=torch.uint8).pin_memory()
    out, _ = call(pool, own, pre, of, q, 0.1, flags=flags, max_len=60, max_pre=200)
    torch.cuda.synchronize()
    assert flags[:5].tolist() == [0, 2, 0, 2, 4] and not out[[1, 3, 4]].any()
    close(out[[0, 2]], want[[0, 2]], tol[[0, 2]], "the sound ones")
    src, dst = pool.tables([60, 33]), pool.tables([30, 16], fill=False)
    src.block_tables[1, 0, 1] = pool.cache.k_pages.shape[0]
    ws = torch.empty(E.pfkv_kv_evict_workspace_size(pool.cache, src, 60, 30), dtype=torch.uint8, device="cuda")
    lens = torch.full((2, 1), -5, dtype=torch.int32).pin_memory()
    flags = torch.full((4,), 0xAA, dtype=torch.uint8).pin_memory()
    E.pfkv_kv_evict(pool.cache, src, dst, i32([[30], [16]]), totals(pool, 2, 60, "plain"), 60, 30, ws, lens, flags=flags)
    torch.cuda.synchronize()
    assert flags[:2].tolist() == [0, 2] and lens.tolist() == [[30], [0]]
