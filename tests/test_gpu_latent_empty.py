"""A step in which no request has new tokens, or none has cached ones: packed arrays of no
rows, which have no address."""
import pytest
import torch

from latent_cases import flags_for, gen, i32, latent_pool, pages, rows, tables
from paged_fp8_kv_decode_gb300 import binding as B
from paged_fp8_kv_decode_gb300 import latent as L
from paged_fp8_kv_decode_gb300 import rope as R

pytestmark = pytest.mark.gpu


def none(*shape):
    return torch.empty(0, *shape, dtype=torch.bfloat16, device="cuda")


@pytest.mark.parametrize("fp8", [False, True])
def test_no_rows(fp8):
    g = gen(98)
    bt, num = tables([3, 2], seed=1)
    rope = R.Rope(torch.ones(32, device="cuda"))
    starts, at = i32([0, 0, 0]), i32([5, 17])
    fl = flags_for(2)
    lat = latent_pool(g, num, fp8)
    k = rows(g, num, 2, 16, 64).view(torch.uint8)[..., :64].contiguous() if fp8 else rows(g, num, 2, 16, 64)
    s = torch.ones(num, 2, device="cuda") if fp8 else None
    kv = B.Cache(k, k.clone(), s, None if s is None else s.clone())
    old = [t.clone() for t in (lat.c_pages, lat.r_pages, kv.k_pages, kv.v_pages)]
    q, qk = none(4, 64), none(2, 64)
    L.pfkv_latent_append(lat, pages(bt, at), rope, at, none(512), none(64), q, q, row_starts=starts, max_new_tokens=9, flags=fl)
    R.pfkv_rope_append(kv, pages(bt, at), rope, at, qk, qk, q, q, row_starts=starts, max_new_tokens=9, flags=fl)
    L.pfkv_latent_gather(lat, pages(bt, i32([0, 0])), starts, 40, none(512), none(64), flags=fl)
    assert not fl.any()
    for t, was in zip((lat.c_pages, lat.r_pages, kv.k_pages, kv.v_pages), old):
        assert torch.equal(t, was)
    # a request that claims rows all the same is flagged
    L.pfkv_latent_append(lat, pages(bt, at), rope, at, none(512), none(64), row_starts=i32([0, 3, 3]), max_new_tokens=9, flags=fl)
    assert fl.tolist()[:2] == [4, 4]                 # rows 0 to 3, and none at 3, of none
    fl.zero_()
    L.pfkv_latent_gather(lat, pages(bt, i32([0, 2])), i32([0, 0, 2]), 40, none(512), none(64), flags=fl)
    assert fl.tolist()[:2] == [0, 4]
