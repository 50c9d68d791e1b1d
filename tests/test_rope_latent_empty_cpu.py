"""Arrays of no rows: they have no address, and the calls take them."""
import pytest

from test_rope_latent_abi_cpu import NO_DEVICE, _append_case, _gather, mods  # noqa: F401

NONE = {n + ".data": None for n in ("k", "v", "q", "o")}


@pytest.mark.parametrize("latent", [False, True])
def test_appends_of_no_rows(mods, latent):  # noqa: F811
    packed = {"tok.row_starts": 0x3000, "tok.total_rows": 0}
    assert _append_case(mods, latent, **packed, **NONE) in NO_DEVICE
    assert _append_case(mods, latent, q=None, o=None, **packed, **NONE) in NO_DEVICE
    assert _append_case(mods, latent, k=None, **packed) == 1
    assert _append_case(mods, latent, heads=0, **packed, **NONE) == 1
    assert _append_case(mods, latent, **{**packed, "tok.total_rows": 1}, **NONE) == 1
    assert _append_case(mods, latent, **NONE) == 1   # padded rows are never none


def test_gather_of_no_rows(mods):  # noqa: F811
    assert _gather(mods, total=0, c=None, r=None) in NO_DEVICE
    assert _gather(mods, total=0, c=None, r=None, starts=None) == 1
    assert _gather(mods, total=1, c=None) == 1 and _gather(mods, total=1, r=None) == 1
