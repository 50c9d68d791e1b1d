"""Refusals of pfkv_latent_prefill_attn that depend on the number of rows."""
from test_rope_latent_abi_cpu import NO_DEVICE, _prefill, mods  # noqa: F401


def test_rows_that_share_an_address(mods):  # noqa: F811
    for n in ("qn", "qr", "kn", "kr", "v", "out"):
        assert _prefill(mods, **{n + ".stride_t": 0}) == 2, n
    assert _prefill(mods, tq=1, **{"qn.stride_t": 0, "qr.stride_t": 0, "out.stride_t": 0}) in NO_DEVICE
    assert _prefill(mods, tk=1, **{"kn.stride_t": 0, "kr.stride_t": 0, "v.stride_t": 0}) in NO_DEVICE


def test_arrays_without_rows_are_not_read(mods):  # noqa: F811
    none = {n + ".data": None for n in ("qn", "qr", "out")}
    assert _prefill(mods, tq=0, **none) in NO_DEVICE
    assert _prefill(mods, tq=1, **none) == 1
    none = {n + ".data": None for n in ("kn", "kr", "v")}
    assert _prefill(mods, tk=0, **none) in NO_DEVICE
    assert _prefill(mods, tk=1, **none) == 1


def test_a_bound_of_no_queries(mods):  # noqa: F811
    assert _prefill(mods, max_q=0) in NO_DEVICE
