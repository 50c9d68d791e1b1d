"""Pools whose tensors are not what the kernels would take them for are refused."""
import pytest
import torch

from test_rope_latent_devices_cpu import Called, Zero, calls, f, i, stand_ins, u, z  # noqa: F401


def h(*shape):
    return torch.zeros(*shape, dtype=torch.float16).as_subclass(Zero)


def call(name, **over):
    fn, args, more = calls()[name]
    for k, t in over.items():
        setattr(args[0], k, t)
    fn(*args, **more, **({} if name == "size" else {"stream": 0}))


LATENT = [
    dict(c_pages=h(9, 16, 512)), dict(c_pages=z(9, 16, 512)), dict(c_pages=i(9, 16, 512)),
    dict(c_pages=u(9, 16, 1024)[..., ::2]), dict(c_pages=u(8, 16, 512)), dict(r_pages=h(9, 16, 64)),
    dict(c_scale=None), dict(c_scale=z(8)), dict(c_scale=z(9).double()), dict(c_scale=f(9)), dict(c_scale=z(18)[::2]),
    dict(page_tags=i(8)), dict(page_tags=i(9).long()), dict(page_tags=i(18)[::2]),
]


@pytest.mark.parametrize("name", ["append", "gather", "size", "decode"])
@pytest.mark.parametrize("over", LATENT, ids=range(len(LATENT)))
def test_latent_pools(name, over):
    with pytest.raises(Called):
        call(name)
    with pytest.raises(ValueError):
        call(name, **over)


@pytest.mark.parametrize("over", [
    dict(k_pages=h(9, 2, 16, 64), v_pages=h(9, 2, 16, 64)), dict(v_pages=f(9, 2, 16, 64)), dict(v_pages=u(8, 2, 16, 64)),
    dict(k_pages=u(9, 2, 16, 128)[..., ::2]), dict(v_pages=u(9, 2, 16, 128)[..., ::2]), dict(k_scale=None),
    dict(k_scale=z(9)), dict(v_scale=z(17)), dict(v_scale=f(9, 2)), dict(page_tags=i(9)), dict(page_tags=i(9, 2).long()),
])
def test_key_and_value_pools(over):
    with pytest.raises(Called):
        call("rope_append")
    with pytest.raises(ValueError):
        call("rope_append", **over)


def test_pools_that_are_taken():
    codes = torch.zeros(9, 16, 512, dtype=torch.uint8).view(torch.float8_e4m3fn).as_subclass(Zero)
    for over in (dict(c_pages=codes), dict(c_pages=f(9, 16, 512), c_scale=None), dict(c_scale=z(12)), dict(page_tags=None)):
        for name in ("append", "gather", "size", "decode"):
            with pytest.raises(Called):
                call(name, **over)


def test_a_pool_in_host_memory_is_not_decoded():
    """Host tensors stand in for pinned ones."""
    with pytest.raises(Called):
        call("append", c_pages=torch.zeros(9, 16, 512, dtype=torch.uint8))
    for k, t in (("c_pages", torch.zeros(9, 16, 512, dtype=torch.uint8)), ("r_pages", torch.zeros(9, 16, 64, dtype=torch.bfloat16))):
        with pytest.raises(ValueError, match="device memory"):
            call("decode", **{k: t})
