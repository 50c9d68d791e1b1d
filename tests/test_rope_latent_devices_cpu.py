"""Tensors of another device than the current one are refused, whichever argument they
are.  Host tensors stand in for device ones; the library is never called."""
import dataclasses

import pytest
import torch

from paged_fp8_kv_decode_gb300 import binding as B
from paged_fp8_kv_decode_gb300 import latent as L
from paged_fp8_kv_decode_gb300 import rope as R


class Zero(torch.Tensor):
    is_cuda = True

    def get_device(self):
        return 0


class One(Zero):
    def get_device(self):
        return 1


class Called(Exception):
    pass


class Library:
    def __getattr__(self, name):
        def call(*args):
            raise Called
        return call


@pytest.fixture(autouse=True)
def stand_ins(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(B, "_ptr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(L, "lib", Library)
    monkeypatch.setattr(R, "lib", Library)


def f(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16).as_subclass(Zero)


def i(*shape):
    return torch.zeros(*shape, dtype=torch.int32).as_subclass(Zero)


def z(*shape):
    return torch.zeros(*shape).as_subclass(Zero)


def u(*shape):
    return torch.zeros(*shape, dtype=torch.uint8).as_subclass(Zero)


def calls():
    pages = lambda: B.Pages(2, 4, i(2, 4), 4, 0, i(2), 1, 0, i(2, 4))  # noqa: E731
    kv = lambda: B.Cache(u(9, 2, 16, 64), u(9, 2, 16, 64), z(9, 2), z(9, 2), i(9, 2))  # noqa: E731
    lat = lambda: L.LatentCache(u(9, 16, 512), u(9, 16, 128).view(torch.bfloat16), z(9), i(9))  # noqa: E731
    rope = lambda: R.Rope(z(32))  # noqa: E731
    more = dict(q=f(5, 4, 64), q_out=f(5, 4, 64), new_lens=i(2), rope_positions=i(2), row_starts=i(3), max_new_tokens=3,
                flags=u(4))
    return {
        "rope_append": (R.pfkv_rope_append, [kv(), pages(), rope(), i(2), f(5, 2, 64), f(5, 2, 64)], dict(more)),
        "append": (L.pfkv_latent_append, [lat(), pages(), rope(), i(2), f(5, 512), f(5, 64)], dict(more)),
        "gather": (L.pfkv_latent_gather, [lat(), pages(), i(3), 9, f(5, 512), f(5, 64)], dict(flags=u(4))),
        "size": (L.pfkv_latent_decode_workspace_size, [lat(), pages(), 4, 1, 9], {}),
        "decode": (L.pfkv_latent_decode_attn, [lat(), pages(), f(2, 1, 4, 512), f(2, 1, 4, 64), 0.1, 9, u(256),
                                               f(2, 1, 4, 512)], dict(flags=u(4))),
        "prefill": (L.pfkv_latent_prefill_attn, [f(5, 2, 128), f(5, 2, 64), f(6, 2, 128), f(6, 64), f(6, 2, 128), i(3), i(3),
                                                 4, 0.1, True, f(5, 2, 128)], dict(flags=u(4))),
    }


def places(args):
    """Every tensor among the arguments, with a function that puts another in its place."""
    for k in (range(len(args)) if isinstance(args, list) else list(args)):
        v = args[k]
        if isinstance(v, torch.Tensor):
            yield str(k), v, lambda t, k=k: args.__setitem__(k, t)
        elif dataclasses.is_dataclass(v):
            for name, t in vars(v).items():
                if isinstance(t, torch.Tensor):
                    yield f"{k}.{name}", t, lambda t, v=v, name=name: setattr(v, name, t)


@pytest.mark.parametrize("name", sorted(calls()))
def test_every_argument(name):
    fn, args, more = calls()[name]
    with pytest.raises(Called):
        fn(*args, **more, **({} if name == "size" else {"stream": 0}))
    tried = 0
    for where, t, put in list(places(args)) + list(places(more)):
        put(t.as_subclass(One))
        with pytest.raises(ValueError, match="device"):
            fn(*args, **more, **({} if name == "size" else {"stream": 0}))
        put(t)
        tried += 1
    assert tried >= (7 if name == "size" else 9), (name, tried)


def test_host_memory_is_of_every_device():
    fn, args, more = calls()["decode"]
    args[1].seq_lens = torch.zeros(2, dtype=torch.int32)   # pinned host memory is addressed as it is
    with pytest.raises(Called):
        fn(*args, **more, stream=0)
