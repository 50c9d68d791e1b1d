"""The eviction's binding without a GPU: what it refuses before the library is called, and what it
hands over.  No call here launches a kernel."""
import types

import pytest
import torch

from paged_fp8_kv_decode_gb300 import binding as B
from paged_fp8_kv_decode_gb300 import evict as E
from paged_fp8_kv_decode_gb300 import prefix as P


def _i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def _args(**over):
    pool = [torch.zeros(8, 2, 16, 128, dtype=torch.bfloat16) for _ in range(2)]
    pages = B.Pages(3, 4, _i32(3, 2, 4), 8, 4, _i32(3, 2), 2, 1)
    new = B.Pages(3, 4, _i32(3, 2, 4), 8, 4, None, 0, 0)
    return {**dict(cache=B.Cache(*pool), pages=pages, new_pages=new, keep_lens=_i32(3, 2), attn_mass=torch.zeros(3, 2, 64),
                   max_seq_len=64, max_keep_len=32, workspace=torch.zeros(1 << 12, dtype=torch.uint8), new_lens=_i32(3, 2)), **over}


@pytest.fixture
def seen(monkeypatch):
    """What reaches the library, whose call is replaced; host tensors count as ones that the GPU maps."""
    calls = []
    fake = types.SimpleNamespace(pfkv_kv_evict=lambda *a: calls.append(a) or 0)
    monkeypatch.setattr(E, "lib", lambda: fake)
    monkeypatch.setattr(B, "_ptr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(E.R, "_stream", lambda stream, dev: None)
    return calls


def test_lengths_of_the_new_pages_may_be_none(seen):
    E.pfkv_kv_evict(**_args())
    assert len(seen) == 1 and seen[0][2]._obj.seq_lens is None and seen[0][1]._obj.seq_lens
    with pytest.raises(ValueError, match="int32"):
        P.pages_struct(B.Pages(2, 4, _i32(2, 4), 4, 0, torch.zeros(2), 1, 0), -1)


@pytest.mark.parametrize("name", ["keep_lens", "new_lens"])
def test_lengths_lie_as_those_of_the_pages(seen, name):
    E.pfkv_kv_evict(**_args(**{name: _i32(6)}))             # as many, in another shape
    E.pfkv_kv_evict(**_args(**{name: _i32(3, 5)[:, :2]}))   # a view that spans more
    for t in (_i32(5), _i32(3), _i32(2, 2), _i32(0), _i32(3, 1), _i32(1, 1).expand(3, 2)):
        with pytest.raises(ValueError, match=name):
            E.pfkv_kv_evict(**_args(**{name: t}))
    with pytest.raises(ValueError, match=name):
        E.pfkv_kv_evict(**_args(**{name: torch.zeros(3, 2, dtype=torch.int64)}))
    # one length a request for all heads
    shared = B.Pages(3, 4, _i32(3, 4), 4, 0, _i32(3), 1, 0)
    E.pfkv_kv_evict(**_args(pages=shared, keep_lens=_i32(3), new_lens=_i32(3)))
    with pytest.raises(ValueError, match=name):
        E.pfkv_kv_evict(**_args(**{"pages": shared, "keep_lens": _i32(3), "new_lens": _i32(3), name: _i32(2)}))
    assert len(seen) == 3


def test_workspace(seen):
    for t in (torch.zeros(1 << 10), torch.zeros(1 << 13, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            E.pfkv_kv_evict(**_args(workspace=t))
    assert not seen
    E.pfkv_kv_evict(**_args())
    assert seen[0][12] == 1 << 12
