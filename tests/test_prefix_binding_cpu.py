"""The prefix attention's binding without a GPU: a workspace that it refuses before the library is
called.  No call here launches a kernel."""
import types

import pytest
import torch

from paged_fp8_kv_decode_gb300 import binding as B
from paged_fp8_kv_decode_gb300 import prefix as P


class Pool(torch.Tensor):
    """A host tensor that counts as device memory."""
    is_cuda = True


def test_workspace(monkeypatch):
    """Bytes that do not follow each other: the size of a strided workspace is not that of what follows its address."""
    calls = []
    monkeypatch.setattr(P, "lib", lambda: types.SimpleNamespace(pfkv_prefix_decode_attn=lambda *a: calls.append(a) or 0))
    monkeypatch.setattr(B, "_ptr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(P.R, "_stream", lambda stream, dev: None)
    k, v = (torch.zeros(8, 2, 16, 128, dtype=torch.bfloat16).as_subclass(Pool) for _ in range(2))
    pages = B.Pages(2, 4, torch.zeros(2, 4, dtype=torch.int32), 4, 0, torch.zeros(2, dtype=torch.int32), 1, 0)
    q, of = torch.zeros(2, 1, 8, 128, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    ws = torch.zeros(1 << 13, dtype=torch.uint8)
    args = B.Cache(k, v), pages, pages, of, q, 0.1, 8, 8
    P.pfkv_prefix_decode_attn(*args, ws, q)
    assert len(calls) == 1 and calls[0][12] == 1 << 13
    with pytest.raises(ValueError, match="workspace"):
        P.pfkv_prefix_decode_attn(*args, ws[::2], q)
    assert len(calls) == 1
