"""The calls on shared prefixes and the eviction without a GPU: headers, exports and
bindings agree, and bad arguments are refused on the host before anything touches
CUDA.  No call here launches a kernel."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NO_DEVICE = (5, 6, 2)  # what a call with good arguments returns where there is no sm_103 GPU


@pytest.fixture(scope="module")
def mods():
    from paged_fp8_kv_decode_gb300 import build as pbuild
    pbuild.build()
    from paged_fp8_kv_decode_gb300 import binding, evict, prefix, rope
    evict.lib(), prefix.lib()
    return binding, rope, prefix, evict


def _declared(name):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", name)).read(), flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(pfkv_\w+)\s*\(", src, flags=re.M)))


def test_headers_exports_and_bindings_agree(mods):
    B, R, P, E = mods
    assert _declared("pfkv_prefix.h") == sorted(P.EXPORTED)
    assert _declared("pfkv_evict.h") == sorted(E.EXPORTED)
    out = subprocess.run(["nm", "-D", "--defined-only", B.LIB_PATH], capture_output=True, text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert set(P.EXPORTED) | set(E.EXPORTED) <= exported
    m = re.search(r"#define\s+PFKV_PREFIX_MAX\s+(\d+)", open(os.path.join(ROOT, "include", "pfkv_prefix.h")).read())
    assert P.PFKV_PREFIX_MAX == int(m.group(1))
    import paged_fp8_kv_decode_gb300 as pkg
    assert {"prefix", "evict"} <= set(pkg.__all__) and "``prefix``" in pkg.__doc__ and "``evict``" in pkg.__doc__


@pytest.mark.parametrize("header", ["pfkv_prefix.h", "pfkv_evict.h"])
def test_headers_compile_as_c(header):
    src = f'#include "{header}"\nint main(void) {{ pfkv_pages p; (void)p; return 0; }}\n'
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-I" + os.path.join(ROOT, "include"), "-xc", "-"],
                   input=src, text=True, check=True)


def _take(over, name, **d):
    return {k: over.get(name + "." + k, v) for k, v in d.items()}


def _cache(B, over):
    return B._CCache(**_take(over, "cache", num_pages=8, num_kv_heads=2, page_size=16, head_dim=128, dtype=1, k_pages=0x100000,
                             v_pages=0x200000, k_scale=0x300000, v_scale=0x400000, page_tags=None))


def _pages(B, over, name, at):
    return B._CPages(**_take(over, name, batch=2, max_pages=4, block_tables=at, bt_stride_b=4, bt_stride_h=0,
                             seq_lens=at + 0x1000, len_stride_b=1, len_stride_h=0, expected_tags=None))


WS = 1 << 30


def _prefix(mods, **over):
    B, R, P, _ = mods
    c, own, pre = _cache(B, over), _pages(B, over, "own", 0x10000), _pages(B, over, "pre", 0x20000)
    q, o = (R._CRows(**_take(over, n, data=at, stride_b=2048, stride_t=1024, stride_h=128)) for n, at in (("q", 0x30000), ("o", 0x40000)))
    ref = lambda n, s: None if over.get(n, 0) is None else ctypes.byref(s)  # noqa: E731
    g = lambda n, v: over.get(n, v)  # noqa: E731
    return P.lib().pfkv_prefix_decode_attn(ref("cache", c), ref("own", own), ref("pre", pre), g("batch", 2), g("of", 0x50000),
                                           ref("q", q), g("heads", 8), g("kq", 1), g("scale", 0.1), g("max_len", 64),
                                           g("max_pre", 64), g("ws", 0x60000), g("ws_bytes", WS), ref("o", o), g("mass", None),
                                           g("mass_sb", 128), g("mass_sh", 64), g("flags", 0x70000), None)


PREFIX = [
    ({"cache": None}, 1), ({"pre": None}, 1), ({"q": None}, 1), ({"o": None}, 1), ({"of": None}, 1), ({"batch": -1}, 1),
    ({"batch": 3}, 1), ({"pre.batch": -1}, 1), ({"pre.batch": 4097}, 2), ({"heads": 0}, 1), ({"heads": 7}, 1), ({"heads": 6}, 2),
    ({"heads": 32}, 2), ({"kq": 0}, 1), ({"kq": 2049}, 2), ({"scale": float("nan")}, 1), ({"scale": float("inf")}, 1),
    ({"max_len": -1}, 1), ({"max_pre": -1}, 1), ({"of": 0x50002}, 3), ({"flags": 0x70001}, 3), ({"mass": 0x80002}, 3),
    ({"mass": 0x80000, "kq": 2}, 2), ({"mass": 0x80000, "own": None}, 1), ({"mass": 0x80000, "mass_sb": -1}, 1),
    ({"mass": 0x80000, "mass_sh": -1}, 1), ({"ws": None}, 4), ({"ws_bytes": 0}, 4), ({"ws": 0x60080}, 3),
    ({"q.data": None}, 1), ({"q.data": 0x30008}, 3), ({"q.stride_h": 4}, 3), ({"q.stride_b": -8}, 1), ({"o.data": 0x40004}, 3),
    ({"o.stride_t": 1020}, 3), ({"cache.page_size": 32}, 2), ({"cache.head_dim": 96}, 2), ({"cache.dtype": 3}, 1),
    ({"cache.k_scale": None}, 1), ({"cache.num_pages": 0}, 1), ({"own.max_pages": 0}, 1), ({"own.block_tables": None}, 1),
    ({"pre.block_tables": None}, 1), ({"pre.seq_lens": None}, 1), ({"pre.seq_lens": 0x21002}, 3), ({"own.bt_stride_b": 3}, 1),
    ({"pre.bt_stride_h": -1}, 1), ({"pre.expected_tags": 0x90000}, 1), ({"own.expected_tags": 0x90000}, 1),
    ({"cache.page_tags": 0x90000}, 1), ({"cache.page_tags": 0x90000, "own.expected_tags": 0x91000}, 1),
    ({"batch": 1 << 29, "own": None}, 2), ({"max_pre": (1 << 30) + 1}, 2), ({"max_len": 0x7FFFFFFF}, 2),
]


@pytest.mark.parametrize("over,code", PREFIX, ids=lambda x: str(x))
def test_prefix_refuses(mods, over, code):
    assert _prefix(mods, **over) == code


def test_prefix_takes(mods):
    for over in ({}, {"own": None}, {"pre.batch": 0, "pre.block_tables": None, "pre.seq_lens": None}, {"mass": 0x80000}, {"kq": 5},
                 {"flags": None}, {"cache.dtype": 0, "cache.k_scale": None, "cache.v_scale": None}, {"cache.head_dim": 64},
                 {"own": None, "max_len": -1}, {"cache.page_tags": 0x90000, "own.expected_tags": 0x91000, "pre.expected_tags": 0x92000}):
        assert _prefix(mods, **over) in NO_DEVICE, over
    assert _prefix(mods, **{"batch": 0, "own": None}) == 0
    assert _prefix(mods, **{"batch": 0, "own.batch": 0, "of": None, "q": None, "ws": None}) == 0


def _evict(mods, **over):
    B, _, _, E = mods
    c, src, dst = _cache(B, over), _pages(B, over, "src", 0x10000), _pages(B, over, "dst", 0x20000)
    ref = lambda n, s: None if over.get(n, 0) is None else ctypes.byref(s)  # noqa: E731
    g = lambda n, v: over.get(n, v)  # noqa: E731
    return E.lib().pfkv_kv_evict(ref("cache", c), ref("src", src), ref("dst", dst), g("keep", 0x50000), g("first", 1), g("last", 1),
                                 g("mass", 0x60000), g("mass_sb", 128), g("mass_sh", 64), g("max_len", 64), g("max_keep", 32),
                                 g("ws", 0x70000), g("ws_bytes", WS), g("new_lens", 0x80000), g("nm", 0x90000), g("nm_sb", 80),
                                 g("nm_sh", 40), g("nm_len", 40), g("kept", 0xA0000), g("kept_sb", 64), g("kept_sh", 32),
                                 g("flags", 0xB0000), None)


EVICT = [
    ({"cache": None}, 1), ({"src": None}, 1), ({"dst": None}, 1), ({"dst.batch": 3}, 1), ({"keep": None}, 1), ({"mass": None}, 1),
    ({"new_lens": None}, 1), ({"first": -1}, 1), ({"last": -1}, 1), ({"mass_sb": -1}, 1), ({"mass_sh": -1}, 1), ({"max_len": -1}, 1),
    ({"max_keep": -1}, 1), ({"nm_sb": -1}, 1), ({"nm_sh": -1}, 1), ({"nm_len": 31}, 1), ({"kept_sb": -1}, 1), ({"kept_sh": -1}, 1),
    ({"nm_sh": 39}, 1), ({"nm_sb": 79}, 1), ({"nm_sb": 40}, 1), ({"kept_sh": 31}, 1), ({"kept_sb": 32}, 1), ({"kept_sb": 63}, 1),
    ({"src.len_stride_b": 0}, 1), ({"keep": 0x50001}, 3), ({"mass": 0x60002}, 3), ({"new_lens": 0x80002}, 3), ({"nm": 0x90001}, 3),
    ({"kept": 0xA0002}, 3), ({"flags": 0xB0002}, 3), ({"ws": None}, 4), ({"ws_bytes": 100}, 4), ({"ws": 0x70010}, 3),
    ({"cache.page_size": 8}, 2), ({"cache.head_dim": 32}, 2), ({"cache.k_pages": None}, 1), ({"src.max_pages": 0}, 1),
    ({"src.block_tables": None}, 1), ({"dst.block_tables": None}, 1), ({"dst.block_tables": 0x20002}, 3), ({"dst.bt_stride_b": 3}, 1),
    ({"src.seq_lens": None}, 1), ({"dst.expected_tags": 0xC0000}, 1), ({"cache.page_tags": 0xC0000}, 1),
    ({"cache.page_tags": 0xC0000, "src.expected_tags": 0xD0000}, 1), ({"nm_len": 0x7FFFFFFF, "nm_sh": 1 << 32, "nm_sb": 1 << 34, "src.batch": 16, "dst.batch": 16}, 2),
    ({"nm_len": 0x7FFFFFFF, "nm_sh": 1 << 32, "nm_sb": 1 << 34}, 2), ({"max_len": 0x7FFFFFF0}, 2),
    ({"max_keep": 0x7FFFFFFF, "nm": None, "ws_bytes": 1 << 40, "kept": None}, 2),
]


@pytest.mark.parametrize("over,code", EVICT, ids=lambda x: str(x))
def test_evict_refuses(mods, over, code):
    assert _evict(mods, **over) == code


def test_evict_takes(mods):
    for over in ({}, {"nm": None, "nm_len": 0}, {"kept": None}, {"flags": None}, {"dst.seq_lens": None}, {"max_keep": 0, "nm_len": 0},
                 {"nm_sb": 40, "nm_sh": 80}, {"kept_sb": 32, "kept_sh": 64}, {"cache.head_dim": 64},
                 {"new_lens": 0x11000}, {"cache.page_tags": 0xC0000, "src.expected_tags": 0xD0000, "dst.expected_tags": 0xE0000}):
        assert _evict(mods, **over) in NO_DEVICE, over
    assert _evict(mods, **{"src.batch": 0, "dst.batch": 0, "keep": None, "mass": None, "ws": None}) == 0


def test_workspace_sizes(mods):
    B, _, P, E = mods
    c, src, pre = _cache(B, {}), _pages(B, {}, "src", 0x10000), _pages(B, {}, "pre", 0x20000)
    n = ctypes.c_size_t(0)
    ref = ctypes.byref
    assert E.lib().pfkv_kv_evict_workspace_size(ref(c), ref(src), 64, 32, ref(n)) == 0 and n.value > 0
    assert E.lib().pfkv_kv_evict_workspace_size(ref(c), ref(src), 64, 32, None) == 1
    assert E.lib().pfkv_kv_evict_workspace_size(ref(c), ref(src), -1, 32, ref(n)) == 1
    size = P.lib().pfkv_prefix_decode_workspace_size
    assert size(ref(c), ref(src), ref(pre), 2, 8, 1, 64, 64, 0, None) == 1
    assert size(ref(c), ref(src), ref(pre), 2, 8, 0, 64, 64, 0, ref(n)) == 1
    assert size(ref(c), ref(src), ref(pre), 2, 8, 2, 64, 64, 1, ref(n)) == 2
    assert size(ref(c), None, ref(pre), 2, 8, 1, 64, 64, 1, ref(n)) == 1


def _tensors(mods):
    B = mods[0]
    pool = [torch.zeros(8, 2, 16, 128, dtype=torch.bfloat16) for _ in range(2)]
    bt, n = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    return B.Cache(*pool), B.Pages(2, 4, bt, 4, 0, n, 1, 0), torch.zeros(1 << 12, dtype=torch.uint8)


def test_prefix_binding_refuses(mods):
    B, _, P, _ = mods
    cache, pages, ws = _tensors(mods)
    q, of = torch.zeros(2, 1, 8, 128, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="device memory"):
        P.pfkv_prefix_decode_attn(cache, pages, pages, of, q, 0.1, 8, 8, ws, q)
    with pytest.raises(ValueError, match="q and out"):
        P.pfkv_prefix_decode_attn(cache, pages, pages, of, q[0], 0.1, 8, 8, ws, q[0])
    with pytest.raises(ValueError, match="q and out"):
        P.pfkv_prefix_decode_attn(cache, pages, pages, of, q, 0.1, 8, 8, ws, q[:, :, :4])
    with pytest.raises(ValueError, match="int32"):
        P.pages_struct(B.Pages(2, 4, pages.block_tables.long(), 4, 0, pages.seq_lens, 1, 0), -1)


def test_evict_binding_refuses(mods):
    B, _, _, E = mods
    cache, pages, ws = _tensors(mods)
    keep, mass = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 2, 64)
    call = lambda **o: E.pfkv_kv_evict(**{**dict(cache=cache, pages=pages, new_pages=pages, keep_lens=keep, attn_mass=mass,  # noqa: E731
                                                 max_seq_len=64, max_keep_len=32, workspace=ws, new_lens=keep), **o})
    for over, what in (({"attn_mass": mass.double()}, "attn_mass"), ({"attn_mass": mass[:, :, :63]}, "attn_mass"),
                       ({"attn_mass": mass.transpose(1, 2)}, "attn_mass"), ({"new_mass": mass[:1]}, "new_mass"),
                       ({"new_mass": mass[:, :, :31]}, "new_mass"), ({"kept": mass}, "kept"),
                       ({"kept": torch.zeros(2, 2, 31, dtype=torch.int32)}, "kept")):
        with pytest.raises(ValueError, match=what):
            call(**over)
    with pytest.raises(ValueError, match="device tensor"):  # host memory that the GPU does not map
        call()
