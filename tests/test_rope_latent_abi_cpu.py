"""The rotary append and the latent cache's calls without a GPU: their headers,
exports and bindings agree, and bad arguments are refused on the host before
anything touches CUDA.  No call here launches a kernel."""
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
    from paged_fp8_kv_decode_gb300 import binding, latent, rope
    latent.lib()
    return binding, rope, latent


def _header(name):
    src = open(os.path.join(ROOT, "include", name)).read()
    return re.sub(r"/\*.*?\*/", "", src, flags=re.S)


def _declared(name):
    return sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(pfkv_\w+)\s*\(", _header(name), flags=re.M)))


def test_headers_exports_and_bindings_agree(mods):
    B, R, L = mods
    assert _declared("pfkv_rope.h") == sorted(R.EXPORTED)
    assert _declared("pfkv_latent.h") == sorted(L.EXPORTED)
    out = subprocess.run(["nm", "-D", "--defined-only", B.LIB_PATH], capture_output=True, text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert set(R.EXPORTED) | set(L.EXPORTED) <= exported
    for name in ("PFKV_LATENT_DIM", "PFKV_LATENT_ROPE", "PFKV_LATENT_NOPE", "PFKV_LATENT_VDIM"):
        m = re.search(r"#define\s+" + name + r"\s+(\d+)", _header("pfkv_latent.h"))
        assert getattr(L, name) == int(m.group(1))


def test_headers_compile_as_c():
    src = '#include "pfkv_latent.h"\nint main(void) { pfkv_latent_cache c; (void)c; return 0; }\n'
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-I" + os.path.join(ROOT, "include"), "-xc", "-"],
                   input=src, text=True, check=True)


def _pages(B, **over):
    p = dict(batch=2, max_pages=4, block_tables=0x50000, bt_stride_b=4, bt_stride_h=0, seq_lens=0x60000,
             len_stride_b=1, len_stride_h=0, expected_tags=None)
    p.update(over)
    return B._CPages(**p)


def _append_case(mods, latent, **over):
    """The status of an append whose good arguments are replaced by `over`."""
    B, R, L = mods
    take = lambda name, **d: {k: over.get(name + "." + k, v) for k, v in d.items()}  # noqa: E731
    pages = _pages(B, **{k[6:]: v for k, v in over.items() if k.startswith("pages.")})
    rope = R._CRope(**take("rope", inv_freq=0x1000, rot_dim=64, interleaved=0, scale=1.0))
    tok = R._CNewTokens(**take("tok", num_new_tokens=3, positions=0x2000, new_lens=None, rope_positions=None,
                               row_starts=None, total_rows=0))
    rows = lambda name, at: R._CRows(**take(name, data=at, stride_b=8192, stride_t=1024, stride_h=128))  # noqa: E731
    k, v, q, o = rows("k", 0x10000), rows("v", 0x20000), rows("q", 0x30000), rows("o", 0x40000)
    ref = ctypes.byref
    if latent:
        cache = L._CLatentCache(**take("cache", num_pages=8, page_size=16, latent_dim=512, rope_dim=64, dtype=1,
                                       c_pages=0x100000, r_pages=0x200000, c_scale=0x300000, page_tags=None))
        fn = L.lib().pfkv_latent_append
    else:
        cache = B._CCache(**take("cache", num_pages=8, num_kv_heads=2, page_size=16, head_dim=128, dtype=1,
                                 k_pages=0x100000, v_pages=0x200000, k_scale=0x300000, v_scale=0x400000,
                                 page_tags=None))
        fn = R.lib().pfkv_rope_append
    arg = lambda name, s: None if over.get(name, 0) is None else ref(s)  # noqa: E731
    return fn(arg("cache", cache), arg("pages", pages), arg("rope", rope), arg("tok", tok), arg("k", k), arg("v", v),
              arg("q", q), arg("o", o), over.get("heads", 4), over.get("flags", 0x5000), None)


APPEND = [
    ({"cache": None}, 1), ({"pages": None}, 1), ({"rope": None}, 1), ({"tok": None}, 1), ({"k": None}, 1), ({"v": None}, 1),
    ({"q": None}, 1), ({"o": None}, 1), ({"heads": 0}, 1), ({"heads": 1 << 28}, 2),
    ({"rope.inv_freq": None}, 1), ({"rope.rot_dim": 0}, 1), ({"rope.rot_dim": 24}, 1), ({"rope.rot_dim": 144}, 1),
    ({"rope.interleaved": 2}, 1), ({"rope.scale": float("nan")}, 1), ({"rope.scale": float("inf")}, 1),
    ({"rope.inv_freq": 0x1002}, 3), ({"tok.num_new_tokens": 0}, 1), ({"tok.num_new_tokens": (1 << 24) + 1}, 2),
    ({"tok.positions": None}, 1), ({"tok.positions": 0x2001}, 3), ({"tok.new_lens": 0x2001}, 3),
    ({"tok.rope_positions": 0x2001}, 3), ({"tok.row_starts": 0x2002}, 3),
    ({"tok.row_starts": 0x2000, "tok.total_rows": -1}, 1),
    ({"k.data": None}, 1), ({"k.data": 0x10008}, 3), ({"k.stride_t": -8}, 1), ({"k.stride_t": 1020}, 3),
    ({"k.stride_b": 4}, 3), ({"v.data": 0x20004}, 3), ({"q.stride_h": 4}, 3), ({"o.data": 0x40002}, 3),
    ({"o.stride_h": -128}, 1), ({"flags": 0x5001}, 3),
    ({"cache.page_size": 32}, 2), ({"cache.dtype": 5}, 1), ({"cache.num_pages": 0}, 1), ({"pages.max_pages": 0}, 1),
    ({"pages.block_tables": None}, 1), ({"pages.bt_stride_b": 3}, 1), ({"pages.expected_tags": 0x7000}, 1),
]


@pytest.mark.parametrize("latent", [False, True])
@pytest.mark.parametrize("over,code", APPEND, ids=lambda x: str(x))
def test_appends_refuse(mods, latent, over, code):
    assert _append_case(mods, latent, **over) == code


def test_appends_of_their_own(mods):
    for latent in (False, True):
        assert _append_case(mods, latent) in NO_DEVICE
        assert _append_case(mods, latent, q=None, o=None, heads=0) in NO_DEVICE
        # packed rows have no stride of the batch
        assert _append_case(mods, latent, **{"tok.row_starts": 0x3000, "tok.total_rows": 9, "k.stride_b": 3}) in NO_DEVICE
        assert _append_case(mods, latent, **{"pages.batch": 0, "pages.block_tables": None, "pages.seq_lens": None}) == 0
    assert _append_case(mods, False, **{"cache.head_dim": 96}) == 2
    # a length a head needs the token's own position
    over = {"pages.len_stride_h": 1, "pages.len_stride_b": 2}
    assert _append_case(mods, False, **over) == 1
    assert _append_case(mods, False, **over, **{"tok.rope_positions": 0x3000}) in NO_DEVICE
    assert _append_case(mods, True, **over, **{"tok.rope_positions": 0x3000}) == 1
    assert _append_case(mods, True, **{"pages.bt_stride_h": 4}) == 1
    assert _append_case(mods, True, **{"cache.latent_dim": 256}) == 2
    assert _append_case(mods, True, **{"cache.rope_dim": 128}) == 2
    assert _append_case(mods, True, **{"rope.rot_dim": 80}) == 1
    assert _append_case(mods, True, **{"cache.c_scale": None}) == 1
    assert _append_case(mods, True, **{"cache.c_scale": None, "cache.dtype": 0}) in NO_DEVICE
    assert _append_case(mods, True, **{"cache.r_pages": 0x200008}) == 3
    # latents and keys have no head stride
    assert _append_case(mods, True, **{"k.stride_h": 3, "v.stride_h": -1}) in NO_DEVICE


def _latent(mods, **over):
    B, R, L = mods
    c = dict(num_pages=8, page_size=16, latent_dim=512, rope_dim=64, dtype=1, c_pages=0x100000, r_pages=0x200000,
             c_scale=0x300000, page_tags=None)
    c.update({k: v for k, v in over.items() if k in c})
    return L._CLatentCache(**c)


def _gather(mods, starts=0x1000, total=50, max_len=64, c=0x10000, cs=512, r=0x20000, rs=64, flags=0x5000, **over):
    B, R, L = mods
    return L.lib().pfkv_latent_gather(ctypes.byref(_latent(mods, **over)), ctypes.byref(_pages(B, **{
        k: v for k, v in over.items() if k == "batch"})), starts, total, max_len, c, cs, r, rs, flags, None)


def test_gather_refuses(mods):
    assert _gather(mods) in NO_DEVICE
    for over, code in ((dict(starts=None), 1), (dict(starts=0x1001), 3), (dict(total=-1), 1), (dict(max_len=-1), 1),
                       (dict(c=None), 1), (dict(r=None), 1), (dict(c=0x10008), 3), (dict(cs=504), 1), (dict(cs=516), 3),
                       (dict(rs=56), 1), (dict(rs=68), 3), (dict(flags=0x5002), 3), (dict(page_size=8), 2),
                       (dict(c_pages=None), 1), (dict(r_pages=0x200001), 3)):
        assert _gather(mods, **over) == code, over
    assert _gather(mods, max_len=0) == 0 and _gather(mods, batch=0) == 0
    assert _gather(mods, batch=1 << 30, max_len=1 << 20) == 2


def _decode(mods, heads=4, kq=2, scale=0.1, max_len=64, ws=0x900000, ws_bytes=1 << 40, flags=0x5000, pages=None, **over):
    B, R, L = mods
    rows = lambda name, at: R._CRows(**{k: over.get(name + "." + k, v) for k, v in dict(  # noqa: E731
        data=at, stride_b=4096, stride_t=2048, stride_h=512).items()})
    return L.lib().pfkv_latent_decode_attn(
        ctypes.byref(_latent(mods, **over)), ctypes.byref(_pages(B, **(pages or {}))), ctypes.byref(rows("qc", 0x10000)),
        ctypes.byref(rows("qr", 0x20000)), heads, kq, scale, max_len, ws, ws_bytes, ctypes.byref(rows("out", 0x30000)),
        flags, None)


def test_decode_refuses(mods):
    B, R, L = mods
    assert _decode(mods) in NO_DEVICE
    for over, code in ((dict(heads=0), 1), (dict(kq=0), 1), (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1),
                       (dict(max_len=-1), 1), (dict(ws=None), 4), (dict(ws=0x900010), 3), (dict(flags=0x5003), 3),
                       (dict(heads=1 << 20, kq=2), 2), (dict(latent_dim=128), 2), (dict(c_scale=None), 1),
                       ({"qc.data": None}, 1), ({"qr.data": 0x20002}, 3), ({"out.stride_t": 2044}, 3),
                       ({"qc.stride_b": -4096}, 1), (dict(pages=dict(seq_lens=None)), 1),
                       (dict(pages=dict(len_stride_h=1)), 1)):
        assert _decode(mods, **over) == code, over
    assert _decode(mods, pages=dict(batch=0)) == 0
    n = ctypes.c_size_t(0)
    size = lambda h, kq, out: L.lib().pfkv_latent_decode_workspace_size(  # noqa: E731
        ctypes.byref(_latent(mods)), ctypes.byref(_pages(B)), h, kq, 64, out)
    assert size(4, 1, None) == 1 and size(0, 1, ctypes.byref(n)) == 1 and size(4, 0, ctypes.byref(n)) == 1
    assert size(4, 1, ctypes.byref(n)) in (0,) + NO_DEVICE


def _prefill(mods, batch=2, heads=4, qs=0x1000, ks=0x2000, tq=10, tk=20, max_q=8, scale=0.1, flags=0x5000, **over):
    B, R, L = mods
    rows = [R._CRows(**{k: over.get(n + "." + k, v) for k, v in dict(data=at, stride_b=0, stride_t=1024, stride_h=256).items()})
            for n, at in (("qn", 0x10000), ("qr", 0x20000), ("kn", 0x30000), ("kr", 0x40000), ("v", 0x50000), ("out", 0x60000))]
    return L.lib().pfkv_latent_prefill_attn(batch, heads, qs, ks, tq, tk, max_q, *[ctypes.byref(r) for r in rows[:5]], scale,
                                            1, ctypes.byref(rows[5]), flags, None)


def test_prefill_refuses(mods):
    assert _prefill(mods) in NO_DEVICE
    assert _prefill(mods, batch=0) == 0
    for over, code in ((dict(batch=-1), 1), (dict(heads=0), 1), (dict(heads=65536), 2), (dict(qs=None), 1), (dict(ks=0x2002), 3),
                       (dict(tq=-1), 1), (dict(tk=1 << 31), 2), (dict(max_q=-1), 1), (dict(scale=float("nan")), 1),
                       (dict(flags=0x5001), 3), ({"qn.data": None}, 1), ({"qr.data": 0x20004}, 3), ({"kn.stride_h": 100}, 3),
                       ({"kr.stride_t": -8}, 1), ({"v.stride_h": -256}, 1), ({"out.data": 0x60008}, 3)):
        assert _prefill(mods, **over) == code, over
    assert _prefill(mods, **{"kr.stride_h": 3, "qn.stride_b": -5}) in NO_DEVICE   # not read


def test_bindings_refuse_shapes(mods, monkeypatch):
    """What the tensors show is refused before the library is called (host
    tensors stand in for device ones, whose addresses alone are taken)."""
    B, R, L = mods
    monkeypatch.setattr(B, "_ptr", lambda t: t if t is None or isinstance(t, int) else t.data_ptr())
    bf = torch.bfloat16
    cache = B.Cache(torch.zeros(4, 2, 16, 64, dtype=bf), torch.zeros(4, 2, 16, 64, dtype=bf))
    one = torch.zeros(1, dtype=torch.int32)
    pages = B.Pages(1, 1, one, 1, 0, one, 1, 0)
    rope = R.Rope(torch.zeros(32))
    k = torch.zeros(1, 3, 2, 64, dtype=bf)
    for bad in (dict(k_new=k[..., :32], v_new=k[..., :32]), dict(k_new=k.float(), v_new=k), dict(k_new=k[:, :, :1], v_new=k[:, :, :1]),
                dict(k_new=k, v_new=k[:, :2]), dict(k_new=k, v_new=k, q=k), dict(k_new=k, v_new=k, q=k, q_out=k[:, :2]),
                dict(k_new=k, v_new=k, max_new_tokens=4), dict(k_new=k[0], v_new=k[0], row_starts=torch.zeros(2, dtype=torch.int32)),
                dict(k_new=k[0], v_new=k[0], row_starts=one, max_new_tokens=3),
                dict(k_new=k.transpose(2, 3), v_new=k.transpose(2, 3))):
        with pytest.raises(ValueError):
            R.pfkv_rope_append(cache, pages, rope, one, **bad)
    lat = L.LatentCache(torch.zeros(4, 16, 512, dtype=bf), torch.zeros(4, 16, 64, dtype=bf))
    c, r = torch.zeros(1, 3, 512, dtype=bf), torch.zeros(1, 3, 64, dtype=bf)
    for bad in (dict(c_new=c, r_new=r[:, :2]), dict(c_new=r, r_new=r), dict(c_new=c, r_new=c), dict(c_new=c[0], r_new=r[0])):
        with pytest.raises(ValueError):
            L.pfkv_latent_append(lat, pages, rope, one, **bad)
    q = torch.zeros(1, 1, 4, 512, dtype=bf)
    qr, ws = torch.zeros(1, 1, 4, 64, dtype=bf), torch.zeros(256, dtype=torch.uint8)
    for a, b, o in ((q, qr[:, :, :2], q), (q, q, q), (q, qr, q[:, :, :2]), (q[0], qr[0], q[0]), (q.float(), qr, q)):
        with pytest.raises(ValueError):
            L.pfkv_latent_decode_attn(lat, pages, a, b, 0.1, 16, ws, o)
    with pytest.raises(ValueError):
        L.pfkv_latent_gather(lat, pages, one, 16, c[0], r[0])
    p = torch.zeros(5, 2, 128, dtype=bf)
    two = torch.zeros(2, dtype=torch.int32)
    pr, kr = torch.zeros(5, 2, 64, dtype=bf), torch.zeros(5, 64, dtype=bf)
    for bad in ((p, pr, p, kr[:4], p, two, two), (p, pr, p[:, :1], kr, p[:, :1], two, two), (p, p, p, kr, p, two, two),
                (p, pr, p, kr, p, two, one), (p, pr, p, kr, p, two.long(), two)):
        with pytest.raises(ValueError):
            L.pfkv_latent_prefill_attn(*bad, 5, 0.1, True, p)
