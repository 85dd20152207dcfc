"""Entry points of a speculative decoding step: argument errors are found on the host, before
anything reaches the GPU (CPU only), and the rotary frequencies against their formulas."""
import ctypes
import math

import pytest
import torch

import speculative_reference as R
from paged_kv_cache_95_gb300 import pagedkv as P

FAKE = 0x100000  # never dereferenced: validation fails before any device access
INV, UNS, WS = P.PKV_ERR_INVALID_ARG, P.PKV_ERR_UNSUPPORTED, P.PKV_ERR_WORKSPACE_TOO_SMALL
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib(built_library):
    return P.load_library()


def desc(num_blocks=100, bs=16, n_kv=8, d=128, dtype=0):
    return P.CacheDesc(num_blocks, bs, n_kv, d, dtype)


BAD_DESC = [(dict(num_blocks=0), INV), (dict(bs=32), UNS), (dict(n_kv=0), INV), (dict(d=64), UNS), (dict(dtype=1), UNS)]


@pytest.mark.parametrize("kw", [
    dict(), dict(scaling="linear", factor=4.0), dict(scaling="linear", factor=0.25), dict(scaling="ntk", factor=8.0),
    dict(scaling="by_parts", factor=32.0, length=4096), dict(scaling="by_parts", factor=0.5, length=100),
    dict(scaling="by_wavelength", factor=8.0, length=8192, low=1.0, high=4.0),
])
@pytest.mark.parametrize("dim,base", [(2, 10000.0), (16, 10000.0), (64, 500000.0), (128, 10000.0), (128, 1.5)])
def test_frequencies(lib, dim, base, kw):
    if kw.get("scaling") == "ntk" and dim == 2:
        pytest.skip("no such base")
    kw = dict(kw)
    length = kw.pop("length", 0)
    freqs, magnitude = P.rotary_frequencies(dim, base, original_length=length, device="cpu", **kw)
    want, mag = R.frequencies(dim, base, length=length, **kw)
    assert magnitude == pytest.approx(mag, rel=2.0 ** -23)
    for got, w in zip(freqs.tolist(), want):
        turns = w / (2 * math.pi)
        # a double holds a turn to 2^-53; powers and logarithms of a few steps: 2^-49 relative; modulo a turn
        off = (got / 2.0 ** 64 - turns) % 1.0
        assert min(off, 1.0 - off) <= 2.0 ** -49 * max(turns, 2.0 ** -12), (got, turns)


@pytest.mark.parametrize("args", [
    (0, 10000.0, 0, 0, 1.0, 1.0, 32.0), (3, 10000.0, 0, 0, 1.0, 1.0, 32.0), (64, 1.0, 0, 0, 1.0, 1.0, 32.0),
    (64, NAN, 0, 0, 1.0, 1.0, 32.0), (64, INF, 0, 0, 1.0, 1.0, 32.0), (64, 1e4, 5, 0, 1.0, 1.0, 32.0),
    (64, 1e4, -1, 0, 1.0, 1.0, 32.0), (64, 1e4, 1, 0, 0.0, 1.0, 32.0), (64, 1e4, 1, 0, NAN, 1.0, 32.0),
    (64, 1e4, 1, 0, INF, 1.0, 32.0), (2, 1e4, 2, 0, 4.0, 1.0, 32.0), (64, 1e4, 2, 0, 1e-9, 1.0, 32.0),
    (64, 1e300, 2, 0, 1e200, 1.0, 32.0), (64, 1e4, 3, 0, 4.0, 1.0, 32.0), (64, 1e4, 3, 100, 4.0, 0.0, 32.0),
    (64, 1e4, 4, 100, 4.0, 4.0, 4.0), (64, 1e4, 4, 100, 4.0, 1.0, INF), (64, 1e4, 4, 100, 4.0, NAN, 4.0),
])
def test_frequency_refusals(lib, args):
    dim, base, kind, length, factor, low, high = args
    out, mag = (ctypes.c_uint64 * 64)(), ctypes.c_float()
    how = P.RotaryScaling(kind, length, factor, low, high)
    assert lib.rotary_frequencies(out, ctypes.byref(mag), dim, base, ctypes.byref(how)) == INV


def test_frequency_pointers(lib):
    out, mag = (ctypes.c_uint64 * 64)(), ctypes.c_float()
    assert lib.rotary_frequencies(None, ctypes.byref(mag), 64, 1e4, None) == INV
    assert lib.rotary_frequencies(out, None, 64, 1e4, None) == INV
    assert lib.rotary_frequencies(out, ctypes.byref(mag), 64, 1e4, None) == 0 and mag.value == 1.0
    with pytest.raises(ValueError):
        P.rotary_frequencies(64, scaling="other", device="cpu")


@pytest.mark.parametrize("kw,want", [
    (dict(out=None), INV), (dict(x=None), INV), (dict(pos=None), INV), (dict(fr=None), INV), (dict(out=FAKE + 8), INV),
    (dict(x=FAKE + 2), INV), (dict(pos=FAKE + 2), INV), (dict(fr=FAKE + 4), INV), (dict(n=-1), INV), (dict(h=0), INV),
    (dict(xr=-8), INV), (dict(xh=4), INV), (dict(outr=12), INV), (dict(outh=1 << 40), INV), (dict(d=0), INV),
    (dict(d=72, r=64), UNS), (dict(d=2048, r=16), UNS), (dict(h=70000), UNS), (dict(r=0), INV), (dict(r=24), UNS),
    (dict(r=144), INV), (dict(layout=2), INV), (dict(layout=-1), INV), (dict(m=NAN), INV), (dict(m=INF), INV),
    (dict(out=FAKE, outr=2048), INV), (dict(n=0), 0),
])
def test_rotary_refusals(lib, kw, want):
    a = dict(out=2 * FAKE, outr=1024, outh=128, x=FAKE, xr=1024, xh=128, pos=FAKE, fr=FAKE, n=4, h=8, d=128, r=128,
             layout=0, m=1.0)
    a.update(kw)
    assert lib.rotary_embedding(a["out"], a["outr"], a["outh"], a["x"], a["xr"], a["xh"], a["pos"], a["fr"], a["n"],
                                a["h"], a["d"], a["r"], a["layout"], a["m"], None) == want


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,want", [
    (dict(qo=None), INV), (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(kc=None), INV),
    (dict(vc=None), INV), (dict(pos=None), INV), (dict(sl=None), INV), (dict(fr=None), INV), (dict(q=FAKE + 8), INV),
    (dict(qo=FAKE + 4), INV), (dict(k=FAKE + 2), INV), (dict(v=FAKE + 8), INV), (dict(kc=FAKE + 8), INV),
    (dict(sl=FAKE + 1), INV), (dict(qr=12), INV), (dict(kh=-8), INV), (dict(vr=7), INV), (dict(n=-1), INV),
    (dict(h=-1), INV), (dict(h=70000), UNS), (dict(r=0), INV), (dict(r=136), INV), (dict(r=40), UNS), (dict(layout=7), INV),
    (dict(m=NAN), INV), (dict(n=0), 0), (dict(q=FAKE, qr=1032), INV), (dict(q=FAKE, qh=256), INV),
    *[(k, w) for k, w in BAD_DESC],
])
def test_rotary_write_refusals(lib, fp8, kw, want):
    a = dict(qo=FAKE, q=2 * FAKE, qr=1024, qh=128, k=FAKE, kr=1024, kh=128, v=FAKE, vr=1024, vh=128, kc=FAKE, vc=FAKE, pos=FAKE,
             sl=FAKE, fr=FAKE, n=4, h=8, r=128, layout=0, m=1.0)
    d = {k: v for k, v in kw.items() if k in ("num_blocks", "bs", "n_kv", "d", "dtype")}
    a.update({k: v for k, v in kw.items() if k not in d})
    c = desc(**{"dtype": 2 if fp8 else 0, **d})
    head = [a[n] for n in ("qo", "q", "qr", "qh", "k", "kr", "kh", "v", "vr", "vh", "kc", "vc")]
    tail = [a[n] for n in ("pos", "sl", "fr", "n", "h", "r", "layout", "m")]
    if fp8:
        assert lib.rotary_reshape_and_cache_fp8(*head, FAKE, FAKE, *tail, ctypes.byref(c), None) == want
    else:
        assert lib.rotary_reshape_and_cache(*head, *tail, ctypes.byref(c), None) == want


@pytest.mark.parametrize("ks,vs,dtype,want", [(None, FAKE, 2, INV), (FAKE, None, 2, INV), (FAKE + 4, FAKE, 2, INV),
                                              (FAKE, FAKE, 0, UNS)])
def test_rotary_write_fp8_scales(lib, ks, vs, dtype, want):
    c = desc(dtype=dtype)
    assert lib.rotary_reshape_and_cache_fp8(FAKE, FAKE, 1024, 128, FAKE, 1024, 128, FAKE, 1024, 128, FAKE, FAKE, ks, vs,
                                            FAKE, FAKE, FAKE, 4, 8, 128, 0, 1.0, ctypes.byref(c), None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(out=None), INV), (dict(path=None), INV), (dict(n=None), INV), (dict(t=None), INV), (dict(tok=None), INV),
    (dict(u=None), INV), (dict(cu=None), INV), (dict(t=FAKE + 2), INV), (dict(tok=FAKE + 2), INV), (dict(st=FAKE + 2), INV),
    (dict(up=FAKE + 2), INV), (dict(B=0), INV), (dict(B=65536), INV), (dict(most=0), INV), (dict(most=65), INV),
    (dict(rows=-1), INV), (dict(V=0), INV), (dict(V=(1 << 24) + 1, ts=1 << 25), UNS), (dict(ts=999), INV),
    (dict(ts=1 << 38), INV), (dict(q=FAKE, qs=999, up=None), INV), (dict(q=FAKE, qs=1000), UNS),
])
def test_verify_refusals(lib, kw, want):
    a = dict(out=FAKE, path=FAKE, n=FAKE, t=FAKE, ts=1000, q=None, qs=0, tok=FAKE, up=FAKE, u=FAKE, cu=FAKE, B=2, most=8,
             rows=10, V=1000, st=None)
    a.update(kw)
    assert lib.speculative_verify(a["out"], a["path"], a["n"], a["t"], a["ts"], a["q"], a["qs"], a["tok"], a["up"], a["u"],
                                  a["cu"], a["B"], a["most"], a["rows"], a["V"], a["st"], None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(kc=None), INV), (dict(vc=None), INV), (dict(bt=None), INV), (dict(cl=None), INV), (dict(cu=None), INV),
    (dict(path=None), INV), (dict(n=None), INV), (dict(kc=FAKE + 8), INV), (dict(bt=FAKE + 2), INV), (dict(st=FAKE + 1), INV),
    (dict(B=0), INV), (dict(mb=0), INV), (dict(mb=1 << 28), INV), (dict(most=0), INV), (dict(most=65), INV),
    (dict(ks=FAKE), INV), (dict(vs=FAKE), INV), (dict(c=dict(dtype=2)), INV),
    (dict(c=dict(dtype=2), ks=FAKE, vs=FAKE + 4), INV), *[(dict(c=k), w) for k, w in BAD_DESC],
])
def test_compact_refusals(lib, kw, want):
    a = dict(kc=FAKE, vc=FAKE, ks=None, vs=None, bt=FAKE, cl=FAKE, cu=FAKE, path=FAKE, n=FAKE, B=2, mb=8, most=8, c={}, st=None)
    a.update(kw)
    c = desc(**a["c"])
    assert lib.kv_compact_path(a["kc"], a["vc"], a["ks"], a["vs"], a["bt"], a["cl"], a["cu"], a["path"], a["n"], a["B"],
                               a["mb"], a["most"], ctypes.byref(c), a["st"], None) == want


def test_reference_rotation_turns_back():
    x = torch.randn(3, 2, 32, dtype=torch.float64)
    w, _ = R.frequencies(16, 100.0)
    for layout in ("half", "interleaved"):
        y = R.rotate(R.rotate(x, [5, 70, 1000], w, layout), [-5, -70, -1000], w, layout)
        assert torch.allclose(x, y, atol=1e-12, rtol=0)


@pytest.mark.parametrize("kw,want", [
    (dict(out=None), INV), (dict(q=None), INV), (dict(m=None), INV), (dict(cu=None), INV), (dict(kc=None), INV),
    (dict(vc=None), INV), (dict(bt=None), INV), (dict(cl=None), INV), (dict(ws=None), INV), (dict(out=FAKE + 8), INV),
    (dict(q=FAKE + 8), INV), (dict(m=FAKE + 4), INV), (dict(kc=FAKE + 8), INV), (dict(cu=FAKE + 2), INV),
    (dict(ws=FAKE + 128), INV), (dict(wb=256), WS), (dict(od=2), UNS), (dict(B=0), INV), (dict(B=65536), INV),
    (dict(most=0), INV), (dict(most=65), INV), (dict(rows=-1), INV), (dict(h=0), INV), (dict(h=12), INV),
    (dict(h=1032), UNS), (dict(mb=0), INV), (dict(mb=1 << 27), INV), (dict(s=NAN), INV), (dict(s=INF), INV),
    (dict(s=3e38), INV), (dict(ks=FAKE), INV), (dict(c=dict(dtype=2)), INV), (dict(c=dict(dtype=2), ks=FAKE, vs=FAKE + 4), INV),
    (dict(c=dict(num_blocks=1 << 30)), UNS), (dict(rows=0), 0), *[(dict(c=k), w) for k, w in BAD_DESC],
])
def test_tree_refusals(lib, kw, want):
    a = dict(out=FAKE, od=0, q=FAKE, m=FAKE, cu=FAKE, most=8, rows=16, kc=FAKE, vc=FAKE, ks=None, vs=None, bt=FAKE, cl=FAKE,
             B=2, h=32, mb=8, s=0.1, c={}, ws=FAKE, wb=1 << 30)
    a.update(kw)
    c = desc(**a["c"])
    assert lib.paged_attention_tree(a["out"], a["od"], a["q"], a["m"], a["cu"], a["most"], a["rows"], a["kc"], a["vc"],
                                    a["ks"], a["vs"], a["bt"], a["cl"], a["B"], a["h"], a["mb"], a["s"], ctypes.byref(c),
                                    a["ws"], a["wb"], None) == want


def test_tree_workspace(lib):
    size = lambda *a, **k: lib.paged_attention_tree_workspace_size(*a, ctypes.byref(desc(**k)))  # noqa: E731
    assert size(0, 32, 8) == size(2, 12, 8) == size(2, 32, 65) == size(2, 32, 8, bs=8) == 0
    # a status word, a record a range, and per range two partials of the rows of a tile: (m, l) and 128 values
    for heads, most, rows in ((32, 8, 32), (64, 64, 128), (8, 1, 1), (40, 3, 15)):
        n = size(2, heads, most)
        assert 304 * rows * 520 <= n <= 304 * rows * 520 + 4096
        assert n == size(60000, heads, most) == size(2, heads, most, dtype=2)
