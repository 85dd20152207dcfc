"""Latent-attention entry points: argument errors are found on the host, before anything
reaches the GPU (CPU only), and the 64-bit reference forms agree with each other."""
import ctypes

import pytest
import torch

import latent_reference as R
from paged_kv_cache_95_gb300 import pagedkv as P

FAKE = 0x100000  # never dereferenced: validation fails before any device access
INV, UNS, WS = P.PKV_ERR_INVALID_ARG, P.PKV_ERR_UNSUPPORTED, P.PKV_ERR_WORKSPACE_TOO_SMALL


@pytest.fixture(scope="module")
def lib(built_library):
    return P.load_library()


def desc(num_blocks=100, bs=16, latent=512, rope=64, dtype=0):
    return P.LatentDesc(num_blocks, bs, latent, rope, dtype)


BAD_DESC = [(dict(num_blocks=0), INV), (dict(bs=32), UNS), (dict(latent=256), UNS), (dict(rope=32), UNS)]


@pytest.mark.parametrize("kw,want", [
    (dict(latent=None), INV), (dict(rope=None), INV), (dict(cache=None), INV), (dict(slots=None), INV),
    (dict(n=-1), INV), (dict(ls=516), INV), (dict(ls=-8), INV), (dict(rs=63), INV), (dict(latent=FAKE + 8), INV),
    (dict(rope=FAKE + 2), INV), (dict(cache=FAKE + 8), INV), (dict(slots=FAKE + 2), INV),
    *[(dict(d=desc(**k)), w) for k, w in BAD_DESC], (dict(d=desc(dtype=2)), UNS), (dict(n=0), 0),
])
def test_write_refusals(lib, kw, want):
    a = dict(latent=FAKE, ls=512, rope=FAKE, rs=64, cache=FAKE, slots=FAKE, n=4, d=desc())
    a.update(kw)
    assert lib.latent_reshape_and_cache(a["latent"], a["ls"], a["rope"], a["rs"], a["cache"], a["slots"], a["n"],
                                        ctypes.byref(a["d"]), None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(rc=None), INV), (dict(sc=None), INV), (dict(rc=FAKE + 8), INV), (dict(sc=FAKE + 4), INV),
    (dict(d=desc(dtype=0)), UNS), (dict(n=0), 0),
])
def test_write_fp8_refusals(lib, kw, want):
    a = dict(rc=FAKE, sc=FAKE, n=4, d=desc(dtype=2))
    a.update(kw)
    assert lib.latent_reshape_and_cache_fp8(FAKE, 576, FAKE, 576, FAKE, a["rc"], a["sc"], FAKE, a["n"],
                                            ctypes.byref(a["d"]), None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(out=None), INV), (dict(cache=None), INV), (dict(bt=None), INV), (dict(cu=None), INV), (dict(B=0), INV),
    (dict(mb=0), INV), (dict(mb=1 << 28), INV), (dict(n=-1), INV), (dict(out=FAKE + 8), INV), (dict(st=FAKE + 2), INV),
    (dict(rc=FAKE), INV), (dict(sc=FAKE), INV), (dict(d=desc(dtype=2)), INV), (dict(d=desc(dtype=1)), UNS),
    *[(dict(d=desc(**k)), w) for k, w in BAD_DESC], (dict(n=0), 0),
])
def test_gather_refusals(lib, kw, want):
    a = dict(out=FAKE, cache=FAKE, rc=None, sc=None, bt=FAKE, cu=FAKE, B=2, mb=8, n=10, d=desc(), st=None)
    a.update(kw)
    assert lib.latent_gather(a["out"], a["cache"], a["rc"], a["sc"], a["bt"], a["cu"], a["B"], a["mb"], a["n"],
                             ctypes.byref(a["d"]), a["st"], None) == want


DECODE = [
    (dict(out=None), INV), (dict(ql=None), INV), (dict(qr=None), INV), (dict(cache=None), INV), (dict(bt=None), INV),
    (dict(cl=None), INV), (dict(ws=None), INV), (dict(ws=FAKE + 64), INV), (dict(wsb=255), WS), (dict(B=0), INV),
    (dict(B=65536), INV), (dict(k=0), INV), (dict(k=17), INV), (dict(h=0), INV), (dict(h=1025), UNS), (dict(mb=0), INV),
    (dict(mb=1 << 28), INV), (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV), (dict(od=2), UNS),
    (dict(qlr=4), INV), (dict(qlh=-512), INV), (dict(out=FAKE + 4), INV), (dict(ql=FAKE + 8), INV),
    (dict(cache=FAKE + 8), INV), *[(dict(d=desc(**k)), w) for k, w in BAD_DESC],
]


def _decode(lib, a, fp8):
    head = (a["out"], a["od"], a["ql"], a["qlr"], a["qlh"], a["qr"], 64 * 32, 64, a["cache"])
    tail = (a["bt"], a["cl"], a["B"], a["k"], a["h"], a["mb"], a["scale"], ctypes.byref(a["d"]), a["ws"], a["wsb"], None)
    if fp8:
        return lib.latent_attention_decode_fp8(*head, a["rc"], a["sc"], *tail)
    return lib.latent_attention_decode(*head, *tail)


def _decode_args(**kw):
    a = dict(out=FAKE, od=1, ql=FAKE, qlr=512 * 32, qlh=512, qr=FAKE, cache=FAKE, rc=FAKE, sc=FAKE, bt=FAKE, cl=FAKE, B=4,
             k=1, h=32, mb=8, scale=0.07, d=desc(), ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,want", DECODE + [(dict(d=desc(dtype=2)), UNS)])
def test_decode_refusals(lib, kw, want):
    assert _decode(lib, _decode_args(**kw), False) == want


@pytest.mark.parametrize("kw,want", [(dict(rc=None), INV), (dict(sc=None), INV), (dict(rc=FAKE + 8), INV),
                                     (dict(sc=FAKE + 8), INV), (dict(d=desc()), UNS), (dict(k=17), INV)])
def test_decode_fp8_refusals(lib, kw, want):
    assert _decode(lib, _decode_args(**{"d": desc(dtype=2), **kw}), True) == want


def test_decode_workspace_size(lib):
    size = lambda *a, **k: lib.latent_attention_workspace_size(*a, ctypes.byref(desc(**k)))  # noqa: E731
    for dtype in (0, 2):
        assert size(4, 1, 32, 64, dtype=dtype) >= 256
        # the call accepts exactly what the query answers
        need = size(64, 4, 128, 256, dtype=dtype)
        a = _decode_args(d=desc(dtype=dtype), B=64, k=4, h=128, mb=256, wsb=need - 1)
        assert _decode(lib, a, dtype == 2) == WS
    for bad in ((0, 1, 32, 64), (4, 0, 32, 64), (4, 17, 32, 64), (4, 1, 0, 64), (4, 1, 1025, 64), (4, 1, 32, 0)):
        assert size(*bad) == 0
    assert size(4, 1, 32, 64, dtype=1) == 0
    assert lib.latent_attention_workspace_size(4, 1, 32, 64, None) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(out=None), INV), (dict(q=None), INV), (dict(kn=None), INV), (dict(v=None), INV), (dict(kr=None), INV),
    (dict(cq=None), INV), (dict(ck=None), INV), (dict(ws=None), INV), (dict(ws=FAKE + 8), INV), (dict(wsb=128), WS),
    (dict(B=0), INV), (dict(B=65536), INV), (dict(h=0), INV), (dict(h=1025), UNS), (dict(mq=-1), INV), (dict(tq=-1), INV),
    (dict(tk=0), INV), (dict(scale=float("nan")), INV), (dict(od=0x7), UNS), (dict(qs=0), INV), (dict(ks=0), INV),
    (dict(rs=0), INV), (dict(qs=100), INV), (dict(rs=68), INV), (dict(out=FAKE + 8), INV), (dict(q=FAKE + 8), INV),
    (dict(v=FAKE + 8), INV), (dict(tq=0), 0), (dict(mq=0), 0),
])
def test_prefill_refusals(lib, kw, want):
    a = dict(out=FAKE, od=1, q=FAKE, qs=192 * 8, kn=FAKE, v=FAKE, ks=256 * 8, kr=FAKE, rs=576, cq=FAKE, ck=FAKE, B=2, h=8,
             mq=16, tq=20, tk=40, scale=0.07, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    assert lib.latent_attention_prefill_chunk(a["out"], a["od"], a["q"], a["qs"], 192, a["kn"], a["v"], a["ks"], 256,
                                              a["kr"], a["rs"], a["cq"], a["ck"], a["B"], a["h"], a["mq"], a["tq"],
                                              a["tk"], a["scale"], a["ws"], a["wsb"], None) == want


def test_null_descriptor(lib):
    assert lib.latent_reshape_and_cache(FAKE, 512, FAKE, 64, FAKE, FAKE, 1, None, None) == INV
    assert lib.latent_gather(FAKE, FAKE, None, None, FAKE, FAKE, 1, 1, 1, None, None, None) == INV


def test_reference_absorbed_equals_expanded():
    """The two forms are the same attention: keys and values mapped from the latents, or the
    maps moved to the query and the output."""
    heads, n = 3, 37
    pool = R.Pool(5, [n])
    g = R.gen(6)
    wk, wv = (torch.randn(heads, 128, 512, generator=g, dtype=torch.float64) * 0.05 for _ in range(2))
    q = torch.randn(4, heads, 192, generator=g, dtype=torch.float64)
    rows = pool.sequence(0)
    absorbed = torch.einsum("rhd,hdc->rhc", q[..., :128], wk)
    out, _ = R.decode(absorbed, q[..., 128:], pool, 4)
    k_nope = torch.einsum("jc,hdc->jhd", rows[:, :512], wk)
    v = torch.einsum("jc,hdc->jhd", rows[:, :512], wv)
    want, _ = R.expanded(q, k_nope, v, rows[:, 512:], [4], [n])
    assert torch.allclose(torch.einsum("rhc,hdc->rhd", out, wv), want, atol=1e-12)


@pytest.mark.parametrize("kw,want", [
    (dict(mb=(1 << 27) - 1), INV), (dict(scale=3e38), INV), (dict(scale=-3e38), INV), (dict(qlr=1 << 38), INV),
    (dict(qlh=1 << 40), INV),
])
def test_decode_refuses_what_overflows(lib, kw, want):
    """Lengths that do not round up to a tile in 32 bits, scales infinite in the log2 domain, strides past a tensor."""
    for fp8 in (False, True):
        assert _decode(lib, _decode_args(d=desc(dtype=2 if fp8 else 0), **kw), fp8) == want


@pytest.mark.parametrize("kw,want", [
    (dict(mq=65535 * 256 + 1, tq=(1 << 30)), UNS), (dict(mq=1 << 30, tq=65535 * 256 + 1), UNS), (dict(tq=2 ** 31 - 1), INV),
    (dict(tk=2 ** 31 - 1), INV), (dict(scale=3e38), INV), (dict(qs=1 << 38), INV),
])
def test_prefill_refuses_what_overflows(lib, kw, want):
    a = dict(qs=192 * 8, mq=16, tq=20, tk=40, scale=0.07)
    a.update(kw)
    assert lib.latent_attention_prefill_chunk(FAKE, 1, FAKE, a["qs"], 192, FAKE, FAKE, 256 * 8, 256, FAKE, 576, FAKE, FAKE, 2, 8,
                                              a["mq"], a["tq"], a["tk"], a["scale"], FAKE, 1 << 30, None) == want


def test_gather_refuses_what_overflows(lib):
    for mb, n in (((1 << 27) - 1, 10), (8, 2 ** 31 - 1)):
        assert lib.latent_gather(FAKE, FAKE, None, None, FAKE, FAKE, 2, mb, n, ctypes.byref(desc()), None, None) == INV


def test_prefill_workspace_size(lib):
    """Parts of the keys need room only where few rows meet many keys; the status word alone is accepted."""
    size = lib.latent_attention_prefill_workspace_size
    assert size(1, 32, 8192, 8192, 8192) == 256 and size(4, 32, 400, 1200, 2000) == 256 and size(1, 8, 100, 100, 500) == 256
    need = size(1, 8, 100, 100, 4000)
    assert need > 256 and (need - 256) % 256 == 0
    assert size(1, 8, 0, 0, 0) == 256
    for bad in ((0, 8, 1, 1, 1), (65536, 8, 1, 1, 1), (1, 0, 1, 1, 1), (1, 1025, 1, 1, 1), (1, 8, -1, 1, 1), (1, 8, 1, -1, 1)):
        assert size(*bad) == 0
