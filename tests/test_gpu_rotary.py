"""Rotary positions, alone and on the way into the paged cache, against 64 bits."""
import random

import pytest
import torch

import speculative_reference as R
from paged_kv_cache_95_gb300 import pagedkv as P

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib(built_library):
    P.load_library()


def normal(*shape, seed=0, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def close(got, want, norm):
    """Half a bf16 step of the value, and 2^-21 of the pair's length: the sine and the cosine (2 ulp each, and a rounding
    of the half turns, 2^-24 of pi at most), a product and a sum in fp32, each 2^-24."""
    got, want = got.double().cpu(), want.double()
    bound = want.abs() * 2.0 ** -8 + norm.double() * 2.0 ** -20 + 2.0 ** -133
    assert bool(((got - want).abs() <= bound).all()), float(((got - want).abs() / bound).max())


def pair_norm(x, r):
    return x.double().cpu().abs().amax(-1, keepdim=True) * 2 ** 0.5 + 0 * x.double().cpu()


FAR = [0, 1, -1, 7, 4095, 131071, 1000003, 2 ** 31 - 1, -2 ** 31]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("tokens,heads,dim,rotary", [(1, 1, 16, 16), (9, 3, 64, 64), (9, 1, 80, 32), (130, 5, 96, 48),
                                                     (33, 40, 128, 128), (700, 32, 128, 64), (3, 2, 1024, 1024)])
def test_rotary(tokens, heads, dim, rotary, layout):
    rng = random.Random(tokens + dim)
    pos = [FAR[i] if i < len(FAR) else rng.randint(0, 200000) for i in range(tokens)]
    x = normal(tokens, heads, dim + 64, seed=tokens)[..., 64:]  # a slice: strided
    freqs, mag = P.rotary_frequencies(rotary, 10000.0, scaling="by_parts", factor=4.0, original_length=2048)
    w, _ = R.frequencies(rotary, 10000.0, "by_parts", 4.0, 2048)
    out = torch.full((tokens + 1, heads, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    P.rotary_embedding(out[:tokens], x, i32(pos), freqs, layout=layout, magnitude=mag)
    close(out[:tokens], R.rotate(x, pos, w, layout, mag), pair_norm(x, rotary) * mag)
    assert torch.equal(out[:tokens, :, rotary:], x[..., rotary:])
    assert bool((out[tokens] == 7).all())
    # in place, the same bits
    y = x.clone()
    P.rotary_embedding(y, y, i32(pos), freqs, layout=layout, magnitude=mag)
    assert torch.equal(y, out[:tokens])


def test_rotary_of_head_major_rows_and_empty():
    x = normal(6, 50, 64, seed=3).transpose(0, 1)  # [tokens, heads, dim] lying head by head
    pos = list(range(100, 150))
    freqs, _ = P.rotary_frequencies(64)
    out = torch.empty(50, 6, 64, dtype=torch.bfloat16, device="cuda")
    P.rotary_embedding(out, x, i32(pos), freqs)
    w, _ = R.frequencies(64, 10000.0)
    close(out, R.rotate(x, pos, w, "half"), pair_norm(x, 64))
    P.rotary_embedding(out[:0], x[:0], i32([]), freqs)


def test_gradient_is_the_turn_back():
    """<turn(x, p), g> has the gradient turn(g, -p): by the formula and by differences in 64 bits."""
    pos = [3, 900, 77777]
    g = normal(3, 2, 32, seed=5)
    freqs, _ = P.rotary_frequencies(16, 1000.0)
    w, _ = R.frequencies(16, 1000.0)
    out = torch.empty_like(g)
    P.rotary_embedding(out, g, i32([-p for p in pos]), freqs, layout="interleaved")
    x = torch.randn(3, 2, 32, dtype=torch.float64)
    want = torch.empty_like(x)
    for i in range(x.numel()):
        step = torch.zeros_like(x).view(-1)
        step[i] = 0.5  # the turn is linear: any step is exact
        d = R.rotate(x + step.view_as(x), pos, w, "interleaved") - R.rotate(x - step.view_as(x), pos, w, "interleaved")
        want.view(-1)[i] = (d * g.double().cpu()).sum()
    close(out, want, pair_norm(g, 16))


def test_nonfinite_stays_in_its_pair():
    x = torch.ones(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    x[0, 0, 3], x[0, 0, 40] = float("nan"), float("inf")
    freqs, _ = P.rotary_frequencies(32)
    out = torch.empty_like(x)
    P.rotary_embedding(out, x, i32([5]), freqs)
    bad = ~torch.isfinite(out[0, 0]).cpu()
    assert bad.nonzero().flatten().tolist() == [3, 19, 40]


def pool(blocks, kv, fp8, seed=0):
    x = normal(2, blocks, kv, 16, 128, seed=seed)
    if not fp8:
        return x[0].clone(), x[1].clone(), None, None
    codes = x.float().to(F8)
    scales = torch.rand(2, blocks, kv, 16, device="cuda")
    return codes[0].clone(), codes[1].clone(), scales[0].clone(), scales[1].clone()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("tokens,heads,kv,rotary", [(1, 8, 8, 128), (5, 0, 1, 64), (67, 4, 1, 128), (64, 32, 8, 96),
                                                    (300, 15, 5, 32), (17, 3, 3, 16)])
def test_append(tokens, heads, kv, rotary, fp8, layout):
    rng = random.Random(tokens)
    blocks = tokens // 16 + 3
    x = normal(tokens, heads + 2 * kv, 128, seed=tokens)
    q, key, value = x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:]
    pos = [rng.randint(0, 1000000) for _ in range(tokens)]
    slots = rng.sample(range(blocks * 16), tokens)
    if tokens > 4:
        slots[1], slots[3] = -1, blocks * 16  # padding, and a slot past the pool
    freqs, _ = P.rotary_frequencies(rotary, 500000.0)
    w, _ = R.frequencies(rotary, 500000.0)
    kc, vc, ks, vs = pool(blocks, kv, fp8)
    before = [t.clone() for t in (kc, vc, ks, vs) if t is not None]
    q_out = torch.empty(tokens, heads, 128, dtype=torch.bfloat16, device="cuda") if heads else None
    args = (q_out, q if heads else None, key, value, kc, vc, *((ks, vs) if fp8 else ()), i32(pos), i32(slots), freqs)
    (P.rotary_reshape_and_cache_fp8 if fp8 else P.rotary_reshape_and_cache)(*args, layout=layout)
    turned = torch.empty(tokens, kv, 128, dtype=torch.bfloat16, device="cuda")
    P.rotary_embedding(turned, key, i32(pos), freqs, layout=layout)
    if heads:
        want = torch.empty(tokens, heads, 128, dtype=torch.bfloat16, device="cuda")
        P.rotary_embedding(want, q, i32(pos), freqs, layout=layout)
        assert torch.equal(q_out, want)
    keep = [i for i, s in enumerate(slots) if 0 <= s < blocks * 16]
    at = torch.tensor([slots[i] for i in keep], device="cuda")
    if not fp8:
        # the same pool as the two calls leave
        k2, v2 = before
        P.kv_reshape_and_cache(turned, value.contiguous(), k2, v2, i32(slots))
        assert torch.equal(kc, k2) and torch.equal(vc, v2)
        return
    # values: the same codes as the append without a turn
    k2, v2, ks2, vs2 = before
    P.kv_reshape_and_cache_fp8(turned, value.contiguous(), k2, v2, ks2, vs2, i32(slots))
    assert torch.equal(vc.view(torch.uint8), v2.view(torch.uint8)) and torch.equal(vs, vs2)
    # keys: against 64 bits, a scale (two fp32 roundings and the turn's 2^-20) and half a code's step (2^-4
    # relative, 2^-10 of the scale's unit below the normal codes)
    exact = R.rotate(key, pos, w, layout)[keep]
    scale = ks[at // 16, :, at % 16].double().cpu()
    want = exact.abs().amax(-1) / 448
    assert bool(((scale - want).abs() <= want * 2.0 ** -18).all())
    got = kc[at // 16, :, at % 16].float().double().cpu() * scale[..., None]
    bound = exact.abs() * 2.0 ** -4 + scale[..., None] * 2.0 ** -10 + scale[..., None] * 448 * 2.0 ** -18
    assert bool(((got - exact).abs() <= bound).all())
    # what has no slot of this call is untouched
    rest = torch.ones(blocks * 16, dtype=torch.bool, device="cuda")
    rest[at] = False
    for got, old in ((kc, k2), (ks, ks2)):
        a, b = (t.view(torch.uint8 if t.dtype == F8 else t.dtype).transpose(1, 2).flatten(0, 1)[rest] for t in (got, old))
        assert torch.equal(a, b)


def test_append_in_place_of_q_and_with_zero_rows():
    q, key, value = normal(20, 4, 128, seed=1), torch.zeros(20, 2, 128, device="cuda").bfloat16(), normal(20, 2, 128, seed=2)
    freqs, _ = P.rotary_frequencies(128)
    want = torch.empty_like(q)
    P.rotary_embedding(want, q, i32(list(range(20))), freqs)
    kc, vc, ks, vs = pool(4, 2, True)
    P.rotary_reshape_and_cache_fp8(q, q, key, value, kc, vc, ks, vs, i32(list(range(20))), i32(list(range(20))), freqs)
    assert torch.equal(q, want)
    assert bool((kc[0].float() == 0).all()) and bool((ks[0] == 2.0 ** -100 / 448).all())
    P.rotary_reshape_and_cache_fp8(q[:0], q[:0], key[:0], value[:0], kc, vc, ks, vs, i32([]), i32([]), freqs)


def test_binding_refusals():
    x, out = normal(4, 2, 64), normal(4, 2, 64, seed=1)
    pos, (freqs, _) = i32([1, 2, 3, 4]), P.rotary_frequencies(64)
    kc, vc, ks, vs = pool(2, 2, False)
    kv = normal(4, 2, 128)
    for call in (lambda: P.rotary_embedding(out[:3], x, pos, freqs), lambda: P.rotary_embedding(out, x, pos[:3], freqs),
                 lambda: P.rotary_embedding(out, x.float(), pos, freqs), lambda: P.rotary_embedding(out, x, pos.long(), freqs),
                 lambda: P.rotary_embedding(out, x, pos, freqs.int()), lambda: P.rotary_embedding(out, x, pos, freqs, layout="x"),
                 lambda: P.rotary_embedding(out, x[..., ::2], pos, freqs), lambda: P.rotary_embedding(out.cpu(), x, pos, freqs),
                 lambda: P.rotary_embedding(None, x, pos, freqs), lambda: P.rotary_embedding(out, None, pos, freqs),
                 lambda: P.rotary_reshape_and_cache(None, None, kv, kv[:3], kc, vc, pos, pos, freqs),
                 lambda: P.rotary_reshape_and_cache(kv, None, kv, kv, kc, vc, pos, pos, freqs),
                 lambda: P.rotary_reshape_and_cache(kv[:, :1], kv, kv, kv, kc, vc, pos, pos, freqs),
                 lambda: P.rotary_reshape_and_cache(kv, kv, kv, kv, kc, vc[:1], pos, pos, freqs),
                 lambda: P.rotary_reshape_and_cache_fp8(kv, kv, kv, kv, kc, vc, None, None, pos, pos, freqs)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(P.PagedKVError):
        P.rotary_embedding(out, x, pos, torch.cat([freqs, freqs]))  # more rotated than there is


def test_other_stream_and_graph():
    x, pos = normal(64, 8, 128, seed=9), i32(list(range(64)))
    freqs, _ = P.rotary_frequencies(128)
    want, out = torch.empty_like(x), torch.zeros_like(x)
    P.rotary_embedding(want, x, pos, freqs)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    P.rotary_embedding(out, x, pos, freqs, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    out.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.rotary_embedding(out, x, pos, freqs)
    x.neg_()
    pos.add_(5)
    graph.replay()
    P.rotary_embedding(want, x, pos, freqs)
    assert torch.equal(out, want)
