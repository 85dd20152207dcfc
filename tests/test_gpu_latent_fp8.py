"""Absorbed attention over an FP8 latent pool: what its codes, scales and factors could get wrong."""
import pytest
import torch

import latent_reference as R
from paged_kv_cache_95_gb300 import pagedkv as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(built_library):
    P.load_library()


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def status_of(ws):
    return int(ws[:4].view(torch.int32).cpu().item()) & 0xFFFFFFFF


@pytest.mark.parametrize("heads", [16, 32, 64])
def test_sequences_of_one_tile_keep_their_own_query_factors(heads):
    """Hundreds of sequences of up to 64 tokens, whose queries differ in size by 2^8 from one to the next: a query's
    factor taken for its neighbour's would make its scores 256 times too large or too small."""
    lens = [1 + (i * 29) % 64 for i in range(400)]
    pool = R.Pool(heads, lens, True)
    g = R.gen(heads + 1)
    size = torch.tensor([1.0 if i % 2 else 2.0 ** -8 for i in range(len(lens))]).bfloat16()[:, None, None]
    ql, qr = R.normal(g, len(lens), heads, 512) * size, R.normal(g, len(lens), heads, 64)
    ref, tol = R.decode(ql, qr, pool, 1)
    d, q, tables, ctx = pool.device(), (ql.cuda(), qr.cuda()), pool.tables.cuda(), i32(lens)
    first = None
    for _ in range(30):
        out = torch.full((len(lens), heads, 512), R.NAN, device="cuda")
        ws = P.latent_attention_decode(out, *q, block_tables=tables, context_lens=ctx, scale=R.SCALE, **d)
        if first is None:
            first = out
            R.assert_within(out, ref, tol, "one tile a sequence")
        assert torch.equal(out, first)
        assert status_of(ws) == 0


# ---- weights far below the largest ---------------------------------------------------------

def _peaked(seed, n, heads, weight, where, common, tail, k=1):
    """A sequence of n tokens of which key `where` has about `weight` of every head's softmax, and the others: "spread"
    (scores half a unit apart), "equal" (one row many times: every weight rounds the same way) or "ramp" (scores that fall by 12).  `common`:
    the size of a vector that all latents share.  Returns (pool, q_latent, q_rope) of k query rows."""
    pool = R.Pool(seed, [n], True, spare=0)
    g = R.gen(seed + 1)
    latent = torch.randn(n, 512, generator=g) + common * torch.randn(512, generator=g)
    rope = R.normal(g, n, 64)
    ql, qr = R.normal(g, k, heads, 512, scale=0.25), R.normal(g, k, heads, 64, scale=0.25)
    qr[..., 0] = qr[..., 1] = 8.0
    if tail == "equal":
        latent[:], rope[:] = latent[(where + 1) % n], rope[(where + 1) % n]
        latent[where] = torch.randn(512, generator=g)
    rope[:, 0], rope[:, 1] = 0, torch.linspace(0, -12 / (8 * R.SCALE), n) if tail == "ramp" else 0
    codes, scale = R.quantise(latent.bfloat16())
    rows = torch.cat([codes.double() * scale.double()[:, None], rope.double()], 1)
    score = (torch.cat([ql, qr], -1).double().reshape(-1, 576) @ rows.T) * R.SCALE
    others = torch.cat([score[:, :where], score[:, where + 1:]], 1).logsumexp(1)
    boost = (others - score[:, where]).mean() + torch.logit(torch.tensor(weight, dtype=torch.float64))
    rope[where, 0] = boost / (8 * R.SCALE)
    rows[where, 512] = rope[where, 0].double()
    slots = (pool.tables[0].long()[:, None] * 16 + torch.arange(16)).flatten()[:n]
    for whole, part in ((pool.cache.view(-1, 512), codes.view(torch.uint8)), (pool.rope_cache.view(-1, 64), rope),
                        (pool.cache_scale.view(-1), scale), (pool.rows, rows)):
        whole[slots] = part
    return pool, ql, qr


def _reference(pool, ql, qr):
    """(out, tolerance, weights) of the k rows of one sequence.  A weight is rounded to fp16 (2^-11) and held as three E5M2
    codes, each off by 2^-3 of what it rounds (2^-9), or by half of the smallest step, 2^-17, where the reference, at most
    the largest weight, is 2^9; the exponential 2^-12; the query as a pair of E4M3 codes and scores over 576 products in
    32 bits; sums over n keys in 32 bits (each addition 2^-23, three products a key and 32 keys an addition)."""
    n, (k, heads, _) = pool.lens[0], ql.shape
    keys, q = pool.sequence(0), torch.cat([ql, qr], -1).double()
    slots = (pool.tables[0].long()[:, None] * 16 + torch.arange(16)).flatten()[:n]
    scale = pool.cache_scale.view(-1)[slots].double()
    codes = pool.cache.view(-1, 512)[slots].view(torch.float8_e4m3fn).double().abs()
    out, tol, weights = [], [], []
    for i in range(k):
        seen = n - k + 1 + i
        c = keys[:seen]
        w = torch.softmax((q[i] @ c.T) * R.SCALE, -1)
        score = R.SCALE * (576 * 2.0 ** -24 * (q[i].abs() @ c.abs().T).amax(-1) +
                           2.0 ** -10 / 224 * q[i][:, :512].abs().amax(-1) * c[:, :512].abs().sum(-1).max())
        rel = 2.0 ** -11 + 2.0 ** -9 + 2 * 2.0 ** -12 + 2 * score + (seen / 8 + 3 * seen / 32) * 2.0 ** -23
        out.append(w @ c[:, :512])
        tol.append((w @ c[:, :512].abs()) * rel[:, None] * 1.01 +
                   (w * scale[:seen]).amax(-1)[:, None] * 2.0 ** -26 * 1.01 * codes[:seen].sum(0))
        weights.append(w)
    return torch.stack(out), torch.stack(tol), weights


def _run_shared(pool, ql, qr, seqs=None):
    """The sequence many times over the same pages, as often as the GPU has ranges (every one lies in a range, whole)."""
    (k, heads, _), n = ql.shape, pool.lens[0]
    if seqs is None:
        tiles = -(-heads * k // 64)
        seqs = torch.cuda.get_device_properties(0).multi_processor_count // tiles
    out = torch.full((seqs * k, heads, 512), R.NAN, device="cuda")
    ws = P.latent_attention_decode(out, ql.cuda().repeat(seqs, 1, 1), qr.cuda().repeat(seqs, 1, 1), q_per_seq=k,
                                   block_tables=pool.tables.cuda().repeat(seqs, 1), context_lens=i32([n] * seqs),
                                   scale=R.SCALE, **pool.device())
    assert status_of(ws) == 0
    return out.view(seqs, k, heads, 512)


def _check_peaked(n, heads, weight, where, common, tail, k=1, seqs=None):
    pool, ql, qr = _peaked(n + heads, n, heads, weight, where, common, tail, k)
    ref, tol, w = _reference(pool, ql, qr)
    got = torch.stack([x[:, where] for x in w])
    assert 0.4 * weight < got.mean() < min(1.0, 1.5 * weight)  # (the case is what it says)
    out = _run_shared(pool, ql, qr, seqs)
    seqs = out.shape[0]
    for b in {0, seqs // 2, seqs - 1}:
        err = (out[b].cpu().double() - ref).norm(dim=-1) / ref.norm(dim=-1)
        assert err.max() < 1e-2 and err.mean() < 3e-3, (b, err.max(), err.mean())
        R.assert_within(out[b], ref, tol, f"sequence {b}")


@pytest.mark.parametrize("heads", [16, 32, 64])
@pytest.mark.parametrize("common", [0.0, 0.5])
@pytest.mark.parametrize("tail", ["spread", "equal", "ramp"])
@pytest.mark.parametrize("weight,where", [(0.3, 0), (0.6, 2001), (0.9, 3999), (0.6, 0)])
def test_one_key_has_most_of_the_weight(weight, where, tail, common, heads):
    _check_peaked(4000, heads, weight, where, common, tail)


@pytest.mark.parametrize("tail", ["spread", "equal"])
@pytest.mark.parametrize("weight,where", [(0.3, 0), (0.6, 7000), (0.9, 13999)])
@pytest.mark.parametrize("heads,k", [(32, 1), (64, 1), (64, 4)])
def test_one_key_has_most_of_the_weight_of_a_long_range(heads, k, weight, where, tail):
    _check_peaked(14000, heads, weight, min(where, 14000 - k), 0.5, tail, k)


@pytest.mark.parametrize("tail", ["spread", "equal", "ramp"])
@pytest.mark.parametrize("seqs", [1, 5])
def test_one_key_has_most_of_the_weight_of_a_split_sequence(seqs, tail):
    for weight, where in ((0.3, 0), (0.9, 20000)):
        _check_peaked(32000, 64, weight, where, 0.5, tail, seqs=seqs)


# ---- scales at their least ------------------------------------------------------------------

def _with_rows(seed, n, latent):
    """A sequence of n tokens with these latents."""
    pool = R.Pool(seed, [n], True, spare=0)
    slots = (pool.tables[0].long()[:, None] * 16 + torch.arange(16)).flatten()[:n]
    codes, scale = R.quantise(latent)
    pool.cache.view(-1, 512)[slots], pool.cache_scale.view(-1)[slots] = codes.view(torch.uint8), scale
    pool.rows[slots, :512] = codes.double() * scale.double()[:, None]
    return pool


@pytest.mark.parametrize("heads", [16, 64])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -10])
@pytest.mark.parametrize("n,seqs,live", [(3000, None, [0]), (3000, 2, [1500, 2000]), (3000, None, []), (40000, None, [39999]),
                                         (120000, 1, [119000]), (120000, 1, [])])
def test_rows_of_zeros_keep_their_weight(n, seqs, live, size, heads):
    """Tokens whose latents are zeros, written with the least scale there is, but for a few: the zeros weigh as much as the
    others in the sum, and thousands of them of equal weight (small queries) do not make it infinite."""
    latent = torch.zeros(n, 512, dtype=torch.bfloat16)
    latent[live] = R.normal(R.gen(heads), len(live), 512)
    pool = _with_rows(heads + 1, n, latent)
    g = R.gen(heads + 2)
    ql, qr = R.normal(g, 1, heads, 512, scale=size), R.normal(g, 1, heads, 64, scale=size)
    ref, tol, _ = _reference(pool, ql, qr)
    out = _run_shared(pool, ql, qr, seqs)
    R.assert_within(out[0], ref, tol, "zeros")
    R.assert_within(out[-1], ref, tol, "zeros")


@pytest.mark.parametrize("heads", [16, 32, 64])
@pytest.mark.parametrize("cleared", [[5], [0, 1, 2, 64, 130], range(300)])
def test_scales_of_zero(cleared, heads):
    """Tokens with a scale of 0 are c = 0 whatever their codes, as the read-back has them; among others, and a pool that
    was cleared and never written."""
    n = 300
    pool = _with_rows(heads, n, R.normal(R.gen(heads + 1), n, 512))
    slots = (pool.tables[0].long()[:, None] * 16 + torch.arange(16)).flatten()[:n][list(cleared)]
    pool.cache_scale.view(-1)[slots], pool.rows[slots, :512] = 0.0, 0.0
    if len(cleared) == n:
        pool.cache.zero_()
    g = R.gen(heads + 2)
    ql, qr = R.normal(g, 1, heads, 512), R.normal(g, 1, heads, 64)
    ref, tol, _ = _reference(pool, ql, qr)
    for seqs in (1, None):
        out = _run_shared(pool, ql, qr, seqs)
        R.assert_within(out[0], ref, tol, "cleared scales")
        R.assert_within(out[-1], ref, tol, "cleared scales")
    rows = torch.empty(n, 576, dtype=torch.bfloat16, device="cuda")
    P.latent_gather(rows, block_tables=pool.tables.cuda(), cu_lens=i32([0, n]), **pool.device())
    assert (rows[list(cleared), :512] == 0).all()


def test_a_scale_that_is_not_finite_spoils_its_sequence():
    pool = _with_rows(1, 200, R.normal(R.gen(2), 200, 512))
    q = R.normal(R.gen(3), 1, 16, 512), R.normal(R.gen(4), 1, 16, 64)
    pool.cache_scale.view(-1)[int(pool.tables[0, 1]) * 16 + 3] = R.NAN
    assert _run_shared(pool, *q, 1).isnan().all()


@pytest.mark.parametrize("heads", [8, 64])
@pytest.mark.parametrize("n", [40, 130, 9000])
def test_a_scale_that_is_not_finite_never_makes_zeros(n, heads):
    """The last key's scale is NaN: its own row is NaN, and the row before it, which does not see the key, is either right or NaN."""
    pool = _with_rows(n, n, R.normal(R.gen(n + 1), n, 512))
    g = R.gen(n + 2)
    ql, qr = R.normal(g, 2, heads, 512), R.normal(g, 2, heads, 64)
    ref, tol, _ = _reference(pool, ql, qr)
    pool.cache_scale.view(-1)[int(pool.tables[0, (n - 1) // 16]) * 16 + (n - 1) % 16] = R.NAN
    out = _run_shared(pool, ql, qr, 1)[0].cpu()
    assert out[1].isnan().all()
    if not out[0].isnan().all():
        R.assert_within(out[0], ref[0], tol[0], "the row before")
