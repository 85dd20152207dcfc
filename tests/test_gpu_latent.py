"""Latent-attention operators on the GPU against their plain 64-bit forms."""
import pytest
import torch

import latent_reference as R
from paged_kv_cache_95_gb300 import pagedkv as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(built_library):
    P.load_library()


def status_of(ws):
    return int(ws[:4].view(torch.int32).cpu().item()) & 0xFFFFFFFF


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def starts(lens):
    return [0] + torch.tensor(lens).cumsum(0).tolist()


def bits(t):
    return t.contiguous().view(torch.uint8 if t.element_size() == 1 else torch.int16 if t.element_size() == 2
                               else torch.int32)


# ---- cache write ----------------------------------------------------------------------

def _slots(tokens, total, g):
    slots = torch.randperm(total, generator=g)[:tokens].int()
    if tokens > 4:
        slots[1], slots[tokens // 2] = -1, total  # padding, and one past the pool
    return slots


def _write_inputs(tokens, layout, g):
    if layout == "packed":
        return R.normal(g, tokens, 512), R.normal(g, tokens, 64)
    if layout == "sliced":
        x = R.normal(g, tokens, 576)
        return x[:, :512], x[:, 512:]
    x = R.normal(g, tokens, 1664)  # latent and rope inside wider rows, in the other order
    return x[:, 1032:1544], x[:, 64:128]


def _to_gpu(t):
    """The same values, strides and storage layout on the GPU."""
    base = t._base if t._base is not None else t
    g = base.cuda()
    return g.as_strided(t.shape, t.stride(), t.storage_offset())


@pytest.mark.parametrize("layout", ["packed", "sliced", "wide"])
@pytest.mark.parametrize("tokens", [1, 5, 33, 1000])
def test_write_is_bit_exact(tokens, layout):
    g = R.gen(tokens)
    blocks = tokens // 16 + 3
    latent, rope = _write_inputs(tokens, layout, g)
    cache = R.normal(g, blocks, 16, 576)
    slots = _slots(tokens, blocks * 16, g)
    got = cache.cuda()
    P.latent_reshape_and_cache(_to_gpu(latent), _to_gpu(rope), got, slots.cuda())
    want = cache.view(-1, 576).clone()
    ok = (slots >= 0) & (slots < blocks * 16)
    want[slots[ok].long()] = torch.cat([latent, rope], 1)[ok]
    assert torch.equal(bits(got).cpu().view(-1, 576), bits(want))


@pytest.mark.parametrize("layout", ["packed", "sliced", "wide"])
@pytest.mark.parametrize("tokens", [1, 7, 600])
def test_write_fp8_is_reproducible(tokens, layout):
    g = R.gen(tokens + 9)
    blocks = tokens // 16 + 3
    latent, rope = _write_inputs(tokens, layout, g)
    if tokens > 6:  # rows of extremes: zeros, tiny, huge, one large value, exact multiples of 448
        latent[0] = 0
        latent[2] = latent[2] * 1e-30
        latent[3] = latent[3] * 1e30
        latent[4, 1:] = 2.0 ** -9
        latent[4, 0] = -448
        latent[5] = latent[5].sign() * 448
    codes, scale = R.quantise(R.normal(g, blocks * 16, 512))
    ropes = R.normal(g, blocks * 16, 64)
    slots = _slots(tokens, blocks * 16, g)
    dev = [codes.view(torch.uint8).view(blocks, 16, 512).cuda(), ropes.view(blocks, 16, 64).cuda(),
           scale.view(blocks, 16).cuda()]
    P.latent_reshape_and_cache_fp8(_to_gpu(latent), _to_gpu(rope), *dev, slots.cuda())
    ok = (slots >= 0) & (slots < blocks * 16)
    at = slots[ok].long()
    new_codes, new_scale = R.quantise(latent[ok])
    codes = codes.view(torch.uint8).clone()
    codes[at], ropes[at], scale[at] = new_codes.view(torch.uint8), rope[ok], new_scale
    assert torch.equal(dev[0].cpu().view(-1, 512), codes)
    assert torch.equal(bits(dev[1]).cpu().view(-1, 64), bits(ropes))
    assert torch.equal(bits(dev[2]).cpu().view(-1), bits(scale))


# ---- read-back ---------------------------------------------------------------------------

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens", [[1], [16], [17, 0, 5], [0, 0, 3], [130, 1, 16, 0, 77], [3] * 70])
def test_gather(lens, fp8):
    pool = R.Pool(len(lens) + sum(lens), lens, fp8)
    total, extra = sum(lens), 5
    out = torch.full((total + extra, 576), 3.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    P.latent_gather(out, block_tables=pool.tables.cuda(), cu_lens=i32(starts(lens)), status=status, **pool.device())
    rows = torch.cat([pool.sequence(b) for b in range(len(lens))])
    # the product code * scale in fp32 (exact codes, one rounding), then bf16
    want = rows.float().bfloat16()
    if fp8:
        slots = torch.cat([(pool.tables[b].long()[:, None] * 16 + torch.arange(16)).flatten()[:n]
                           for b, n in enumerate(lens)])
        codes = pool.cache.view(-1, 512)[slots].view(torch.float8_e4m3fn).float()
        want[:, :512] = (codes * pool.cache_scale.view(-1)[slots][:, None]).bfloat16()
    assert torch.equal(bits(out[:total]).cpu(), bits(want))
    assert (out[total:] == 3.0).all()  # rows behind the last sequence
    assert status.item() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("count", [32, 33, 1025, 2100])
def test_gather_many_sequences(count, fp8):
    """More than 32 and 1024 lengths to search, empty sequences among them, first and last."""
    test_gather([(i * 7) % 4 for i in range(count - 1)] + [0], fp8)


@pytest.mark.parametrize("fp8", [False, True])
def test_gather_bad_blocks_and_lengths(fp8):
    pool = R.Pool(3, [40, 20], fp8, table_pad=0)
    pool.tables[0, 1] = pool.num_blocks
    pool.tables[1, 0] = -1
    cu = i32([0, 40, 40 + 16 * pool.max_blocks + 9])  # the second sequence passes its table
    out = torch.full((int(cu[-1]), 576), 3.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    P.latent_gather(out, block_tables=pool.tables.cuda(), cu_lens=cu, status=status, **pool.device())
    o = out.cpu().double()
    assert (o[16:32] == 0).all() and (o[40:56] == 0).all() and (o[40 + 16 * pool.max_blocks:] == 0).all()
    assert torch.isfinite(o[:16]).all() and (o[:16] != 0).any() and (o[56:60] != 0).any()
    assert status.item() == P.PKV_STATUS_BAD_BLOCK_ID | P.PKV_STATUS_BAD_CONTEXT_LEN


# ---- absorbed attention --------------------------------------------------------------------

def run_decode(pool, q_latent, q_rope, q_per_seq, dtype=torch.float32, lens=None, workspace=None):
    out = torch.full((*q_latent.shape[:2], 512), R.NAN, dtype=dtype, device="cuda")
    ws = P.latent_attention_decode(out, _to_gpu(q_latent), _to_gpu(q_rope), block_tables=pool.tables.cuda(),
                                   context_lens=i32(pool.lens if lens is None else lens), scale=R.SCALE,
                                   q_per_seq=q_per_seq, workspace=workspace, **pool.device())
    return out, ws


def queries(seed, rows, heads, scale=1.0):
    g = R.gen(seed)
    return R.normal(g, rows, heads, 512, scale=scale), R.normal(g, rows, heads, 64, scale=scale)


LENS = {
    "one": [1],
    "edges": [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129],
    "ragged": [700, 3, 129, 64, 1000],
    "long": [9000],
    "many": [1 + (i * 37) % 90 for i in range(200)],
}


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("heads", [1, 16, 24, 64, 128])
def test_decode(heads, lens, fp8):
    pool = R.Pool(heads, LENS[lens], fp8)
    q = queries(heads + 1, len(pool.lens), heads)
    out, ws = run_decode(pool, *q, 1)
    ref, tol = R.decode(*q, pool, 1)
    R.assert_within(out, ref, tol, f"heads {heads}, {lens}")
    assert status_of(ws) == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,k", [(1, 2), (1, 16), (5, 3), (16, 4), (20, 7), (64, 2), (128, 3)])
def test_verify(heads, k, fp8):
    pool = R.Pool(heads * k, [k, k + 1, 63 + k, 64, 65, 200, 700], fp8)
    q = queries(heads + k, len(pool.lens) * k, heads)
    out, ws = run_decode(pool, *q, k)
    ref, tol = R.decode(*q, pool, k)
    R.assert_within(out, ref, tol, f"heads {heads}, {k} rows")
    assert status_of(ws) == 0


@pytest.mark.parametrize("lens", [[64], [500, 300], [4000]])
def test_decode_fp8_error_in_norm(lens):
    """The elementwise bound adds every weight's worst step; the steps are independent, so in norm the
    result is off by about one bf16 rounding of the weights (2^-8 / sqrt 3 of it and less): 4e-3 is
    twice what the three roundings together come to."""
    pool = R.Pool(3, lens, True)
    q = queries(4, len(lens), 64)
    out, _ = run_decode(pool, *q, 1)
    ref, _ = R.decode(*q, pool, 1)
    err = (out.cpu().double() - ref).norm(dim=-1) / ref.norm(dim=-1)
    assert err.max() < 8e-3 and err.mean() < 4e-3, (err.max(), err.mean())


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_bf16_output(fp8):
    pool = R.Pool(4, [300, 17, 1], fp8)
    q = queries(5, 3, 40)
    out, _ = run_decode(pool, *q, 1, dtype=torch.bfloat16)
    R.assert_within(out, *R.decode(*q, pool, 1), "bf16 output")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("scale", [1e-3, 12.0])
def test_decode_flat_and_sharp_scores(scale, fp8):
    """Scores near zero (all weights alike) and far apart (the reference raised in mid-sequence)."""
    pool = R.Pool(8, [900, 65, 130], fp8)
    q = queries(9, 3, 16, scale=scale)
    out, _ = run_decode(pool, *q, 1)
    R.assert_within(out, *R.decode(*q, pool, 1), f"q scaled by {scale}")


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_zero_query_is_the_mean(fp8):
    pool = R.Pool(10, [77, 640], fp8)
    q = [torch.zeros(2, 16, 512, dtype=torch.bfloat16), torch.zeros(2, 16, 64, dtype=torch.bfloat16)]
    out, _ = run_decode(pool, *q, 1)
    R.assert_within(out, *R.decode(*q, pool, 1), "zero query")


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_latents_of_uneven_sizes(fp8):
    """Tokens whose latents differ by powers of ten (an FP8 pool's scales with them)."""
    pool = R.Pool(12, [200], fp8)
    g = R.gen(13)
    size = 10.0 ** (torch.rand(pool.num_blocks * 16, generator=g) * 4 - 3)
    if fp8:
        pool.cache_scale = (pool.cache_scale.view(-1) * size).view_as(pool.cache_scale)
        pool.rows[:, :512] = (pool.cache.view(-1, 512).view(torch.float8_e4m3fn).double() *
                              pool.cache_scale.view(-1)[:, None].double())
    else:
        latent = (pool.cache.view(-1, 576)[:, :512].float() * size[:, None]).bfloat16()
        pool.cache.view(-1, 576)[:, :512] = latent
        pool.rows[:, :512] = latent.double()
    q = queries(14, 1, 32)
    out, _ = run_decode(pool, *q, 1)
    R.assert_within(out, *R.decode(*q, pool, 1), "uneven latents")


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_strided_queries(fp8):
    pool = R.Pool(15, [40, 100, 7], fp8)
    g = R.gen(16)
    ql = R.normal(g, 24, 3, 512).transpose(0, 1)              # [heads][rows][512]
    qr = R.normal(g, 3, 24, 192)[..., 128:]                   # the rotated part of whole heads
    out, _ = run_decode(pool, ql, qr, 1)
    R.assert_within(out, *R.decode(ql, qr, pool, 1), "strided q")


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_bad_lengths_and_blocks(fp8):
    pool = R.Pool(17, [100, 40, 70, 33, 300], fp8, table_pad=0)
    k = 2
    q = queries(18, 5 * k, 16)
    pool.tables[0, 2] = pool.num_blocks + 5
    pool.tables[1, :] = -3   # a sequence of which nothing is left
    pool.tables[4, 0:9] = 1 << 30
    lens = list(pool.lens)
    lens[2], lens[3] = 0, 1  # empty, and shorter than its rows
    skip = [(0, 2), (1, 0), (1, 1), (1, 2)] + [(4, i) for i in range(9)]
    out, ws = run_decode(pool, *q, k, lens=lens)
    pool.lens = lens
    ref, tol = R.decode(*q, pool, k, skip)
    R.assert_within(out, ref, tol, "bad blocks")
    assert (out[2:8] == 0).all()
    assert status_of(ws) == P.PKV_STATUS_BAD_BLOCK_ID | P.PKV_STATUS_BAD_CONTEXT_LEN | P.PKV_STATUS_BAD_Q_LEN


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_length_past_the_table(fp8):
    pool = R.Pool(19, [48, 30], fp8, table_pad=0)
    q = queries(20, 2, 16)
    out, ws = run_decode(pool, *q, 1, lens=[48 + 1000, 30])  # counts as the table's 48
    R.assert_within(out, *R.decode(*q, pool, 1), "long length")
    assert status_of(ws) == P.PKV_STATUS_BAD_CONTEXT_LEN


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_padded_batch(fp8):
    """Empty sequences between, before and behind others."""
    lens = [0, 0, 200, 0, 1, 0, 65, 0]
    pool = R.Pool(21, lens, fp8)
    q = queries(22, len(lens), 32)
    out, ws = run_decode(pool, *q, 1)
    R.assert_within(out, *R.decode(*q, pool, 1), "padded batch")
    assert status_of(ws) == P.PKV_STATUS_BAD_CONTEXT_LEN
    out, _ = run_decode(pool, *q, 1, lens=[0] * len(lens))
    assert (out == 0).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_repeats_bitwise_and_shares_a_workspace(fp8):
    """One workspace serves calls of other sizes in between; the same call gives the same bits."""
    a, b = R.Pool(23, [900, 20, 333], fp8), R.Pool(24, [64] * 20, fp8)
    qa, qb = queries(25, 3, 64), queries(26, 40, 8)
    desc = P.latent_cache_desc(a.device()["cache"])
    size = max(P.latent_attention_workspace_size(3, 1, 64, a.max_blocks, desc),
               P.latent_attention_workspace_size(20, 2, 8, b.max_blocks, desc))
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    first, _ = run_decode(a, *qa, 1, workspace=ws)
    other, _ = run_decode(b, *qb, 2, workspace=ws)
    again, _ = run_decode(a, *qa, 1, workspace=ws)
    assert torch.equal(first, again)
    R.assert_within(other, *R.decode(*qb, b, 2), "between")
    assert status_of(ws) == 0


def _decode_call(pool, q, dtype=torch.float32):
    """A prepared call: (function, out)."""
    d = pool.device()
    out = torch.full((*q[0].shape[:2], 512), R.NAN, dtype=dtype, device="cuda")
    tables, lens, ql, qr = pool.tables.cuda(), i32(pool.lens), q[0].cuda(), q[1].cuda()
    ws = torch.zeros(P.latent_attention_workspace_size(len(pool.lens), 1, q[0].shape[1], pool.max_blocks,
                                                       P.latent_cache_desc(d["cache"])), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    return (lambda: P.latent_attention_decode(out, ql, qr, block_tables=tables, context_lens=lens, scale=R.SCALE,
                                              workspace=ws, **d)), out


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_on_two_streams_and_in_a_graph(fp8):
    pools = [R.Pool(27 + i, [500, 77, 260], fp8) for i in range(2)]
    qs = [queries(30 + i, 3, 32) for i in range(2)]
    calls = [_decode_call(p, q) for p, q in zip(pools, qs)]
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        for (call, _), s in zip(calls, streams):
            with torch.cuda.stream(s):
                call()
    torch.cuda.synchronize()
    refs = [R.decode(*q, p, 1) for p, q in zip(pools, qs)]
    for (_, out), ref in zip(calls, refs):
        R.assert_within(out, *ref, "two streams")
    want = [out.clone() for _, out in calls]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for call, _ in calls:
            call()
    for _, out in calls:
        out.fill_(R.NAN)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for (_, out), w in zip(calls, want):
        assert torch.equal(out, w)


@pytest.mark.parametrize("fp8", [False, True])
def test_offsets_past_32_bits(fp8):
    """A pool above 4 GiB whose sequences lie in its last blocks."""
    small = R.Pool(33, [130, 40], fp8)
    row = 512 if fp8 else 1152
    blocks = (1 << 32) // (row * 16) + 64
    lo = blocks - small.num_blocks
    d = small.device()
    big = torch.zeros(blocks, 16, d["cache"].shape[2], dtype=d["cache"].dtype, device="cuda")
    big[lo:] = d["cache"]
    args = dict(cache=big)
    if fp8:
        args["rope_cache"] = torch.zeros(blocks, 16, 64, dtype=torch.bfloat16, device="cuda")
        args["cache_scale"] = torch.zeros(blocks, 16, device="cuda")
        args["rope_cache"][lo:], args["cache_scale"][lo:] = d["rope_cache"], d["cache_scale"]
    tables = (small.tables + lo).cuda()
    q = queries(34, 2, 16)
    out = torch.empty(2, 16, 512, device="cuda")
    P.latent_attention_decode(out, q[0].cuda(), q[1].cuda(), block_tables=tables, context_lens=i32(small.lens),
                              scale=R.SCALE, **args)
    R.assert_within(out, *R.decode(*q, small, 1), "high blocks")
    rows = torch.empty(170, 576, dtype=torch.bfloat16, device="cuda")
    P.latent_gather(rows, block_tables=tables, cu_lens=i32([0, 130, 170]), **args)
    near = torch.empty_like(rows)
    P.latent_gather(near, block_tables=small.tables.cuda(), cu_lens=i32([0, 130, 170]), **d)
    assert torch.equal(bits(rows), bits(near))
    slot = (blocks - 1) * 16 + 15
    latent, rope = R.normal(R.gen(35), 1, 512), R.normal(R.gen(36), 1, 64)
    if fp8:
        P.latent_reshape_and_cache_fp8(latent.cuda(), rope.cuda(), **args, slot_mapping=i32([slot]))
        assert torch.equal(big[-1, -1].cpu(), R.quantise(latent)[0].view(torch.uint8)[0])
    else:
        P.latent_reshape_and_cache(latent.cuda(), rope.cuda(), big, i32([slot]))
        assert torch.equal(bits(big[-1, -1]).cpu(), bits(torch.cat([latent, rope], 1)[0]))


# ---- expanded attention -----------------------------------------------------------------------

def prefill_inputs(seed, q_lens, k_lens, heads, spare=4, scale=1.0):
    """Keys and values as halves of one product, rotated keys inside read-back rows; spare rows hold NaN."""
    g = R.gen(seed)
    tq, tk = sum(q_lens), sum(k_lens)
    q = R.normal(g, tq + spare, heads, 192, scale=scale)
    kv = R.normal(g, tk + spare, heads, 256)
    rows = R.normal(g, tk + spare, 576)
    q[tq:], kv[tk:], rows[tk:] = R.NAN, R.NAN, R.NAN
    return q, kv, rows


def run_prefill(q, kv, rows, q_lens, k_lens, dtype=torch.float32, max_q=None):
    out = torch.full((q.shape[0], q.shape[1], 128), 5.0, dtype=dtype, device="cuda")
    kvd = kv.cuda()
    ws = P.latent_attention_prefill_chunk(out, _to_gpu(q), kvd[..., :128], kvd[..., 128:], rows.cuda()[:, 512:],
                                          i32(starts(q_lens)), i32(starts(k_lens)),
                                          max(q_lens) if max_q is None else max_q, R.SCALE)
    return out, ws


def check_prefill(q, kv, rows, q_lens, k_lens, **kw):
    out, ws = run_prefill(q, kv, rows, q_lens, k_lens, **kw)
    tq = sum(q_lens)
    ref, tol = R.expanded(q[:tq], kv[..., :128], kv[..., 128:], rows[:, 512:], q_lens, k_lens)
    R.assert_within(out[:tq], ref, tol, f"q {q_lens}, k {k_lens}")
    assert (out[tq:] == 5.0).all()  # rows behind the last sequence
    assert status_of(ws) == 0


PREFILL = [
    ([1], [1]), ([1], [300]), ([5], [5]), ([64], [64]), ([127, 128, 129], [127, 128, 129]),
    ([3, 0, 130, 1], [3, 9, 400, 64]), ([255, 257], [256, 700]), ([700], [700]), ([33] * 9, [33 + 50 * i for i in range(9)]),
]


@pytest.mark.parametrize("heads", [1, 3, 8])
@pytest.mark.parametrize("q_lens,k_lens", PREFILL)
def test_prefill(q_lens, k_lens, heads):
    check_prefill(*prefill_inputs(heads + sum(k_lens), q_lens, k_lens, heads), q_lens, k_lens)


def test_prefill_bf16_output_and_loose_bound():
    q_lens, k_lens = [130, 20, 300], [200, 20, 301]
    check_prefill(*prefill_inputs(1, q_lens, k_lens, 4), q_lens, k_lens, dtype=torch.bfloat16, max_q=777)


@pytest.mark.parametrize("scale", [1e-3, 12.0])
def test_prefill_flat_and_sharp_scores(scale):
    q_lens, k_lens = [300, 70], [500, 70]
    check_prefill(*prefill_inputs(2, q_lens, k_lens, 2, scale=scale), q_lens, k_lens)


def test_prefill_many_sequences():
    q_lens = [1 + (i * 13) % 40 for i in range(90)]
    k_lens = [n + (i * 7) % 30 for i, n in enumerate(q_lens)]
    check_prefill(*prefill_inputs(3, q_lens, k_lens, 2), q_lens, k_lens)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("k_lens", [[1000, 897, 128, 140], [129, 256, 257, 1153], [385, 1, 4000, 512]])
def test_prefill_one_row_tile(k_lens, dtype):
    """Up to 128 rows over one, even and odd numbers of key tiles."""
    q_lens = [100, 1, 128, 7]
    check_prefill(*prefill_inputs(sum(k_lens), q_lens, k_lens, 3), q_lens, k_lens, dtype=dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("q_lens,k_lens", [
    ([100], [2500]), ([1], [9000]), ([300, 20], [2900, 1500]), ([128, 0, 129], [3000, 700, 4100]), ([700], [4000]),
    ([5, 260], [5, 6000]),
])
def test_prefill_keys_over_several_ctas(q_lens, k_lens, dtype):
    """Few rows over many keys: parts of the keys, joined; rows and tiles that see nothing of a part."""
    for heads in (1, 5):
        args = prefill_inputs(sum(k_lens) + heads, q_lens, k_lens, heads)
        assert P.latent_attention_prefill_workspace_size(len(q_lens), heads, max(q_lens), args[0].shape[0], args[1].shape[0]) > 256
        check_prefill(*args, q_lens, k_lens, dtype=dtype)


def test_prefill_parts_in_a_graph_share_a_workspace():
    """Two calls whose parts lie in one workspace, one behind the other, replayed: the same bits."""
    calls = []
    for i, (ql, kl, heads) in enumerate([(100, 3000, 4), (260, 1800, 2)]):
        q, kv, rows = prefill_inputs(90 + i, [ql], [kl], heads, spare=0)
        calls.append((dict(out=torch.full((ql, heads, 128), R.NAN, dtype=torch.bfloat16, device="cuda"), q=q.cuda(), kv=kv.cuda(),
                           rows=rows.cuda(), cq=i32([0, ql]), ck=i32([0, kl]), n=ql),
                      R.expanded(q, kv[..., :128], kv[..., 128:], rows[:, 512:], [ql], [kl])))
    ws = torch.zeros(max(P.latent_attention_prefill_workspace_size(1, d["out"].shape[1], d["n"], d["n"], d["kv"].shape[0])
                         for d, _ in calls), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()

    def run(d):
        P.latent_attention_prefill_chunk(d["out"], d["q"], d["kv"][..., :128], d["kv"][..., 128:], d["rows"][:, 512:], d["cq"],
                                         d["ck"], d["n"], R.SCALE, workspace=ws)

    for d, ref in calls:
        run(d)
        R.assert_within(d["out"], *ref, "parts")
    want = [d["out"].clone() for d, _ in calls]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for d, _ in calls:
            run(d)
    for d, _ in calls:
        d["out"].fill_(R.NAN)
    ws[256:] = 0xFF  # parts of an earlier call are not read
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for (d, _), w in zip(calls, want):
        assert torch.equal(bits(d["out"]), bits(w))
    assert status_of(ws) == 0


def test_prefill_split_bad_lengths_and_values():
    """With the keys in parts: a sequence with more queries than keys, one whose keys lie outside, a query and a key
    that are not finite, and a workspace that has room for the status word alone."""
    q_lens, k_lens = [20, 30, 150], [4000, 10, 4000]
    q, kv, rows = prefill_inputs(80, q_lens, k_lens, 2, spare=0)
    ref, tol = R.expanded(q, kv[..., :128], kv[..., 128:], rows[:, 512:], q_lens, k_lens)  # (of rows that see neither NaN)
    q[3, 1, 7], kv[3995, 0, 3] = R.NAN, R.NAN
    broken = torch.zeros(200, 2, dtype=torch.bool)
    broken[3, 1] = broken[15:20, 0] = True  # (key 3995 is row 15's own)
    for ws in (None, torch.zeros(256, dtype=torch.uint8, device="cuda")):
        out = torch.full((200, 2, 128), 5.0, device="cuda")
        ws = P.latent_attention_prefill_chunk(out, q.cuda(), kv.cuda()[..., :128], kv.cuda()[..., 128:], rows.cuda()[:, 512:],
                                              i32(starts(q_lens)), i32(starts(k_lens)), 150, R.SCALE, workspace=ws)
        assert status_of(ws) == P.PKV_STATUS_BAD_Q_LEN
        o = out.cpu()
        assert o[broken].isnan().all() and (o[20:50] == 0).all()
        R.assert_within(o[~broken], ref[~broken], tol[~broken], "the others")
    out, ws = run_prefill(q, kv, rows, [20, 0, 180], [4000, 10, 4010])  # key rows past the tensor
    assert (out[20:] == 0).all() and status_of(ws) == P.PKV_STATUS_BAD_Q_LEN
    out, ws = run_prefill(q, kv, rows, [20, 30, 150], k_lens, max_q=100)  # a chunk longer than its bound
    assert (out[20:] == 0).all() and status_of(ws) == P.PKV_STATUS_BAD_Q_LEN


def test_prefill_strides():
    """Heads outermost, and packed keys and values of their own."""
    g = R.gen(4)
    q = R.normal(g, 3, 90, 192).transpose(0, 1)
    k, v = R.normal(g, 3, 140, 128).transpose(0, 1), R.normal(g, 3, 140, 128).transpose(0, 1)
    kr = R.normal(g, 140, 64)
    out = torch.empty(90, 3, 128, device="cuda")
    P.latent_attention_prefill_chunk(out, _to_gpu(q), _to_gpu(k), _to_gpu(v), kr.cuda(), i32([0, 90]), i32([0, 140]),
                                     90, R.SCALE)
    R.assert_within(out, *R.expanded(q, k, v, kr, [90], [140]), "strides")


def test_prefill_chunks_equal_the_whole():
    """A prompt in two chunks against the whole: the same rows within both tolerances."""
    q, kv, rows = prefill_inputs(5, [400], [400], 2, spare=0)
    whole, _ = run_prefill(q, kv, rows, [400], [400])
    head, _ = run_prefill(q[:150], kv[:150], rows[:150], [150], [150])
    tail, _ = run_prefill(q[150:], kv, rows, [250], [400])
    _, tol = R.expanded(q, kv[..., :128], kv[..., 128:], rows[:, 512:], [400], [400])
    R.assert_within(torch.cat([head, tail]), whole.cpu().double(), 2 * tol, "two chunks")


def test_prefill_bad_lengths():
    q, kv, rows = prefill_inputs(6, [20, 30, 10], [40, 10, 10], 2, spare=0)  # 30 queries over 10 keys
    out, ws = run_prefill(q, kv, rows, [20, 30, 10], [40, 10, 10])
    ref, tol = R.expanded(q, kv[..., :128], kv[..., 128:], rows[:, 512:], [20, 30, 10], [40, 10, 10])
    R.assert_within(out, ref, tol, "bad length")
    assert (out[20:50] == 0).all()
    assert status_of(ws) == P.PKV_STATUS_BAD_Q_LEN
    out, ws = run_prefill(q, kv, rows, [20, 0, 40], [40, 10, 90])  # key rows past the tensor
    assert (out[20:] == 0).all() and status_of(ws) == P.PKV_STATUS_BAD_Q_LEN


@pytest.mark.parametrize("factor", [0.0, -1.0])
def test_scales_of_zero_and_below(factor):
    """A scale of -s is a query of the other sign; a scale of 0 is the mean of what a row sees."""
    for fp8 in (False, True):
        pool = R.Pool(60, [900, 65, 3], fp8)
        q = queries(61, 3, 20)
        out = torch.empty(3, 20, 512, device="cuda")
        P.latent_attention_decode(out, q[0].cuda(), q[1].cuda(), block_tables=pool.tables.cuda(), context_lens=i32(pool.lens),
                                  scale=factor * R.SCALE, **pool.device())
        R.assert_within(out, *R.decode(*(x * factor for x in q), pool, 1), f"scale x {factor}")
    q, kv, rows = prefill_inputs(62, [150, 3], [300, 3], 3, spare=0)
    out = torch.empty(153, 3, 128, device="cuda")
    P.latent_attention_prefill_chunk(out, q.cuda(), kv.cuda()[..., :128], kv.cuda()[..., 128:], rows.cuda()[:, 512:],
                                     i32([0, 150, 153]), i32([0, 300, 303]), 150, factor * R.SCALE)
    R.assert_within(out, *R.expanded(q * factor, kv[..., :128], kv[..., 128:], rows[:, 512:], [150, 3], [300, 3]),
                    f"prefill, scale x {factor}")


@pytest.mark.parametrize("fp8", [False, True])
def test_more_columns_than_the_gpu_holds(fp8):
    """1024 heads x 3 rows are 48 column tiles; x 16 rows 256, more than there are SMs."""
    pool = R.Pool(63, [130, 20], fp8)
    for k in (3, 16):
        q = queries(64, 2 * k, 1024)
        out, ws = run_decode(pool, *q, k, dtype=torch.bfloat16)
        R.assert_within(out, *R.decode(*q, pool, k), f"{k} rows of 1024 heads")
        assert status_of(ws) == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_one_block_of_many_sequences(fp8):
    """Sequences that share their pages (a common prefix) and one that names a block twice."""
    pool = R.Pool(65, [320] * 6, fp8, table_pad=0)
    pool.tables[:] = pool.tables[0]
    pool.tables[3, 7] = pool.tables[3, 2]
    q = queries(66, 6, 32)
    out, _ = run_decode(pool, *q, 1)
    R.assert_within(out, *R.decode(*q, pool, 1), "shared blocks")


@pytest.mark.parametrize("fp8", [False, True])
def test_a_query_that_is_not_finite_stays_alone(fp8):
    pool = R.Pool(67, [200, 90], fp8)
    q = queries(68, 2, 24)
    want, _ = run_decode(pool, *q, 1)
    q[0][0, 5, 17], q[0][1, 7, 300], q[1][1, 2, 9] = float("inf"), R.NAN, R.NAN
    out, ws = run_decode(pool, *q, 1)
    broken = torch.zeros(2, 24, dtype=torch.bool)
    broken[0, 5] = broken[1, 7] = broken[1, 2] = True
    assert torch.equal(out.cpu()[~broken], want.cpu()[~broken])
    assert out.cpu()[broken].isnan().all()
    assert status_of(ws) == 0


def test_prefill_queries_and_keys_that_are_not_finite():
    """A query spoils its own row; a key only the rows that see it."""
    q, kv, rows = prefill_inputs(69, [300], [300], 2, spare=0)
    want, _ = run_prefill(q, kv, rows, [300], [300])
    q[7, 1, 40], kv[250, 0, 3] = R.NAN, R.NAN
    out, ws = run_prefill(q, kv, rows, [300], [300])
    broken = torch.zeros(300, 2, dtype=torch.bool)
    broken[7, 1] = broken[250:, 0] = True
    assert torch.equal(out.cpu()[~broken], want.cpu()[~broken])
    assert out.cpu()[broken].isnan().all()
    assert status_of(ws) == 0


def test_prefill_on_two_streams_and_in_a_graph():
    """Calls at once on two streams, then captured one behind the other over one workspace."""
    sizes = [([200, 65], [400, 65]), ([300], [301])]
    calls, refs = [], []
    for i, (ql, kl) in enumerate(sizes):
        q, kv, rows = prefill_inputs(70 + i, ql, kl, 3, spare=0)
        refs.append(R.expanded(q, kv[..., :128], kv[..., 128:], rows[:, 512:], ql, kl))
        d = dict(q=q.cuda(), kv=kv.cuda(), rows=rows.cuda(), cq=i32(starts(ql)), ck=i32(starts(kl)), n=max(ql),
                 out=torch.full((sum(ql), 3, 128), R.NAN, device="cuda"), ws=torch.zeros(256, dtype=torch.uint8, device="cuda"))
        calls.append(d)
    shared = torch.zeros(256, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()

    def run(d, ws):
        P.latent_attention_prefill_chunk(d["out"], d["q"], d["kv"][..., :128], d["kv"][..., 128:], d["rows"][:, 512:], d["cq"],
                                         d["ck"], d["n"], R.SCALE, workspace=ws)

    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(4):
        for d, s in zip(calls, streams):
            with torch.cuda.stream(s):
                run(d, d["ws"])
    torch.cuda.synchronize()
    want = [d["out"].clone() for d in calls]
    for w, ref in zip(want, refs):
        R.assert_within(w, *ref, "two streams")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for d in calls:
            run(d, shared)
    for d in calls:
        d["out"].fill_(R.NAN)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for d, w in zip(calls, want):
        assert torch.equal(d["out"], w)
    assert status_of(shared) == 0


# ---- refusals of the binding ------------------------------------------------------------------------

def test_binding_refusals():
    pool = R.Pool(40, [20])
    d, q = pool.device(), queries(41, 1, 16)
    out = torch.empty(1, 16, 512, device="cuda")
    good = dict(out=out, q_latent=q[0].cuda(), q_rope=q[1].cuda(), block_tables=pool.tables.cuda(),
                context_lens=i32([20]), scale=R.SCALE, **d)
    P.latent_attention_decode(**good)
    for bad in (dict(q_latent=q[0]), dict(q_latent=q[0].cuda().float()), dict(out=out.half()), dict(q_per_seq=2),
                dict(q_latent=q[0].cuda()[..., ::2]), dict(cache=d["cache"][:, :8]), dict(context_lens=i32([20, 3])),
                dict(cache_scale=torch.ones(3, 16, device="cuda")), dict(q_rope=q[1].cuda()[:, :8])):
        with pytest.raises((ValueError, P.PagedKVError)):
            P.latent_attention_decode(**{**good, **bad})


# ---- a run of them together ----------------------------------------------------------------------------

@pytest.mark.parametrize("fp8", [False, True])
def test_a_served_sequence(fp8):
    """Two prompts prefilled in chunks (write, read back, expand, attend), then decoded and
    verified over the pages, each against 64 bits on the same cached rows."""
    heads, blocks = 4, 40
    g = R.gen(50)
    wk, wv = (R.normal(g, heads, 128, 512, scale=512 ** -0.5) for _ in range(2))
    bm = P.BlockManager(blocks)
    pool = R.Pool(51, [1], fp8, spare=blocks - 1)
    d = pool.device()
    for t in d.values():
        t.view(torch.uint8).fill_(0xFF)  # every slot NaN until it is written
    write = P.latent_reshape_and_cache_fp8 if fp8 else P.latent_reshape_and_cache
    lens = {7: 0, 9: 0}
    for i in lens:
        bm.add(i)

    def append(counts):
        slots, pairs = bm.append_batch(list(counts), list(counts.values()))
        assert len(pairs) == 0
        x = R.normal(g, len(slots), 576).cuda()
        write(x[:, :512], x[:, 512:], **d, slot_mapping=torch.from_numpy(slots).cuda())
        for i, n in counts.items():
            lens[i] += n
        tables, ctx = bm.block_tables(list(counts), 16)
        return torch.from_numpy(tables).cuda(), torch.from_numpy(ctx).cuda()

    def cached(tables, ctx):
        cu = i32(starts(ctx.tolist()))
        rows = torch.empty(int(cu[-1]), 576, dtype=torch.bfloat16, device="cuda")
        P.latent_gather(rows, block_tables=tables, cu_lens=cu, **d)
        return rows, cu

    for counts in ({7: 100, 9: 33}, {7: 29, 9: 64}):
        tables, ctx = append(counts)
        rows, cu_k = cached(tables, ctx)
        kv = torch.einsum("jc,hdc->jhd", rows[:, :512].float(), torch.cat([wk, wv], 1).cuda().float()).bfloat16()
        n = list(counts.values())
        q = R.normal(g, sum(n), heads, 192)
        out = torch.empty(sum(n), heads, 128, device="cuda")
        P.latent_attention_prefill_chunk(out, q.cuda(), kv[..., :128], kv[..., 128:], rows[:, 512:], i32(starts(n)), cu_k,
                                         max(n), R.SCALE)
        kvc = kv.cpu()
        ref, tol = R.expanded(q, kvc[..., :128], kvc[..., 128:], rows.cpu()[:, 512:], n, ctx.tolist())
        R.assert_within(out, ref, tol, f"chunk {counts}")
    for k in (1, 1, 3):
        tables, ctx = append({7: k, 9: k})
        pool.lens, pool.tables = ctx.tolist(), tables.cpu()
        c = {name: t.cpu() for name, t in d.items()}
        if fp8:
            latent = c["cache"].view(torch.float8_e4m3fn).double() * c["cache_scale"].double()[..., None]
            pool.rows = torch.cat([latent, c["rope_cache"].double()], -1).view(-1, 576)
        else:
            pool.rows = c["cache"].double().view(-1, 576)
        q = queries(60 + k, 2 * k, heads)
        out = torch.empty(2 * k, heads, 512, device="cuda")
        P.latent_attention_decode(out, q[0].cuda(), q[1].cuda(), block_tables=tables, context_lens=ctx, scale=R.SCALE,
                                  q_per_seq=k, **d)
        R.assert_within(out, *R.decode(*q, pool, k), f"decode of {k}")
    bm.close()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("value", [R.NAN, float("inf")])
@pytest.mark.parametrize("q_len,k_len,keys", [(1, 129, [128]), (3, 131, [128]), (100, 400, range(128, 256)), (1, 200, range(128)),
                                              (40, 300, range(256)), (2, 2000, range(1920, 2000))])
def test_prefill_split_keys_that_are_not_finite(q_len, k_len, keys, value, dtype):
    """One row tile, whose even and odd key tiles are joined: keys that fill what one side sees, NaN or with scores of
    infinity, make every row that sees one NaN, as they do where nothing is split."""
    heads = 3
    q, kv, rows = prefill_inputs(k_len, [q_len], [k_len], heads, spare=0)
    q = q.abs() + 0.1  # (scores of an infinite key are +infinity, never NaN)
    keys = list(keys)
    kv[keys, 1, 5] = value
    out, ws = run_prefill(q, kv, rows, [q_len], [k_len], dtype=dtype)
    sees = torch.arange(q_len) + k_len - q_len >= keys[0]
    assert out[:, 1].cpu()[sees].isnan().all()
    assert torch.isfinite(out[:, 1].cpu()[~sees]).all() and torch.isfinite(out[:, [0, 2]]).all()
    assert status_of(ws) == 0


def _busy():
    """Work of a tenth of a second on the current stream."""
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_decode_allocates_its_workspace_on_the_stream_it_is_given(fp8, handle):
    """The current stream is busy: the call on another one neither waits for it nor loses its status to a clear there."""
    pool = R.Pool(95, [0, 700, 90], fp8)
    q = queries(96, 3, 16)
    d, ql, qr, tables, lens = pool.device(), q[0].cuda(), q[1].cuda(), pool.tables.cuda(), i32(pool.lens)
    out = torch.full((3, 16, 512), R.NAN, device="cuda")
    s = torch.cuda.Stream()
    run_decode(pool, *q, 1)  # (the kernels are loaded)
    _busy()
    ws = P.latent_attention_decode(out, ql, qr, block_tables=tables, context_lens=lens, scale=R.SCALE,
                                   stream=s.cuda_stream if handle else s, **d)
    s.synchronize()
    assert not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    R.assert_within(out, *R.decode(*q, pool, 1), "another stream")
    assert status_of(ws) == P.PKV_STATUS_BAD_CONTEXT_LEN  # (of the empty sequence)


def test_decode_on_the_default_stream_by_its_handle():
    pool = R.Pool(97, [0, 300])
    q = queries(98, 2, 16)
    d, ql, qr, tables, lens = pool.device(), q[0].cuda(), q[1].cuda(), pool.tables.cuda(), i32(pool.lens)
    out = torch.full((2, 16, 512), R.NAN, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        ws = P.latent_attention_decode(out, ql, qr, block_tables=tables, context_lens=lens, scale=R.SCALE, stream=0, **d)
    torch.cuda.synchronize()
    R.assert_within(out, *R.decode(*q, pool, 1), "default stream")
    assert status_of(ws) == P.PKV_STATUS_BAD_CONTEXT_LEN


def test_prefill_allocates_its_workspace_on_the_stream_it_is_given():
    q_lens, k_lens = [100, 5], [3000, 3]  # parts of the keys, and a sequence with more queries than keys
    q, kv, rows = prefill_inputs(99, q_lens, k_lens, 2, spare=0)
    ref, tol = R.expanded(q, kv[..., :128], kv[..., 128:], rows[:, 512:], q_lens, k_lens)
    qd, kvd, rowsd, cq, ck = q.cuda(), kv.cuda(), rows.cuda(), i32(starts(q_lens)), i32(starts(k_lens))
    out = torch.full((105, 2, 128), R.NAN, device="cuda")
    s = torch.cuda.Stream()
    run_prefill(q, kv, rows, q_lens, k_lens)  # (the kernels are loaded)
    _busy()
    ws = P.latent_attention_prefill_chunk(out, qd, kvd[..., :128], kvd[..., 128:], rowsd[:, 512:], cq, ck, 100, R.SCALE, stream=s)
    s.synchronize()
    assert not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    R.assert_within(out, ref, tol, "another stream")
    assert status_of(ws) == P.PKV_STATUS_BAD_Q_LEN


@pytest.mark.parametrize("size", [1.0, 100.0])
@pytest.mark.parametrize("low", [-1e6, -3e12, torch.finfo(torch.bfloat16).min, -float("inf")])
@pytest.mark.parametrize("q_len,k_len,first", [(1, 400, 130), (100, 600, 260), (300, 900, 300), (2, 4000, 3000)])
def test_prefill_first_keys_masked_by_low_scores(q_len, k_len, first, low, size):
    """The keys that a row sees first have a score of a large negative number or -infinity (a mask that the caller put into
    the rotated key): those behind them are weighed as if the first were not there."""
    q, kv, rows = prefill_inputs(k_len, [q_len], [k_len], 2, spare=0, scale=size)
    q[..., 128] = 1.0
    rows[:, 512] = 0
    rows[:first, 512] = low
    out, ws = run_prefill(q, kv, rows, [q_len], [k_len])
    R.assert_within(out, *R.expanded(q, kv[first:, :, :128], kv[first:, :, 128:], rows[first:, 512:], [q_len], [k_len - first]),
                    f"low {low}")
    assert status_of(ws) == 0
