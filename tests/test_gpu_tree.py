"""Attention of trees of drafted tokens over the paged cache, against 64 bits."""
import random

import pytest
import torch

import speculative_reference as R
from paged_kv_cache_95_gb300 import pagedkv as P

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
SCALE = 128.0 ** -0.5
POOLS = [False, True]


@pytest.fixture(scope="module", autouse=True)
def _lib(built_library):
    P.load_library()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def i64(bits):
    return torch.tensor(R.as_int64(bits), dtype=torch.int64, device="cuda")


def starts(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def status_of(ws):
    return int(ws[:4].view(torch.int32).cpu().item()) & 0xFFFFFFFF


class Problem:
    """Sequences of nodes[b] nodes behind ctx[b] - nodes[b] tokens; every slot that is no key is poisoned with NaN."""

    def __init__(self, nodes, ctx, heads, kv, fp8=False, seed=0, masks=None, scales=(0.01, 1.0), spare=3):
        rng = random.Random(seed)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.nodes, self.ctx, self.heads, self.kv, self.fp8 = nodes, ctx, heads, kv, fp8
        self.cu, self.most = starts(nodes), max(nodes)
        rows = self.cu[-1]
        need = [-(-c // 16) for c in ctx]
        self.blocks = sum(need) + spare
        ids = rng.sample(range(self.blocks), sum(need))
        self.tables, at = [], 0
        for n in need:
            self.tables.append(ids[at:at + n] + [-7] * (max(need) - n))  # entries past the context are never looked at
            at += n
        key = torch.zeros(self.blocks, 16, dtype=torch.bool)
        for table, c in zip(self.tables, ctx):
            for j in range(0, c, 16):
                key[table[j // 16], :min(16, c - j)] = True
        hole = ~key.cuda()[:, None, :, None]
        x = torch.randn(2, self.blocks, kv, 16, 128, generator=g, device="cuda")
        self.q = torch.randn(rows, heads, 128, generator=g, device="cuda").bfloat16()
        self.scales = {}
        if fp8:
            s = torch.rand(2, self.blocks, kv, 16, generator=g, device="cuda") * (scales[1] - scales[0]) + scales[0]
            codes = (x * 100).clamp(-448, 448).to(F8)
            self.kd, self.vd = (codes.float() * s[..., None]).double()
            s = s.masked_fill(hole[..., 0], float("nan"))
            codes = codes.view(torch.uint8).masked_fill(hole, 0x7F).view(F8)  # the code of NaN
            self.k, self.v = codes[0].clone(), codes[1].clone()
            self.scales = dict(k_scale=s[0].clone(), v_scale=s[1].clone())
            # scores of a few units whatever the codes' scales are
            self.scale = SCALE / (100 * scales[1])
        else:
            x = x.bfloat16()
            self.kd, self.vd = x.double()
            x = x.masked_fill(hole, float("nan"))
            self.k, self.v, self.scale = x[0].clone(), x[1].clone(), SCALE
        if masks is None:
            masks = [m for n in nodes for m in R.ancestors(R.random_tree(rng, n) if n else [])]
        self.masks = masks

    def call(self, dtype=torch.float32, workspace=None, extra=2, stream=None, scale=None, q=None, out=None):
        if out is None:
            out = torch.full((self.cu[-1] + extra, self.heads, 128), 7.0, dtype=dtype, device="cuda")
        q = self.q if q is None else q
        # rows behind the last sequence: queries of their own, outputs left as they were
        q = torch.cat([q, torch.full((extra, self.heads, 128), 3.0, device="cuda").bfloat16()])
        masks = i64(self.masks + [~0 & (1 << 64) - 1] * extra)
        ws = P.paged_attention_tree(out, q, masks, i32(self.cu), self.most, self.k, self.v, i32(self.tables), i32(self.ctx),
                                    self.scale if scale is None else scale, workspace=workspace, stream=stream, **self.scales)
        if extra:
            assert bool((out[self.cu[-1]:] == 7).all())
        return out[:self.cu[-1]], ws

    def want(self, scale=None):
        return R.tree_attention(self.q, self.masks, self.cu, self.kd, self.vd, self.tables, self.ctx,
                                self.scale if scale is None else scale)

    def bound(self, want, dtype=torch.float32, scale=None):
        """A score is a sum of 128 fp32 products: off by up to 128 x 2^-23 of sum |q k| (an accumulator that truncates); a
        weight by twice that, by 2^-15 for its two bf16 parts and 2^-21 for exp2; a weighted mean of values by the
        weights' error, twice (numerator, sum), times the largest value; and half a step of the output."""
        scale = abs(self.scale if scale is None else scale)
        live = torch.unique(torch.tensor([b for t, c in zip(self.tables, self.ctx) for b in t[:-(-c // 16)]]))
        most = self.q.double().norm(dim=-1).max().cpu() * self.kd[live.cuda()].norm(dim=-1).max().cpu()
        weight = 2 * float(most) * scale * 128 * 2.0 ** -23 + 2.0 ** -15 + 2.0 ** -21
        if self.fp8:
            weight += 2.0 ** -11  # weights times V scales are rounded to fp16 (half a step; the scales' products are far below)
        b = 2 * weight * float(self.vd[live.cuda()].abs().max())
        return b + (want.abs() * 2.0 ** -8 if dtype is torch.bfloat16 else want.abs() * 2.0 ** -22)

    def bound_of(self, want):
        """The bound of the lengths that test_what_only_the_device_sees starts from."""
        return Problem(self.nodes, [40, 100, 30], self.heads, self.kv, self.fp8, seed=1).bound(want)

    def check(self, dtype=torch.float32, **kw):
        got, ws = self.call(dtype, **kw)
        want = self.want(kw.get("scale"))
        off = (got.double().cpu() - want).abs()
        assert bool((off <= self.bound(want, dtype, kw.get("scale"))).all()), (float(off.max()), float(off.max() / self.bound(want).max()))
        assert status_of(ws) == 0
        return got, ws


@pytest.mark.parametrize("fp8", POOLS)
@pytest.mark.parametrize("nodes,ctx,heads,kv", [
    ([1], [1], 1, 1),
    ([1], [17], 8, 8),
    ([5], [5], 4, 1),
    ([16], [1000], 32, 8),
    ([64], [64], 8, 1),            # no prefix, four row tiles
    ([64], [191], 2, 1),           # the tree across a tile's border
    ([64, 1, 33], [200, 128, 129], 16, 1),
    ([3, 0, 7, 1], [130, 50, 7, 256], 6, 2),
    ([0, 0, 2], [1, 1, 2], 4, 4),
    ([9, 31], [300, 127], 48, 2),  # 24 heads a KV head
    ([2] * 40, list(range(2, 282, 7)), 10, 2),
    ([43], [5000], 3, 1),
    ([7, 64, 12], [3000, 777, 1], 12, 4),
])
def test_tree(nodes, ctx, heads, kv, fp8):
    ctx = [max(c, n) for c, n in zip(ctx, nodes)]
    p = Problem(nodes, ctx, heads, kv, fp8, seed=sum(ctx))
    p.check()


@pytest.mark.parametrize("fp8", POOLS)
def test_tree_bf16_output_and_repeated(fp8):
    p = Problem([16, 5, 40], [900, 4000, 64], 16, 4, fp8, seed=3)
    got, ws = p.check(torch.bfloat16)
    again, _ = p.call(torch.bfloat16, workspace=ws)
    assert torch.equal(got, again)


@pytest.mark.parametrize("fp8", POOLS)
def test_any_mask(fp8):
    rng = random.Random(5)
    nodes, ctx = [64, 20, 1, 8], [64, 150, 1, 8]
    masks = [rng.getrandbits(64) for _ in range(64 + 20)] + [0] + [0, 255, 1, 128, 0, 1 << 8, 1 << 63, 3]
    masks[0], masks[1], masks[64] = 0, 1 << 63, 0  # rows that see nothing; the last node alone; the prefix alone
    p = Problem(nodes, ctx, 6, 2, fp8, seed=8, masks=masks)
    got, _ = p.check()
    assert not got[0].any() and not got[84].any() and not got[85].any()
    assert not got[90].any()  # bits past the tree


@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-30, 8.0])
def test_scales(scale):
    Problem([16, 30], [500, 30], 4, 2, seed=4).check(scale=scale)


def test_long_context_in_many_parts():
    p = Problem([12], [70000], 2, 1, seed=6)
    got, ws = p.call()
    keys, values = (t[p.tables[0]].transpose(0, 1).reshape(1, -1, 128)[0, :70000] for t in (p.kd, p.vd))
    seen = torch.ones(12, 70000, dtype=torch.bool, device="cuda")
    seen[:, 70000 - 12:] = torch.tensor([[m >> j & 1 for j in range(12)] for m in p.masks], device="cuda").bool()
    s = torch.einsum("nhd,cd->nhc", p.q.double(), keys) * p.scale
    want = torch.softmax(s.masked_fill(~seen[:, None], float("-inf")), -1) @ values
    assert bool(((got.double() - want).abs().cpu() <= p.bound(want.cpu())).all())


def test_many_sequences():
    rng = random.Random(2)
    nodes = [rng.randint(0, 3) for _ in range(700)]
    ctx = [n + rng.randint(0 if n else 1, 40) for n in nodes]
    Problem(nodes, ctx, 2, 1, seed=2).check()


def test_large_scores_and_equal_ones():
    """Weights that pass the running reference in every tile, far and by little; and a row of equal scores."""
    p = Problem([4, 4], [1500, 1400], 8, 2, seed=12)
    ramp = torch.linspace(0, 60, 1500, device="cuda")
    for b, up in ((0, ramp), (1, ramp.flip(0)[:1400])):
        for j in range(0, p.ctx[b], 16):
            n = min(16, p.ctx[b] - j)
            p.k[p.tables[b][j // 16], :, :n, 0] = (up[j:j + n] * 16).bfloat16()
            p.kd[p.tables[b][j // 16], :, :n, 0] = (up[j:j + n] * 16).bfloat16().double()
    p.q[..., 0] = 1.0
    p.q[3] = 0.0
    p.check()


@pytest.mark.parametrize("fp8", POOLS)
def test_one_node_is_a_decode_row_and_a_chain_is_verify(fp8):
    p = Problem([1, 1, 1], [300, 17, 2000], 8, 2, fp8, seed=9, spare=0)
    got, _ = p.call(extra=0)
    out = torch.empty_like(got)
    P.paged_attention_decode(out, p.q, p.k, p.v, i32(p.tables), i32(p.ctx), p.scale, **p.scales)
    assert bool(((got - out).abs().double().cpu() <= 2 * p.bound(p.want())).all())
    p = Problem([4, 4], [300, 2000], 8, 2, fp8, seed=9, spare=0, masks=[1, 3, 7, 15] * 2)
    got, _ = p.call(extra=0)
    out = torch.empty_like(got)
    P.paged_attention_verify(out, p.q, 4, p.k, p.v, i32(p.tables), i32(p.ctx), p.scale, **p.scales)
    assert bool(((got - out).abs().double().cpu() <= 2 * p.bound(p.want())).all())


@pytest.mark.parametrize("fp8", POOLS)
def test_shared_blocks(fp8):
    p = Problem([3, 3], [200, 200], 4, 2, fp8, seed=10)
    p.tables[1][:10] = p.tables[0][:10]
    p.check()


@pytest.mark.parametrize("fp8", POOLS)
def test_scales_of_many_sizes(fp8):
    """E4M3 scales that differ by 2^40 within a tile; values of one key far above the others."""
    p = Problem([8], [400], 4, 1, fp8, seed=11)
    if fp8:
        grow = torch.logspace(-20, 20, 16, base=2, device="cuda").repeat(p.blocks, 1, 1)
        p.scales["v_scale"] *= grow
        p.vd = p.vd * grow[..., None].double()
        p.check()
        return
    p.v[p.tables[0][3], 0, 5] = 1e30
    p.vd[p.tables[0][3], 0, 5] = torch.tensor(1e30).bfloat16().double()
    p.check()


@pytest.mark.parametrize("fp8", POOLS)
def test_what_only_the_device_sees(fp8):
    for change, bits, zero, whole in (
            (dict(ctx=[0, 100, 30]), P.PKV_STATUS_BAD_CONTEXT_LEN, [0], [1, 2]),
            (dict(ctx=[-3, 100, 30]), P.PKV_STATUS_BAD_CONTEXT_LEN, [0], [1, 2]),
            (dict(ctx=[40, 100000, 30]), P.PKV_STATUS_BAD_CONTEXT_LEN, [1], [0, 2]),
            (dict(ctx=[40, 100, 5]), P.PKV_STATUS_BAD_Q_LEN, [2], [0, 1]),
            (dict(most=7), P.PKV_STATUS_BAD_Q_LEN, [2], [0, 1]),
            (dict(ctx=[0, 100, 5]), P.PKV_STATUS_BAD_CONTEXT_LEN | P.PKV_STATUS_BAD_Q_LEN, [0, 2], [1])):
        p = Problem([4, 7, 9], [40, 100, 30], 4, 2, fp8, seed=1)
        want = p.want()
        p.ctx = change.get("ctx", p.ctx)
        p.most = change.get("most", p.most)
        got, ws = p.call()
        assert status_of(ws) == bits, change
        for b in zero:
            assert not got[p.cu[b]:p.cu[b + 1]].any(), change
        for b in whole:
            rows = slice(p.cu[b], p.cu[b + 1])
            assert bool(((got[rows].double().cpu() - want[rows]).abs() <= p.bound_of(want[rows])).all()), change
    for cu, left in (([0, 4, 2, 9], slice(4, 9)), ([0, 4, 11, 50], slice(11, 20)), ([-4, 4, 11, 20], slice(0, 0))):
        p = Problem([4, 7, 9], [40, 100, 30], 4, 2, fp8, seed=1)
        out = torch.full((22, 4, 128), 7.0, device="cuda")
        p.cu = cu
        rows = p.q
        ws = P.paged_attention_tree(out[:20], rows, i64(p.masks), i32(cu), p.most, p.k, p.v, i32(p.tables), i32(p.ctx), p.scale,
                                    **p.scales)
        assert status_of(ws) & P.PKV_STATUS_BAD_Q_LEN
        assert bool((out[20:] == 7).all())
    # an invalid block contributes nothing
    for b, block in ((0, 1), (1, 6), (1, 0)):
        p = Problem([4, 7, 9], [40, 100, 30], 4, 2, fp8, seed=1)
        want = Problem([4, 7, 9], [40, 100, 30], 4, 2, fp8, seed=1)
        old = p.tables[b][block]
        for bad in (-1, p.blocks, 2 ** 31 - 1):
            p.tables[b][block] = bad
            got, ws = p.call()
            assert status_of(ws) == P.PKV_STATUS_BAD_BLOCK_ID
            p.tables[b][block] = old
            ref = drop_block(want, b, block)
            assert bool(((got.double().cpu() - ref).abs() <= p.bound_of(ref)).all())


def drop_block(p, b, block):
    """The reference without one block of a sequence."""
    out = p.want()
    n, c = p.nodes[b], p.ctx[b]
    k, v = (t[p.tables[b][:-(-c // 16)]].transpose(0, 1).reshape(p.kv, -1, 128)[:, :c].cpu() for t in (p.kd, p.vd))
    group = p.heads // p.kv
    for i in range(n):
        seen = [j for j in range(c) if j // 16 != block and (j < c - n or p.masks[p.cu[b] + i] >> (j - c + n) & 1)]
        for h in range(p.heads):
            row = p.q[p.cu[b] + i, h].double().cpu()
            out[p.cu[b] + i, h] = torch.softmax(k[h // group, seen] @ row * p.scale, 0) @ v[h // group, seen] if seen else 0
    return out


def test_a_key_that_is_not_finite():
    """Rows that see it are NaN; the others, and other sequences and heads, are not."""
    p = Problem([4, 4], [300, 300], 4, 2, seed=13, masks=[1, 3, 5, 9] * 2)
    p.k[p.tables[0][297 // 16], 0, 297 % 16, 5] = float("nan")  # node 1 of sequence 0, KV head 0
    got, _ = p.call()
    nan = torch.isnan(got).all(-1).cpu()
    assert nan[1, :2].all() and int(nan.sum()) == 2 and int(torch.isnan(got).any(-1).sum()) == 2
    p.v[p.tables[1][0], 1, 3, 7] = float("inf")  # a key of the prefix
    got, _ = p.call()
    assert bool((got[4:, 2:, 7] == float("inf")).all()) and bool(torch.isfinite(got[4:, :2]).all())


def test_graph_streams_and_a_shared_workspace():
    p, r = Problem([8, 3], [600, 40], 8, 2, seed=14), Problem([64], [2500], 4, 4, seed=15)
    want_p, ws = p.call()
    need = P.paged_attention_tree_workspace_size(1, 4, 64, P.cache_desc(r.k))
    ws = torch.zeros(max(need, ws.numel()), dtype=torch.uint8, device="cuda")
    want_r, _ = r.call()
    out_p, out_r = torch.zeros_like(want_p), torch.zeros_like(want_r)
    args = [(x.q, i64(x.masks), i32(x.cu), x.most, x.k, x.v, i32(x.tables), i32(x.ctx), x.scale) for x in (p, r)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.paged_attention_tree(out_p, *args[0], workspace=ws)
        P.paged_attention_tree(out_r, *args[1], workspace=ws)
    for _ in range(3):
        out_p.zero_(), out_r.zero_()
        graph.replay()
        assert torch.equal(out_p, want_p) and torch.equal(out_r, want_r)
    # lengths changed under the graph
    args[0][7].copy_(i32([600 - 100, 40]))
    graph.replay()
    torch.cuda.synchronize()
    p.ctx = [500, 40]
    assert torch.equal(out_p, p.call()[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out_r.zero_()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    P.paged_attention_tree(out_r, *args[1], stream=s)
    s.synchronize()
    assert not torch.cuda.current_stream().query()
    assert torch.equal(out_r, want_r)


def test_binding_refusals():
    p = Problem([2, 2], [20, 20], 4, 2, seed=1, spare=0)
    out, m, cu, t, c = torch.empty_like(p.q), i64(p.masks), i32(p.cu), i32(p.tables), i32(p.ctx)
    good = dict(out=out, q=p.q, tree_mask=m, cu_q_lens=cu, max_q_len=2, k_cache=p.k, v_cache=p.v, block_tables=t, context_lens=c,
                scale=SCALE)
    P.paged_attention_tree(**good)
    for bad in (dict(out=out[:3]), dict(out=out.half()), dict(q=p.q.float()), dict(tree_mask=m[:3]), dict(tree_mask=m.int()),
                dict(cu_q_lens=cu[:2]), dict(context_lens=c[:1]), dict(v_cache=p.v[:1]), dict(k_scale=c), dict(q=p.q[:, ::2]),
                dict(workspace=torch.empty(10, device="cuda")), dict(max_q_len=65), dict(k_cache=p.k.cpu())):
        with pytest.raises(ValueError):
            P.paged_attention_tree(**{**good, **bad})
    for bad in (dict(workspace=torch.zeros(256, dtype=torch.uint8, device="cuda")), dict(scale=float("nan"))):
        with pytest.raises(P.PagedKVError):
            P.paged_attention_tree(**{**good, **bad})


@pytest.mark.parametrize("fp8", POOLS)
@pytest.mark.parametrize("heads,kv", [(6, 2), (8, 2), (7, 1)])
def test_empty_sequences_at_every_place(heads, kv, fp8):
    """Ranges that begin anywhere among 100 sequences, most of them empty, and go on past the 32nd and the 64th."""
    rng = random.Random(heads)
    nodes = [0 if rng.random() < 0.6 or 28 < b < 36 or b in (0, 63, 64, 99) else rng.choice([1, 2, 9, 33]) for b in range(100)]
    Problem(nodes, [max(1, n + rng.choice([0, 1, 60, 150])) for n in nodes], heads, kv, fp8, seed=heads).check()


@pytest.mark.parametrize("fp8", POOLS)
@pytest.mark.parametrize("heads,nodes", [(128, 3), (256, 2), (130, 3), (64, 5), (96, 2), (1, 64), (2, 64)])
def test_rows_of_a_tile(heads, nodes, fp8):
    """One KV head: tiles of whole nodes, of parts of a node, and of rows of several nodes' parts."""
    Problem([nodes, 1], [nodes + 70, 5], heads, 1, fp8, seed=heads).check()


@pytest.mark.parametrize("heads,n", [(1022, 16500), (1002, 17400)])  # (501 heads: from row 17354 on)
def test_a_refused_length_of_many_rows(heads, n):
    """A sequence longer than max_q_len (zeros, and a status bit) whose row numbers pass 2^32 / heads-of-a-group squared."""
    kv = 2
    p = Problem([1], [20], heads, kv, seed=3)
    q = torch.cat([p.q, torch.ones(n, heads, 128, dtype=torch.bfloat16, device="cuda")])
    out = torch.full((n + 3, heads, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    q = torch.cat([q, q[:2]])
    masks = torch.ones(n + 3, dtype=torch.int64, device="cuda")
    tables, ctx = i32(p.tables * 2), i32([20, 40])
    ws = P.paged_attention_tree(out, q, masks, i32([0, 1, n + 1]), 4, p.k, p.v, tables, ctx, p.scale)
    assert status_of(ws) == P.PKV_STATUS_BAD_Q_LEN | P.PKV_STATUS_BAD_CONTEXT_LEN  # (40 tokens are more than 2 blocks hold)
    want = p.want()
    assert bool(((out[:1].double().cpu() - want).abs() <= p.bound(want, torch.bfloat16)).all())
    assert not bool(out[1:n + 1].any()) and bool((out[n + 1:] == 7).all())


@pytest.mark.parametrize("count", [256, 257, 700])
def test_hundreds_of_sequences(count):
    rng = random.Random(count)
    nodes = [rng.choice([0, 0, 1, 2, 5]) for _ in range(count)]
    nodes[-1] = 3
    Problem(nodes, [max(1, n + rng.choice([0, 3, 64, 130])) for n in nodes], 4, 2, count == 257, seed=count).check()
