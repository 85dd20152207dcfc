"""Tree attention over an FP8 pool where it can go wrong in ways of its own: V scales of every size, rows of Q as codes,
weights times scales; and partials whose loss no average hides (both pools)."""
import math

import pytest
import torch

import speculative_reference as R
from paged_kv_cache_95_gb300 import pagedkv as P
from test_gpu_tree import F8, POOLS, SCALE, Problem, i32, i64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(built_library):
    P.load_library()


def shrink(p, by, where=slice(None)):
    """V scales times `by` (a power of two: exact), in the pool and in the reference."""
    p.scales["v_scale"][where] *= by
    p.vd[where] *= by


def put(pool, at, x):
    """Values into a pool of either type (codes move as bytes)."""
    x = x.to(pool.dtype)
    (pool.view(torch.uint8) if pool.dtype is F8 else pool)[at] = x.view(torch.uint8) if pool.dtype is F8 else x


def off(got, want, bound):
    gap = (got.double().cpu() - want).abs()
    assert bool((gap <= bound).all()), (float(gap.max()), float((gap / bound.clamp(min=1e-300)).max()))


# ---- V scales that are small -------------------------------------------------------------

@pytest.mark.parametrize("by", [-8, -15, -20, -24, -60, -90])
@pytest.mark.parametrize("ctx", [40, 64, 100, 128, 200])
def test_small_v_scales(by, ctx):
    """Outputs shrink with the V scales, in a context's last tile as in its others: slots behind the context (NaN in these
    pools) weigh nothing.  The bound is relative to the problem's own values."""
    p = Problem([9, 16], [ctx, ctx + 3], 8, 2, True, seed=ctx)
    shrink(p, 2.0 ** by)
    p.check()


@pytest.mark.parametrize("by", [-8, -24])
def test_small_v_scales_beside_a_bad_block(by):
    p = Problem([4, 7], [192, 128], 4, 2, True, seed=7)
    shrink(p, 2.0 ** by)
    want = p.want()  # as if block 5 of sequence 0 were not there
    n, c = p.nodes[0], p.ctx[0]
    k, v = (t[p.tables[0]].transpose(0, 1).reshape(p.kv, -1, 128)[:, :c].cpu() for t in (p.kd, p.vd))
    for i in range(n):
        seen = [j for j in range(c) if j // 16 != 5 and (j < c - n or p.masks[i] >> (j - c + n) & 1)]
        for h in range(p.heads):
            g = h // (p.heads // p.kv)
            want[i, h] = torch.softmax(k[g, seen] @ p.q[i, h].double().cpu() * p.scale, 0) @ v[g, seen]
    bound = p.bound(want)
    p.tables[0][5] = -1
    got, _ = p.call()
    off(got, want, bound)


# ---- V scales of keys that a row does not see ---------------------------------------------

@pytest.mark.parametrize("up", [12, 24, 60])
@pytest.mark.parametrize("ctx", [30, 64, 131])
def test_a_hidden_node_with_a_far_larger_v_scale(up, ctx):
    """Rows that do not see the node are as exact as without it (the bound leaves it out); rows that see it, as with it."""
    nodes, hidden = 5, 2
    masks = [1 << i for i in range(nodes)]
    masks[4] |= 1 << hidden
    p = Problem([nodes], [ctx], 8, 2, True, seed=ctx, masks=masks)
    at = ctx - nodes + hidden
    where = (p.tables[0][at // 16], slice(None), at % 16)
    small = p.bound(p.want())
    shrink(p, 2.0 ** up, where)
    got, _ = p.call()
    want = p.want()
    blind = [i for i in range(nodes) if i != hidden and i != 4]
    off(got[blind], want[blind], small[blind])
    off(got, want, p.bound(want))


# ---- weights ------------------------------------------------------------------------------

class Exact(Problem):
    """Rows of Q with one value other than 0 (a power of two) and whole numbers of up to 15 as its keys' codes, so that q k is
    exact whatever the accumulator; K scales, V scales and V as they come."""

    def __init__(self, nodes, ctx, heads, kv, seed, spread=8.0):
        super().__init__(nodes, ctx, heads, kv, True, seed=seed)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + 1)
        self.q.zero_()
        self.q[..., 3] = 1.0
        whole = torch.randint(-15, 16, self.k.shape[:3], generator=g, device="cuda").float()
        hole = self.k.view(torch.uint8)[..., 0] == 0x7F
        s = torch.where(hole, 1.0, self.scales["k_scale"])
        put(self.k, (..., 3), torch.where(hole, float("nan"), whole))
        self.kd[..., 3] = (whole * s).double()
        self.scale = spread / 15  # scores in +-spread

    def tight(self, want):
        """A score of up to 8 (12 in the log2 domain) is off by 2^-24 of it for each of three roundings (the K scale, the row's
        factor, the reference): 12 x 3 x 2^-24 x ln 2 < 2^-19 of a weight; exp2 by 2^-21; its product with the V scale by
        2^-24, its two fp16 parts by 2^-22 or 2^-31 of the row's largest times the tile's largest V scale (here at most 2^7
        above the least); a sum of n fp32 terms, each entering as two, by 2 n 2^-23.  A mean by these of sum w |v|, once
        for the numerator and once for the sum."""
        n = max(self.ctx)
        each = 2.0 ** -19 + 2.0 ** -21 + 2.0 ** -24 + 2.0 ** -22 + n * 2.0 ** -22
        mean = R.tree_attention(self.q, self.masks, self.cu, self.kd, self.vd.abs(), self.tables, self.ctx, self.scale)
        live = torch.unique(torch.tensor([b for t, c in zip(self.tables, self.ctx) for b in t[:-(-c // 16)]])).cuda()
        return each * (mean + want.abs()) + n * 2.0 ** -30 * float(self.vd[live].abs().max()) + want.abs() * 2.0 ** -23


@pytest.mark.parametrize("nodes,ctx", [([1], [7]), ([3], [24]), ([4, 9], [64, 40]), ([16], [150]), ([5], [300])])
def test_weights_keep_22_bits(nodes, ctx):
    """As the FP8 decode and verify of the same pool do.  (With one fp16 value a weight, off by up to 2^-11, rows of few keys are past
    the bound.)"""
    p = Exact(nodes, ctx, 8, 2, seed=sum(ctx))
    got, ws = p.call()
    want = p.want()
    off(got, want, p.tight(want))


@pytest.mark.parametrize("ctx", [40, 150])
def test_a_chain_holds_what_verify_holds(ctx):
    """The same rows through both entry points: off the definition by the same bound."""
    p = Exact([4, 4], [ctx, ctx + 9], 4, 2, seed=ctx)
    p.masks = [1, 3, 7, 15] * 2
    got, _ = p.call(extra=0)
    out = torch.empty_like(got)
    P.paged_attention_verify(out, p.q, 4, p.k, p.v, i32(p.tables), i32(p.ctx), p.scale, kernel=P.PKV_VERIFY_DECODE_KERNEL,
                             **p.scales)
    want = p.want()
    off(out, want, p.tight(want))
    off(got, want, p.tight(want))


@pytest.mark.parametrize("gap", [0, 8, 16, 20])
def test_a_heavy_key_with_a_small_v_scale(gap):
    """A key with nearly all of the weight and a V scale 2^-gap of its tile's largest keeps 2^-(31 - gap) of its value."""
    p = Exact([1], [20], 4, 1, seed=gap)
    b, i = p.tables[0][0], 5
    low = torch.full((1, 16), -15.0, device="cuda")
    put(p.k, (b, slice(None), slice(None), 3), low)
    put(p.k, (p.tables[0][1], slice(None), slice(0, 4), 3), low[:, :4])
    put(p.k, (b, slice(None), i, 3), -low[:, 0])
    s = p.scales["k_scale"]
    s[p.tables[0]] = torch.where(torch.isnan(s[p.tables[0]]), s[p.tables[0]], 1.0)
    p.kd[p.tables[0]] = 0
    p.kd[p.tables[0], ..., 3] = -15
    p.kd[b, :, i, 3] = 15
    p.scale = 1.0  # the others weigh e^-30
    vs = p.scales["v_scale"]
    vs[p.tables[0]] = torch.where(torch.isnan(vs[p.tables[0]]), vs[p.tables[0]], 1.0)
    vs[b, :, i] = 1.2987013 * 2.0 ** -gap
    p.vd[b, :, i] = p.v[b, :, i].double() * float(vs[b, 0, i])
    got, _ = p.call()
    want = p.vd[b, 0, i].cpu().expand(1, 4, 128)
    # the others: 19 of e^-30 x 448; the key's: two fp16 parts
    off(got, want, 19 * math.exp(-30) * 448 + (2.0 ** -20 + 2.0 ** -(30 - gap)) * want.abs() + 1e-12)


# ---- rows of Q ----------------------------------------------------------------------------

@pytest.mark.parametrize("fp8,what", [(False, float("nan")), (True, float("nan")), (True, float("inf")), (True, float("-inf"))])
def test_rows_of_q_that_are_not_finite(fp8, what):
    """Such a row is NaN, or zero where it sees no key; the others are what they were."""
    masks = [0, 1 << 1, 0, 1 << 3]
    p = Problem([4, 3], [4, 150], 4, 2, fp8, seed=21, masks=masks + [1, 3, 5])
    whole, _ = p.call()
    p.q[0, 1, 5], p.q[1, 2, 127], p.q[5, 0, 64] = what, what, what
    got, _ = p.call()
    nan = torch.zeros(7, 4, dtype=torch.bool)
    nan[1, 2] = nan[5, 0] = True
    assert torch.equal(torch.isnan(got).all(-1).cpu(), nan)
    keep = ~nan.cuda()
    assert torch.equal(got[keep], whole[keep]) and not got[0].any() and not got[2].any()


@pytest.mark.parametrize("by", [-100, -30, 40, 100])
def test_rows_of_q_of_any_size(by):
    """Powers of two that the softmax scale undoes change no bit: a row's codes are those of its largest value."""
    p = Problem([5, 16], [300, 90], 8, 2, True, seed=22)
    want, _ = p.check()
    p.q *= 2.0 ** by
    got, _ = p.call(scale=p.scale * 2.0 ** -by)
    assert torch.equal(got, want)


def test_rows_of_q_that_are_zero_or_nearly():
    p = Problem([4, 2], [200, 64], 4, 2, True, seed=23)
    p.q[0], p.q[4, 1] = 0.0, 0.0
    p.q[1] *= 2.0 ** -120
    p.q[2, 0] *= 2.0 ** -133  # the least bf16 numbers
    p.check()


@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-30, 8.0])
def test_softmax_scales(scale):
    p = Problem([16, 30], [500, 30], 4, 2, True, seed=4)
    p.check(scale=scale / SCALE * p.scale)


def test_large_scores_and_equal_ones():
    """Weights that pass the running reference in every tile, far and by little; and a row of equal scores."""
    p = Exact([4, 4], [1500, 1400], 8, 2, seed=12)
    s = p.scales["k_scale"]
    s[:] = torch.where(torch.isnan(s), s, 1.0)
    p.kd.zero_()
    ramp = torch.linspace(0, 60, 1500, device="cuda")
    for b, up in ((0, ramp), (1, ramp.flip(0)[:1400])):
        for j in range(0, p.ctx[b], 16):
            n = min(16, p.ctx[b] - j)
            codes = (up[j:j + n] * 7).to(F8)
            put(p.k, (p.tables[b][j // 16], slice(None), slice(0, n), 3), codes.expand(2, n))
            p.kd[p.tables[b][j // 16], :, :n, 3] = codes.double()
    p.scale = 1 / 7
    p.q[3] = 0.0
    got, _ = p.call()
    want = p.want()
    # (scores of up to 60: 87 x 3 x 2^-24 x ln 2 < 2^-16 of a weight in the place of 2^-19)
    off(got, want, 2 * p.tight(want))


def test_keys_that_are_not_finite():
    """A code of NaN, and scales that are NaN or infinite, reach the rows that see their key and no others."""
    p = Problem([4, 4], [300, 300], 4, 2, True, seed=13, masks=[1, 3, 5, 9] * 2)
    p.k.view(torch.uint8)[p.tables[0][297 // 16], 0, 297 % 16, 5] = 0x7F  # the code of NaN: node 1 of sequence 0, KV head 0
    got, _ = p.call()
    nan = torch.isnan(got).all(-1).cpu()
    assert nan[1, :2].all() and int(nan.sum()) == 2 and int(torch.isnan(got).any(-1).sum()) == 2
    p.scales["k_scale"][p.tables[0][298 // 16], 1, 298 % 16] = float("nan")  # node 2, KV head 1
    got, _ = p.call()
    nan = torch.isnan(got).all(-1).cpu()
    assert nan[1, :2].all() and nan[2, 2:].all() and int(nan.sum()) == 4 and int(torch.isnan(got).any(-1).sum()) == 4
    p.v.view(torch.uint8)[p.tables[1][0], 1, 3, 7] = 0xFF  # a key of the prefix
    got, _ = p.call()
    assert bool(torch.isnan(got[4:, 2:, 7]).all()) and bool(torch.isfinite(got[4:, :2]).all())
    p.scales["v_scale"][p.tables[1][2], 0, 1] = float("inf")
    got, _ = p.call()
    assert not bool(torch.isfinite(got[4:, :2]).any())


def test_graph_streams_and_a_shared_workspace():
    p, r = Problem([8, 3], [600, 40], 8, 2, True, seed=14), Problem([64], [2500], 4, 4, True, seed=15)
    want_p, ws = p.call()
    need = P.paged_attention_tree_workspace_size(1, 4, 64, P.cache_desc(r.k))
    ws = torch.zeros(max(need, ws.numel()), dtype=torch.uint8, device="cuda")
    want_r, _ = r.call()
    out_p, out_r = torch.zeros_like(want_p), torch.zeros_like(want_r)
    args = [(x.q, i64(x.masks), i32(x.cu), x.most, x.k, x.v, i32(x.tables), i32(x.ctx), x.scale) for x in (p, r)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.paged_attention_tree(out_p, *args[0], workspace=ws, **p.scales)
        P.paged_attention_tree(out_r, *args[1], workspace=ws, **r.scales)
    for _ in range(3):
        out_p.zero_(), out_r.zero_()
        graph.replay()
        assert torch.equal(out_p, want_p) and torch.equal(out_r, want_r)
    args[0][7].copy_(i32([600 - 100, 40]))  # lengths changed under the graph
    graph.replay()
    torch.cuda.synchronize()
    p.ctx = [500, 40]
    assert torch.equal(out_p, p.call()[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out_r.zero_()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    P.paged_attention_tree(out_r, *args[1], stream=s, **r.scales)
    s.synchronize()
    assert not torch.cuda.current_stream().query()
    assert torch.equal(out_r, want_r)


# ---- partials -----------------------------------------------------------------------------

@pytest.mark.parametrize("peaks", [False, True])
@pytest.mark.parametrize("fp8", POOLS)
@pytest.mark.parametrize("nodes,ctx,heads", [(12, 70000, 2), (43, 5000, 3), (5, 3300, 8), (64, 9000, 4)])
def test_every_part_counts(nodes, ctx, heads, fp8, peaks):
    """The values say which tile of 64 keys they come from (a 1 in the place of the tile's number modulo 128), so that an output
    is the share of few tiles: a part left out or taken twice changes its tiles' places by a tenth and more.

    Equal scores: weights of 1 and whole sums below 2^24, exact but for the division and the output (2^-22).  Scores of whole
    numbers by the tile (0 .. 4 natural units, in no order): a weight is off by 6 x 3 x 2^-24 ln 2 + 2^-21 < 2^-19 and
    2^-16 (bf16 parts); sums run over a part (8 tiles at most: 512 keys, each entering as two values) and over up to
    152 parts: (2 x 512 + 152) x 2^-23 < 2^-12; 2^-11 covers numerator and sum."""
    p = Problem([nodes], [ctx], heads, 1, fp8, seed=6)
    key = torch.arange(ctx, device="cuda")
    tile = key // 64
    table = torch.tensor(p.tables[0], device="cuda")
    at = (table[key // 16], 0, key % 16)
    units = (tile * 37 % 5).float()
    values = torch.nn.functional.one_hot(tile % 128, 128).float()
    keys = torch.zeros(ctx, 128, device="cuda")
    keys[:, 0] = units
    p.q.zero_()
    if peaks:
        p.q[..., 0] = 1.0
    p.scale = 1.0
    for pool, x in ((p.k, keys), (p.v, values)):
        put(pool, at, x)
    for s in p.scales.values():
        s[at] = 1.0
    seen = torch.ones(nodes, ctx, dtype=torch.bool)
    seen[:, ctx - nodes:] = torch.tensor([[m >> j & 1 for j in range(nodes)] for m in p.masks]).bool()
    weight = torch.exp(units.double() * (1.0 if peaks else 0.0)).cpu() * seen
    want = (weight / weight.sum(-1, keepdim=True)) @ values.double().cpu()
    got, _ = p.call()
    off(got, want[:, None].expand(-1, heads, -1), want[:, None] * 2.0 ** (-11 if peaks else -22))
