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
