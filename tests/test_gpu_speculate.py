"""Verification of drafted tokens and compaction of the accepted path, against their definitions in 64 bits."""
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


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def starts(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def call(target, tokens, uniforms, cu, most, parents=None, draft=None, status=None):
    B = len(cu) - 1
    out, path = (torch.full((B, most), 77, dtype=torch.int32, device="cuda") for _ in "ab")
    counts = torch.full((B,), 77, dtype=torch.int32, device="cuda")
    P.speculative_verify(out, path, counts, target, i32(tokens), i32(cu), most, uniforms,
                         parents=None if parents is None else i32(parents), draft_probs=draft, status=status)
    return out.tolist(), path.tolist(), counts.tolist()


def problem(seed, lens, vocab, tree, sharp=2.0, odd=False):
    rng = random.Random(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rows = sum(lens)
    wide = vocab + (3 if odd else 0)
    logits = torch.randn(rows, wide, generator=g, device="cuda") * sharp
    target = torch.softmax(logits, -1)[:, :vocab]
    draft = torch.softmax(logits + 0.5 * torch.randn(rows, wide, generator=g, device="cuda"), -1)[:, :vocab]
    parents = [u for n in lens for u in (R.random_tree(rng, n, 3) if n else [])]
    up = [a + max(u, 0) for a, n in zip(starts(lens), lens) for u in parents[a:a + n]] if tree else \
        [a + max(j - 1, 0) for a, n in zip(starts(lens), lens) for j in range(n)]
    tokens = torch.multinomial(draft, 1, generator=g).flatten()[up].tolist() if rows else []
    uniforms = torch.rand(rows, generator=g, device="cuda")
    return target, draft, parents, tokens, uniforms


@pytest.mark.parametrize("vocab,odd", [(1, False), (5, False), (127, True), (1000, False), (4096, False), (50257, True),
                                       (128000, False), (152064, True)])
@pytest.mark.parametrize("tree", [False, True])
def test_verify(vocab, odd, tree):
    lens = [1, 5, 0, 2, 64, 9, 33, 8]
    for seed in range(3):
        target, draft, parents, tokens, uniforms = problem(seed, lens, vocab, tree, odd=odd)
        cu, most = starts(lens), max(lens)
        kw = dict(parents=parents) if tree else dict(draft=draft)
        want = R.verify(target, tokens, uniforms.tolist(), cu, most, **kw)
        assert call(target, tokens, uniforms, cu, most, **kw) == want
        assert call(target, tokens, uniforms, cu, most) == R.verify(target, tokens, uniforms.tolist(), cu, most)


def test_every_draft_accepted_and_every_draft_refused():
    vocab, lens = 777, [6, 6]
    target, draft, _, tokens, _ = problem(11, lens, vocab, False)
    cu = starts(lens)
    for u in (0.0, 1.0 - 2.0 ** -24):
        uniforms = torch.full((12,), u, device="cuda")
        for q in (target, draft):  # the drafter right: all stand, and the last token comes from the last row
            assert call(target, tokens, uniforms, cu, 6, draft=q) == \
                R.verify(target, tokens, uniforms.tolist(), cu, 6, draft=q)
    out, path, counts = call(target, tokens, torch.zeros(12, device="cuda"), cu, 6, draft=target)
    assert counts == [6, 6] and path == [[0, 1, 2, 3, 4, 5]] * 2
    tokens = [vocab, -1] * 6  # no such tokens
    out, path, counts = call(target, tokens, torch.zeros(12, device="cuda"), cu, 6, draft=draft)
    assert counts == [1, 1] and path == [[0, -1, -1, -1, -1, -1]] * 2 and all(r[0] >= 0 for r in out)


def test_borders():
    """Products and sums next to a border: u q against p one step apart, a draw on the boundary of two tokens."""
    # u q = q - 1.2 steps of q: above p = q - 2 steps, below q - 1 step (to which fp32 would round it)
    q, p = torch.zeros(2, 8), torch.zeros(2, 8)
    q[:, 3], p[:, 5], u = 0.6, 0.25, 1.0 - 2.0 ** -23
    for steps, accepted in ((2, False), (1, True)):
        p[:, 3] = q[0, 3] - steps * 2.0 ** -24
        counts = call(p.cuda(), [0, 3], torch.tensor([0.0, u], device="cuda"), [0, 2], 2, draft=q.cuda())[2]
        assert (counts == [2]) == accepted
    # four tokens of a quarter each: the draw at a multiple of a quarter takes the token behind the border
    p = torch.zeros(1, 4000, device="cuda")
    p[0, [1, 999, 2000, 3999]] = 0.25
    for u, token in ((0.0, 1), (0.25 - 2.0 ** -26, 1), (0.25, 999), (0.5, 2000), (0.75 - 2.0 ** -24, 2000), (0.75, 3999),
                     (1.0 - 2.0 ** -24, 3999)):
        assert call(p, [0], torch.tensor([u], device="cuda"), [0, 1], 1)[0] == [[token]]


def test_odd_probabilities():
    """NaN and below 0 count as 0, above 1 as 1; rows of nothing; weights that are all taken by refused siblings."""
    nan, inf = float("nan"), float("inf")
    p = torch.zeros(4, 600, device="cuda")
    p[0, 5], p[0, 6], p[0, 7], p[0, 500] = nan, -3.0, 7.0, inf
    p[2, 9] = 1.0
    u = torch.tensor([0.6, 0.0, 0.5, 0.999], device="cuda")
    cases = [([0, 1], [0], 1, dict()), ([1, 2], [0, 0], 1, dict()), ([2, 4], [0, 9], 2, dict()),
             ([2, 4], [0, 9], 2, dict(draft=p)), ([0, 2, 4], [0, 7, 0, 9], 2, dict(parents=[-1, 0, -1, 0]))]
    for cu, _, most, kw in cases:
        full = [0, 7, 0, 9]
        full_kw = {k: v for k, v in kw.items()}
        if "parents" in kw and len(kw["parents"]) != 4:
            full_kw["parents"] = [-1, 0, -1, 0]
        assert call(p, full, u, cu, most, **full_kw) == R.verify(p, full, u.tolist(), cu, most, **full_kw)
    assert call(p, [0] * 4, u, [1, 2], 1)[0] == [[-1]]  # a row of zeros


def test_siblings_with_one_token_and_bad_parents():
    vocab = 50
    p = torch.full((6, vocab), 1.0 / vocab, device="cuda")
    for parents in ([-1, 0, 0, 0, 0, 0], [-1, 0, 0, 5, 9, -4], [-1, 0, 1, 2, 3, 4], [-1, 0, 0, 1, 1, 2]):
        for seed in range(20):
            u = torch.rand(6, generator=torch.Generator().manual_seed(seed)) ** 4
            tokens = [0, 3, 3, 3, 4, 3]
            assert call(p, tokens, u.cuda(), [0, 6], 6, parents=parents) == \
                R.verify(p, tokens, u.tolist(), [0, 6], 6, parents=parents)


def test_bad_lengths_are_flagged():
    p = torch.full((5, 10), 0.1, device="cuda")
    u = torch.zeros(5, device="cuda")
    for cu, want in (([0, 3, 2], [3, 0]), ([0, 5, 5], [0, 0]), ([0, 2, 9], [2, 0]), ([-1, 1, 2], [0, 1])):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, path, counts = call(p, [0] * 5, u, cu, 4, status=status)
        assert [min(c, 1) for c in counts] == [min(w, 1) for w in want]
        assert int(status) == (0 if cu == [0, 5, 5] and counts[0] else P.PKV_STATUS_BAD_Q_LEN)
        for c, o, x in zip(counts, out, path):
            assert o[c:] == [-1] * (4 - c) and x[c:] == [-1] * (4 - c)


def test_many_sequences_strides_graph_and_stream():
    lens = [3] * 300
    target, draft, _, tokens, uniforms = problem(4, lens, 3001, False)
    wide = torch.full((900, 4096), float("nan"), device="cuda")
    wide[:, 64:3065] = target
    cu = starts(lens)
    want = R.verify(target, tokens, uniforms.tolist(), cu, 3, draft=draft)
    assert call(wide[:, 64:3065], tokens, uniforms, cu, 3, draft=draft) == want
    out, path = (torch.empty(300, 3, dtype=torch.int32, device="cuda") for _ in "ab")
    counts, tok, cud = torch.empty(300, dtype=torch.int32, device="cuda"), i32(tokens), i32(cu)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.speculative_verify(out, path, counts, target, tok, cud, 3, uniforms, draft_probs=draft)
    graph.replay()
    assert (out.tolist(), path.tolist(), counts.tolist()) == want
    uniforms.mul_(0.5)
    graph.replay()
    assert (out.tolist(), path.tolist(), counts.tolist()) == R.verify(target, tokens, uniforms.tolist(), cu, 3, draft=draft)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    counts.zero_()
    torch.cuda.synchronize()
    P.speculative_verify(out, path, counts, target, tok, cud, 3, uniforms, draft_probs=draft, stream=s)
    s.synchronize()
    assert counts.tolist() == R.verify(target, tokens, uniforms.tolist(), cu, 3, draft=draft)[2]


def test_verify_keeps_the_targets_distribution():
    """A chain and a tree of one draft, 60000 times: tokens as often as the target draws them (5 sigma)."""
    vocab = 6
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    p = torch.tensor([0.4, 0.05, 0.25, 0.1, 0.15, 0.05], device="cuda")
    q = torch.tensor([0.1, 0.3, 0.2, 0.2, 0.1, 0.1], device="cuda")
    B = 60000
    rows = 2 * B
    tokens = torch.zeros(B, 2, dtype=torch.int32, device="cuda")
    tokens[:, 1] = torch.multinomial(q.expand(B, -1), 1, generator=g).flatten().int()
    cu = torch.arange(0, rows + 1, 2, device="cuda").int()
    out, path = (torch.empty(B, 2, dtype=torch.int32, device="cuda") for _ in "ab")
    counts = torch.empty(B, dtype=torch.int32, device="cuda")
    for kw in (dict(draft_probs=q.expand(rows, -1).contiguous()), dict()):
        u = torch.rand(rows, generator=g, device="cuda")
        P.speculative_verify(out, path, counts, p.expand(rows, -1).contiguous(), tokens.flatten(), cu, 2, u, **kw)
        seen = torch.bincount(out[:, 0].long(), minlength=vocab).double() / B
        sigma = (p.double() * (1 - p.double()) / B).sqrt()
        assert bool(((seen - p.double()).abs() <= 5 * sigma).all()), seen


# ---- compaction -------------------------------------------------------------------------

def pool(blocks, kv, fp8, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(2, blocks, kv, 16, 128, generator=g, device="cuda")
    if not fp8:
        return [t.clone() for t in x.bfloat16()]
    s = torch.rand(2, blocks, kv, 16, generator=g, device="cuda")
    return [x[0].to(F8), x[1].to(F8), s[0].clone(), s[1].clone()]


def moved(pools, tables, ctx, cu, paths, counts):
    out = []
    for t in pools:
        rows = t.view(torch.uint8 if t.dtype == F8 else t.dtype).transpose(1, 2).flatten(0, 1).clone()
        for b, (c, path, count) in enumerate(zip(ctx, paths, counts)):
            n = cu[b + 1] - cu[b]
            at = lambda j: int(tables[b][(c - n + j) // 16]) * 16 + (c - n + j) % 16  # noqa: E731
            for i in range(1, count):
                rows[at(i)] = rows[at(path[i])]
        out.append(rows)
    return out


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kv", [1, 3, 8])
def test_compact(fp8, kv):
    rng = random.Random(kv)
    lens = [1, 16, 64, 64, 30, 2, 0, 40]
    ctx = [max(1, n + rng.choice([0, 1, 15, 16, 100])) for n in lens]
    need = [-(-c // 16) for c in ctx]
    ids = rng.sample(range(sum(need) + 5), sum(need))
    tables, at = [], 0
    for n in need:
        tables.append(ids[at:at + n] + [-9] * (max(need) - n))
        at += n
    paths, counts = [], []
    for n in lens:
        c = rng.randint(1, n) if n else 0
        if n == 64:
            c = 64 if not counts or counts[-1] != 64 else 20
        path = [0] + sorted(rng.sample(range(1, n), c - 1)) if c else []
        paths.append(path + [-1] * (64 - len(path)))
        counts.append(c)
    pools = pool(sum(need) + 5, kv, fp8)
    cu = starts(lens)
    want = moved(pools, tables, ctx, cu, paths, counts)
    scales = dict(k_scale=pools[2], v_scale=pools[3]) if fp8 else {}
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    P.kv_compact_path(pools[0], pools[1], i32(tables), i32(ctx), i32(cu), i32(paths), i32(counts), status=status, **scales)
    for t, w in zip(pools, want):
        assert torch.equal(t.view(torch.uint8 if t.dtype == F8 else t.dtype).transpose(1, 2).flatten(0, 1), w)
    assert int(status) == 0


@pytest.mark.parametrize("change,bit", [
    (dict(counts=[9]), P.PKV_STATUS_BAD_Q_LEN), (dict(ctx=[7]), P.PKV_STATUS_BAD_Q_LEN),
    (dict(ctx=[33]), P.PKV_STATUS_BAD_CONTEXT_LEN), (dict(ctx=[-5]), P.PKV_STATUS_BAD_CONTEXT_LEN),
    (dict(cu=[0, -4]), P.PKV_STATUS_BAD_Q_LEN), (dict(paths=[[0, 8, -1, 1]]), P.PKV_STATUS_BAD_Q_LEN),
    (dict(paths=[[0, 8, 99, 0]]), P.PKV_STATUS_BAD_Q_LEN), (dict(tables=[[99, -1]], paths=[[0, 2, 3, 7]]), P.PKV_STATUS_BAD_BLOCK_ID),
])
def test_compact_checks_what_only_the_device_sees(change, bit):
    a = dict(tables=[[0, 1]], ctx=[20], cu=[0, 8], paths=[[0, 1, 2, 3]], counts=[4])
    a.update(change)
    pools = pool(2, 2, False)
    before = [t.clone() for t in pools]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    P.kv_compact_path(*pools, i32(a["tables"]), i32(a["ctx"]), i32(a["cu"]), i32(a["paths"]), i32(a["counts"]), status=status)
    assert int(status) == bit
    assert all(torch.equal(x, y) for x, y in zip(pools, before))


def test_binding_refusals():
    p, u = torch.full((4, 10), 0.1, device="cuda"), torch.zeros(4, device="cuda")
    out, n, cu, tok = i32([[0, 0], [0, 0]]), i32([0, 0]), i32([0, 2, 4]), i32([0] * 4)
    k = pool(2, 2, False)
    lens = i32([8, 8])
    for call_ in (lambda: P.speculative_verify(out, out, n, p, tok, cu, 3, u),
                  lambda: P.speculative_verify(out, out, n[:1], p, tok, cu, 2, u),
                  lambda: P.speculative_verify(out, out, n, p.double(), tok, cu, 2, u),
                  lambda: P.speculative_verify(out, out, n, p[:3], tok, cu, 2, u),
                  lambda: P.speculative_verify(out, out, n, p.T, tok, cu, 2, u),
                  lambda: P.speculative_verify(out, out, n, p, tok, cu, 2, u[:3]),
                  lambda: P.speculative_verify(out, out, n, p, tok, cu, 2, u, parents=tok[:2]),
                  lambda: P.speculative_verify(out, out, n, p, tok, cu, 2, u, draft_probs=p[:, :4]),
                  lambda: P.speculative_verify(out.long(), out, n, p, tok, cu, 2, u),
                  lambda: P.kv_compact_path(*k, out, lens, cu[:2], out, n), lambda: P.kv_compact_path(*k, out, lens, cu, out[:1], n),
                  lambda: P.kv_compact_path(*k, out, lens, cu, out, n, k_scale=u)):
        with pytest.raises(ValueError):
            call_()
    with pytest.raises(P.PagedKVError):
        P.speculative_verify(out, out, n, p, tok, cu, 2, u, parents=tok, draft_probs=p)
