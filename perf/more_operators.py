"""Measured cases of a speculative decoding step's operators.

A step of speculative decoding checks a tree (or a chain) of drafted tokens in one pass
of the target model.  Node 0 of a sequence's tree is the token sampled last, whose keys
and values are not cached yet; the other nodes are drafts, each behind its parent.  The
operators, in the order a step calls them: rotary positions (alone, and on the way into
the paged cache, bf16 or E4M3 with one scale per token and head), attention of the
tree's rows over the cached prefix and their own ancestors, verification of the drafts
against the target's probabilities with given random numbers, and moving the accepted
path's rows to consecutive slots.

``run`` makes one pass: with ``own`` through the library's entry points, without it in
elementary torch operations, in 32 bits (64 for angles, for the sums that a token is
drawn by and for products next to a border), rounded once at the end.  ``exact``
computes the same from the definition in 64 bits.
"""
import math
import random

import torch

own = False

D, BLOCK = 128, 16
SCALE = 1.0 / math.sqrt(D)
F8 = torch.float8_e4m3fn


def listed():
    return [
        # The rotated parts of latent attention's queries in one decode step: slices of wider heads, interleaved pairs.
        dict(name="rotate step", kind="rotate", tokens=64, heads=32, dim=64, wide=192, rotary=64, layout="interleaved",
             scaling="none", far=4096),
        # A prefill chunk's keys and queries in one projection, half of each head rotated, positions stretched 32-fold.
        dict(name="rotate chunk", kind="rotate", tokens=8192, heads=40, dim=128, wide=128, rotary=64, layout="half",
             scaling="by_parts", far=131072),
        # One decode step of 64 sequences (five of them padding): the smallest call, where the launch counts.
        dict(name="append step", kind="append", fp8=False, tokens=64, padded=5, heads=32, kv=8, rotary=128,
             layout="half", scaling="none", far=4096),
        # Prefill of a long chunk into an 8-bit cache, far into a long document.
        dict(name="append chunk fp8", kind="append", fp8=True, tokens=16384, padded=0, heads=32, kv=8, rotary=128,
             layout="half", scaling="by_wavelength", far=1000000),
        # One sequence of a thousand tokens and a small tree: the latency of a lone request.
        dict(name="tree one", kind="tree", fp8=False, seqs=1, lo=1000, hi=1000, nodes_lo=16, nodes=16, heads=32, kv=8,
             lens=1),
        # The ragged batch of the library's benchmark (64 sequences of 512 to 4096 tokens, 32 heads over 8), small trees.
        dict(name="tree ragged", kind="tree", fp8=False, seqs=64, lo=512, hi=4096, nodes_lo=5, nodes=16, heads=32, kv=8,
             lens=2),
        # The long-context batch (8 sequences of 32K tokens, 64 heads over 8).
        dict(name="tree long", kind="tree", fp8=False, seqs=8, lo=32768, hi=32768, nodes_lo=16, nodes=16, heads=64,
             kv=8, lens=3),
        # The ragged batch over an 8-bit cache, trees of up to 32 nodes.
        dict(name="tree ragged fp8", kind="tree", fp8=True, seqs=64, lo=512, hi=4096, nodes_lo=16, nodes=32, heads=32,
             kv=8, lens=4),
        # Chains of four drafts with the drafter's probabilities, a large vocabulary.
        dict(name="verify chain", kind="verify", tree=False, seqs=64, nodes_lo=5, nodes=5, vocab=128000, lens=5),
        # Trees verified against the target alone, an odd vocabulary.
        dict(name="verify tree", kind="verify", tree=True, seqs=16, nodes_lo=8, nodes=32, vocab=50257, lens=6),
        # Accepted paths of a batch's small trees moved together.
        dict(name="compact step", kind="compact", fp8=False, seqs=64, lo=512, hi=4096, nodes_lo=5, nodes=16, kv=8,
             lens=7),
        # A large batch of large trees over an 8-bit cache.
        dict(name="compact fp8", kind="compact", fp8=True, seqs=256, lo=64, hi=2048, nodes_lo=16, nodes=64, kv=8,
             lens=8),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    kind = rng.choice(["rotate", "append", "tree", "tree", "verify", "compact"])
    lens = rng.randint(1, 1 << 30)
    turn = dict(layout=rng.choice(["half", "interleaved"]), far=_spread(rng, 64, 1000000),
                scaling=rng.choice(["none", "linear", "ntk", "by_parts", "by_wavelength"]))
    if kind == "rotate":
        dim, heads = rng.choice([64, 80, 96, 128, 256]), rng.choice([1, 5, 8, 32, 40])
        return dict(kind=kind, tokens=_spread(rng, 1, 8192 * 40 // (heads * max(1, dim // 128))), heads=heads, dim=dim,
                    wide=dim + rng.choice([0, 64, 128]), rotary=rng.choice([16, 32, 48, 64, dim]), **turn)
    if kind == "append":
        tokens, kv = _spread(rng, 1, 16384), rng.choice([1, 2, 4, 8])
        return dict(kind=kind, fp8=rng.random() < 0.5, tokens=tokens, padded=rng.randint(0, min(5, tokens - 1)),
                    heads=kv * rng.choice([1, 3, 4]), kv=kv, rotary=rng.choice([32, 64, 96, 128, 128]), **turn)
    if kind == "tree":
        kv, group, nodes = rng.choice([1, 2, 8]), rng.choice([1, 4, 5, 8]), _spread(rng, 1, 64)
        seqs = _spread(rng, 1, 96)
        hi = _spread(rng, nodes, max(nodes, 32768 * 64 * 64 // (seqs * kv * max(32, group * nodes))))
        hi = max(nodes, min(hi, 65536))
        return dict(kind=kind, fp8=rng.random() < 0.5, seqs=seqs, lo=max(nodes, hi // rng.randint(1, 8)), hi=hi,
                    nodes_lo=rng.randint(1, nodes), nodes=nodes, heads=kv * group, kv=kv, lens=lens)
    if kind == "verify":
        tree = rng.random() < 0.5
        nodes, vocab = _spread(rng, 1, 64 if tree else 9), _spread(rng, 500, 160000)
        seqs = _spread(rng, 1, max(1, min(128, 64 * 5 * 128000 // (nodes * vocab))))
        return dict(kind=kind, tree=tree, seqs=seqs, nodes_lo=rng.randint(1, nodes), nodes=nodes, vocab=vocab, lens=lens)
    nodes = _spread(rng, 2, 64)
    return dict(kind=kind, fp8=rng.random() < 0.5, seqs=_spread(rng, 1, 256), lo=64, hi=_spread(rng, 64, 2048),
                nodes_lo=rng.randint(2, nodes), nodes=nodes, kv=rng.choice([1, 2, 5, 8]), lens=lens)


def _shape(case):
    """What a case's ``lens`` settles: the trees' parents, the context lengths (nodes counted), the accepted paths."""
    rng = random.Random(case["lens"])
    nodes = [rng.randint(case["nodes_lo"], case["nodes"]) for _ in range(case["seqs"])]
    chain = case["kind"] == "verify" and not case["tree"]
    parents = [[-1] + [j - 1 if chain else rng.randint(max(0, j - 8), j - 1) for j in range(1, n)] for n in nodes]
    ctx = [max(n, rng.randint(case["lo"], case["hi"])) for n in nodes] if "lo" in case else None
    # A path's nodes lie behind the slots it moves to, as in a tree that is numbered level by level.
    kept = [rng.randint(1, max(1, min(8, n // 2))) for n in nodes]
    paths = [[0] + sorted(rng.sample(range(c, n), c - 1)) for c, n in zip(kept, nodes)]
    return nodes, parents, ctx, paths


def _masks(parents):
    """Per node the nodes that it sees, as bits: its ancestors and itself."""
    out = []
    for tree in parents:
        seen = []
        for j, up in enumerate(tree):
            seen.append((seen[up] if up >= 0 else 0) | 1 << j)
        out += seen
    return out


def work(case):
    kind = case["kind"]
    if kind == "rotate":
        n = case["tokens"] * case["heads"]
        return dict(bytes=n * case["dim"] * 4 + case["tokens"] * 4, flops=n * case["rotary"] * 3)
    if kind == "append":
        t, h, kv, real = case["tokens"], case["heads"], case["kv"], case["tokens"] - case["padded"]
        row = D + 4 if case["fp8"] else 2 * D
        return dict(bytes=t * (h * 4 * D + 8) + real * kv * 2 * (2 * D + row),
                    flops=(t * h + real * kv) * case["rotary"] * 3 + (real * kv * 2 * D * 3 if case["fp8"] else 0))
    nodes, _, ctx, paths = _shape(case)
    if kind == "tree":
        h, row = case["heads"], D + 4 if case["fp8"] else 2 * D
        seen = sum(n * (c - n) + sum(bin(m).count("1") for m in _masks([p]))
                   for n, c, p in zip(nodes, ctx, _shape(case)[1]))
        return dict(bytes=sum(ctx) * case["kv"] * 2 * row + sum(nodes) * (h * 4 * D + 8), flops=4 * D * h * seen)
    if kind == "verify":
        # A sequence's last token is drawn from one row of the target's probabilities, less the drafter's of that row.
        return dict(bytes=case["seqs"] * case["vocab"] * 4 * (1 if case["tree"] else 2) + sum(nodes) * 24,
                    flops=case["seqs"] * case["vocab"] * 3)
    row = D + 4 if case["fp8"] else 2 * D
    moved = sum(len(p) - 1 for p in paths)
    return dict(bytes=moved * case["kv"] * 4 * row + 8 * case["seqs"], flops=0)


# ---- inputs -----------------------------------------------------------------------

def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).bfloat16()


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def _plan(case):
    """The scaling of a case's positions: (kind, factor, length before the scaling, low, high)."""
    return dict(none=("none", 1.0, 0, 0.0, 0.0), linear=("linear", 4.0, 0, 0.0, 0.0), ntk=("ntk", 4.0, 0, 0.0, 0.0),
                by_parts=("by_parts", 32.0, 4096, 1.0, 32.0),
                by_wavelength=("by_wavelength", 8.0, 8192, 1.0, 4.0))[case["scaling"]]


BASE = 500000.0


def _frequencies(case):
    """Angles per position of the rotated pairs in 64 bits, and what the sines and cosines are multiplied by."""
    d, (kind, factor, length, low, high) = case["rotary"], _plan(case)
    base = BASE * factor ** (d / (d - 2)) if kind == "ntk" else BASE
    i = torch.arange(d // 2, dtype=torch.float64, device="cuda")
    f = torch.exp(-2.0 * i / d * math.log(base))
    if kind == "linear":
        f = f / factor
    elif kind == "by_parts":
        # The pair that turns n times over the length before: slower pairs are stretched, faster ones left.
        at = [d * math.log(length / (2 * math.pi * n)) / (2 * math.log(base)) for n in (high, low)]
        a, b = max(0, math.floor(at[0])), min(d - 1, math.ceil(at[1]))
        ramp = ((i - a) / max(b - a, 0.001)).clamp(0, 1)
        f = f / factor * ramp + f * (1 - ramp)
    elif kind == "by_wavelength":
        turns = length * f / (2 * math.pi)
        keep = ((turns - low) / (high - low)).clamp(0, 1)
        f = (1 - keep) * f / factor + keep * f
    return f, 0.1 * math.log(factor) + 1 if kind == "by_parts" else 1.0


def _rotary(s, case, gen):
    s["layout"], s["rotary"] = case["layout"], case["rotary"]
    s["positions"] = torch.randint(0, case["far"], (case["tokens"],), generator=gen, device="cuda").int()
    s["angles"], s["magnitude"] = _frequencies(case)
    if own:
        from paged_kv_cache_95_gb300 import pagedkv as P
        kind, factor, length, low, high = _plan(case)
        s["frequencies"], s["magnitude"] = P.rotary_frequencies(case["rotary"], BASE, scaling=kind, factor=factor,
                                                                original_length=length, low=low, high=high)


def _pool(gen, blocks, kv, fp8):
    """K and V pools.  One more block lies behind them, where the plain form puts padding tokens."""
    s = {}
    for n in ("k", "v"):
        x = _normal(gen, blocks + 1, kv, BLOCK, D)
        if fp8:
            a = x.float().abs().amax(-1, keepdim=True)
            s[n + "_all"] = (x.float() * (448.0 / a)).to(F8)
            s[n + "_all_scale"] = (a / 448.0).squeeze(-1).contiguous()
            s[n + "_scale"] = s[n + "_all_scale"][:blocks]
        else:
            s[n + "_all"] = x
        s[n + "_cache"] = s[n + "_all"][:blocks]
    return s


def _tables(gen, s, lens):
    """Block tables over permuted blocks."""
    need = [-(-n // BLOCK) for n in lens]
    perm = torch.randperm(sum(need), generator=gen, device="cuda").int()
    col = torch.arange(max(need), device="cuda")
    at = torch.tensor(_starts(need)[:-1], device="cuda")[:, None] + col
    have = col < torch.tensor(need, device="cuda")[:, None]
    s["block_tables"] = torch.where(have, perm[at.clamp(max=sum(need) - 1)], 0).int().contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    kind = case["kind"]
    s = {}
    if kind == "rotate":
        _rotary(s, case, gen)
        x = _normal(gen, case["tokens"], case["heads"], case["wide"])
        s["x"] = x[..., case["wide"] - case["dim"]:]
        s["out"] = torch.empty(case["tokens"], case["heads"], case["dim"], dtype=torch.bfloat16, device="cuda")
    elif kind == "append":
        t, h, kv = case["tokens"], case["heads"], case["kv"]
        blocks = -(-t // BLOCK) + 64
        s = _pool(gen, blocks, kv, case["fp8"])
        _rotary(s, case, gen)
        x = _normal(gen, t, h + 2 * kv, D)  # one projection gives all three
        s["q"], s["key"], s["value"] = x[:, :h], x[:, h:h + kv], x[:, h + kv:]
        s["q_out"] = torch.empty(t, h, D, dtype=torch.bfloat16, device="cuda")
        slots = torch.randperm(blocks * BLOCK, generator=gen, device="cuda")[:t].int()
        if case["padded"]:
            slots[t - case["padded"]:] = -1
        s["slots"], s["blocks"] = slots, blocks
    else:
        nodes, parents, ctx, paths = _shape(case)
        s["cu"], s["most"] = _i32(_starts(nodes)), max(nodes)
        rows = sum(nodes)
        if kind == "verify":
            s["parents"] = _i32([u for tree in parents for u in tree]) if case["tree"] else None
            logits = 2.0 * torch.randn(rows, case["vocab"], generator=gen, device="cuda")
            # The drafter knows the target's mind, not all of it.
            draft = logits + 0.7 * torch.randn(rows, case["vocab"], generator=gen, device="cuda")
            s["target"] = torch.softmax(2.0 * logits, -1)
            s["draft"] = torch.softmax(2.0 * draft, -1)
            up = torch.tensor([a + max(u, 0) for a, tree in zip(_starts(nodes), parents) for u in tree], device="cuda")
            s["tokens"] = torch.multinomial(s["draft"], 1, generator=gen).flatten()[up].int()
            if case["tree"]:  # siblings hold the tokens that the drafter likes best, in their order
                rank, count = [], {}
                for a, tree in zip(_starts(nodes), parents):
                    for u in tree:
                        rank.append(count.get(a + u, 0))
                        count[a + u] = rank[-1] + 1
                best = s["draft"].topk(min(64, case["vocab"]), -1).indices
                s["tokens"] = best[up, torch.tensor(rank, device="cuda")].int()
                s["draft"] = None
            s["uniforms"] = torch.rand(rows, generator=gen, device="cuda")
            n = case["seqs"]
            s["tokens_out"], s["path"] = (torch.empty(n, s["most"], dtype=torch.int32, device="cuda") for _ in "ab")
            s["counts"] = torch.empty(n, dtype=torch.int32, device="cuda")
        else:
            s.update(_pool(gen, sum(-(-n // BLOCK) for n in ctx), case["kv"], case["fp8"]))
            _tables(gen, s, ctx)
            s["context_lens"] = _i32(ctx)
            if kind == "tree":
                bits = [m - (1 << 64) if m >> 63 else m for m in _masks(parents)]
                s["mask"] = torch.tensor(bits, dtype=torch.int64, device="cuda")
                s["q"] = _normal(gen, rows, case["heads"], D)
                s["out"] = torch.empty(rows, case["heads"], D, dtype=torch.bfloat16, device="cuda")
                s["workspace"] = None
            else:
                s["path"] = _i32([p + [-1] * (s["most"] - len(p)) for p in paths])
                s["counts"] = _i32([len(p) for p in paths])
    s["kind"], s["fp8"] = kind, bool(case.get("fp8"))
    return s


# ---- one pass -----------------------------------------------------------------------

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _pools(s):
    return [s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale") if n in s]


def _run_own(s):
    from paged_kv_cache_95_gb300 import pagedkv as P
    scales = dict(k_scale=s["k_scale"], v_scale=s["v_scale"]) if s["fp8"] else {}
    if s["kind"] == "rotate":
        P.rotary_embedding(s["out"], s["x"], s["positions"], s["frequencies"], layout=s["layout"],
                           magnitude=s["magnitude"])
        return [s["out"]]
    if s["kind"] == "append":
        call = P.rotary_reshape_and_cache_fp8 if s["fp8"] else P.rotary_reshape_and_cache
        call(s["q_out"], s["q"], s["key"], s["value"], *_pools(s), s["positions"], s["slots"], s["frequencies"],
             layout=s["layout"], magnitude=s["magnitude"])
        return [s["q_out"], *_pools(s)]
    if s["kind"] == "tree":
        s["workspace"] = P.paged_attention_tree(s["out"], s["q"], s["mask"], s["cu"], s["most"], s["k_cache"],
                                                s["v_cache"], s["block_tables"], s["context_lens"], SCALE,
                                                workspace=s["workspace"], **scales)
        return [s["out"]]
    if s["kind"] == "verify":
        P.speculative_verify(s["tokens_out"], s["path"], s["counts"], s["target"], s["tokens"], s["cu"], s["most"],
                             s["uniforms"], parents=s["parents"], draft_probs=s["draft"])
        return [s["tokens_out"], s["path"], s["counts"]]
    P.kv_compact_path(s["k_cache"], s["v_cache"], s["block_tables"], s["context_lens"], s["cu"], s["path"], s["counts"],
                      **scales)
    return _pools(s)


def _run_plain(s):
    return dict(rotate=_plain_rotate, append=_plain_append, tree=_plain_tree, verify=_plain_verify,
                compact=_plain_compact)[s["kind"]](s)


def _turned(s, x):
    """Rows [tokens][heads][dim] with their first values rotated, in 32 bits."""
    x, r = x.float(), s["rotary"]
    angle = s["positions"].double()[:, None] * s["angles"]  # far positions: 64 bits
    cos = (torch.cos(angle) * s["magnitude"]).float()[:, None]
    sin = (torch.sin(angle) * s["magnitude"]).float()[:, None]
    if s["layout"] == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., r:]], -1)
    a, b = x[..., 0:r:2], x[..., 1:r:2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), x[..., r:]], -1)


def _plain_rotate(s):
    return [_turned(s, s["x"]).bfloat16()]


def _plain_append(s):
    at = torch.where(s["slots"] < 0, s["blocks"] * BLOCK, s["slots"]).long()
    for n, x in (("k", _turned(s, s["key"])), ("v", s["value"].float())):
        if not s["fp8"]:
            s[n + "_all"][at // BLOCK, :, at % BLOCK] = x.bfloat16()
            continue
        a = x.abs().amax(-1).clamp(min=2.0 ** -100)
        most = torch.full_like(a, 448.0)  # a number over a tensor would be a reciprocal and a product
        # E4M3 codes are moved as bytes: indexing has no 8-bit float form.
        s[n + "_all"].view(torch.uint8)[at // BLOCK, :, at % BLOCK] = (x * (most / a)[..., None]).to(F8).view(torch.uint8)
        s[n + "_all_scale"][at // BLOCK, :, at % BLOCK] = a / most
    return [_turned(s, s["q"]).bfloat16(), *_pools(s)]


def _places(s, rows):
    """Each row's sequence, and its node."""
    r = torch.arange(rows, device="cuda")
    b = torch.searchsorted(s["cu"][1:].contiguous(), r.int(), right=True)
    return b, r - s["cu"][b].long()


def _plain_tree(s):
    rows, h, _ = s["q"].shape
    n, kv, most = s["context_lens"].numel(), s["k_cache"].shape[1], s["most"]
    b, node = _places(s, rows)
    q = torch.zeros(n, most, h, D, device="cuda")
    q[b, node] = s["q"].float()
    q = q.view(n, most, kv, h // kv, D).permute(0, 2, 1, 3, 4).reshape(n * kv, -1, D)
    mask = torch.zeros(n, most, dtype=torch.int64, device="cuda")
    mask[b, node] = s["mask"]
    pools = []
    for name in ("k", "v"):
        pool, blocks = s[name + "_cache"], s["block_tables"].long()
        x = (pool.view(torch.uint8)[blocks].view(F8).float() * s[name + "_scale"][blocks][..., None] if s["fp8"]
             else pool[blocks].float())
        pools.append(x.permute(0, 2, 1, 3, 4).reshape(n * kv, -1, D))
    score = torch.bmm(q, pools[0].transpose(1, 2)) * SCALE
    key = torch.arange(score.shape[-1], device="cuda")
    prefix = (s["context_lens"] - s["cu"].diff()).long()[:, None, None]
    bit = (key - prefix).clamp(0, 63)
    tree = ((mask[:, :, None] >> bit) & 1).bool() & (key - prefix < 64)
    seen = (key < prefix) | tree
    score = score.view(n, kv, most, h // kv, -1).masked_fill_(~seen[:, None, :, None], -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True).clamp(min=-1e30))
    total = p.sum(-1).view(n * kv, -1, 1)
    out = torch.bmm(p.view(n * kv, most * (h // kv), -1), pools[1]) / total.clamp(min=1e-30)
    out = out.view(n, kv, most, h // kv, D).transpose(1, 2).reshape(n, most, h, D)
    return [out[b, node].bfloat16()]


def _plain_verify(s):
    cu, most, n = s["cu"].long(), s["most"], s["counts"].numel()
    size, first = cu.diff(), cu[:-1]
    rows = s["tokens"].numel()
    cur = torch.zeros(n, dtype=torch.int64, device="cuda")
    rest = torch.ones(n, dtype=torch.float64, device="cuda")
    count = (size > 0).long()
    path = torch.full((n, most), -1, dtype=torch.int64, device="cuda")
    tokens = torch.full((n, most), -1, dtype=torch.int64, device="cuda")
    path[:, 0] = torch.where(size > 0, 0, -1)
    refused = torch.zeros(n, s["target"].shape[1], dtype=torch.bool, device="cuda")
    every = torch.arange(n, device="cuda")
    for j in range(1, most):
        row = (first + j).clamp(max=rows - 1)
        here = j < size
        up = torch.full_like(cur, j - 1) if s["parents"] is None else s["parents"][row].long()
        asked = here & (up == cur)
        token, u = s["tokens"][row].long(), s["uniforms"][row].double()
        at = (first + cur).clamp(max=rows - 1)
        p = s["target"][at, token].double()
        if s["draft"] is not None:
            yes = asked & (u * s["draft"][at, token].double() < p)
        else:
            p = torch.where(refused[every, token], 0.0, p)
            yes = asked & (u * rest < p)
            rest = torch.where(yes, 1.0, torch.where(asked, rest - p, rest))
            refused[every, token] |= asked
            refused &= ~yes[:, None]
        cur = torch.where(yes, j, cur)
        at = count.clamp(max=most - 1)
        path[every, at] = torch.where(yes, j, path[every, at])
        tokens[every, at - 1] = torch.where(yes, token, tokens[every, at - 1])
        count = count + yes
    at = (first + cur).clamp(max=rows - 1)
    p = s["target"][at].double()
    if s["draft"] is not None:
        last = cur + 1 == size
        weight = torch.where(last[:, None], p, (p - s["draft"][at].double()).clamp(min=0))
    else:
        weight = p.masked_fill(refused, 0)
    weight = torch.where(weight.sum(-1, keepdim=True) > 0, weight, p)
    below = weight.cumsum(-1)
    goal = s["uniforms"][first.clamp(max=rows - 1)].double() * below[:, -1]
    drawn = torch.searchsorted(below, goal[:, None], right=True).flatten()
    index = torch.arange(weight.shape[1], device="cuda")
    drawn = torch.minimum(drawn, torch.where(weight > 0, index, 0).amax(-1))
    at = (count - 1).clamp(min=0)
    tokens[every, at] = torch.where(size > 0, drawn, -1)
    return [tokens.int(), path.int(), count.int()]


def _plain_compact(s):
    path, size = s["path"].long(), s["cu"].diff().long()
    i = torch.arange(path.shape[1], device="cuda")
    b, i = ((i < s["counts"].long()[:, None]) & (i > 0)).nonzero(as_tuple=True)
    start = (s["context_lens"].long() - size)[b]
    src, dst = start + path[b, i], start + i
    src_block, dst_block = (s["block_tables"][b, x // BLOCK].long() for x in (src, dst))
    for name in ("k_cache", "v_cache", "k_scale", "v_scale"):
        if name in s:
            pool = s[name].view(torch.uint8) if s[name].dtype == F8 else s[name]
            pool[dst_block, :, dst % BLOCK] = pool[src_block, :, src % BLOCK]
    return _pools(s)


# ---- the definition in 64 bits --------------------------------------------------------

def _exact_turned(s, x):
    """Pair by pair: (a + ib) e^(i angle)."""
    x, r = x.double().clone(), s["rotary"]
    for i in range(r // 2):
        m, n = (i, i + r // 2) if s["layout"] == "half" else (2 * i, 2 * i + 1)
        angle = s["positions"].double() * s["angles"][i]
        turn = torch.polar(torch.full_like(angle, s["magnitude"]), angle)[:, None]
        z = torch.complex(x[..., m], x[..., n]) * turn
        x[..., m], x[..., n] = z.real, z.imag
    return x


def _exact_pool(s, name):
    pool = s[name + "_cache"].double()
    return pool * s[name + "_scale"].double()[..., None] if s["fp8"] else pool


def _exact_append(s):
    keep = (s["slots"] >= 0).nonzero().flatten()
    block, place = (f(s["slots"][keep].long(), BLOCK) for f in (torch.div, torch.remainder))
    block = block.floor().long()
    pools, scales = [], []
    for n, x in (("k", _exact_turned(s, s["key"])[keep]), ("v", s["value"][keep].double())):
        pool = s[n + "_cache"].double()
        if s["fp8"]:
            scale = torch.clamp(x.abs().max(-1).values, min=2.0 ** -100) / 448.0
            x = x / scale[..., None]
            held = s[n + "_scale"].double().clone()
            held[block, :, place] = scale
            scales.append(held)
        pool[block, :, place] = x
        pools.append(pool)
    return [_exact_turned(s, s["q"]), *pools, *scales]


def _exact_tree(case, s):
    nodes, parents, ctx, _ = _shape(case)
    group, kv = case["heads"] // case["kv"], case["kv"]
    out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    pools = [_exact_pool(s, n) for n in "kv"]
    row = 0
    for b, (n, c, tree) in enumerate(zip(nodes, ctx, parents)):
        seen = torch.zeros(n, c, dtype=torch.bool)
        seen[:, :c - n] = True
        for j in range(n):
            up = j
            while up >= 0:
                seen[j, c - n + up] = True
                up = tree[up]
        hide = torch.where(seen.cuda(), 0.0, -math.inf).double()
        blocks = s["block_tables"][b, :-(-c // BLOCK)].long()
        k, v = (p[blocks].transpose(0, 1).reshape(kv, -1, D)[:, :c] for p in pools)
        for g in range(kv):
            q = s["q"][row:row + n, g * group:(g + 1) * group].double()
            score = torch.einsum("ngd,cd->ngc", q, k[g]) * SCALE + hide[:, None]
            w = torch.exp(score - torch.logsumexp(score, -1, keepdim=True))
            out[row:row + n, g * group:(g + 1) * group] = torch.einsum("ngc,cd->ngd", w, v[g])
        row += n
    return [out]


def _exact_verify(case, s):
    """One sequence after the other, node by node."""
    nodes, parents, _, _ = _shape(case)
    most = max(nodes)
    tokens, uniforms = s["tokens"].tolist(), s["uniforms"].tolist()
    out_tokens, out_path, counts, row = [], [], [], 0
    for n, tree in zip(nodes, parents):
        path, words = [0], []
        while True:
            at, rest, gone, found = row + path[-1], 1.0, set(), None
            for j in [j for j in range(1, n) if tree[j] == path[-1]]:
                token, u = tokens[row + j], uniforms[row + j]
                p = 0.0 if token in gone else float(s["target"][at, token])
                other = float(s["draft"][at, token]) if s["draft"] is not None else rest
                if u * other < p:
                    found = j
                    break
                gone.add(token)
                rest -= p
            if found is None:
                break
            path.append(found)
            words.append(tokens[row + found])
        p = s["target"][row + path[-1]].double()
        w = p.clone()
        if s["draft"] is None:
            w[list(gone)] = 0.0
        elif path[-1] + 1 < n:
            w = torch.clamp(p - s["draft"][row + path[-1]].double(), min=0.0)
        if not w.sum() > 0:
            w = p
        below = torch.cumsum(w, 0)
        later = (below > uniforms[row] * below[-1]).nonzero().flatten()
        words.append(int(later[0]) if later.numel() else int(w.nonzero().max()))
        counts.append(len(path))
        out_path.append(path + [-1] * (most - len(path)))
        out_tokens.append(words + [-1] * (most - len(words)))
        row += n
    return [torch.tensor(x) for x in (out_tokens, out_path, counts)]


def _exact_compact(case, s):
    """Token by token in path order, every head at once."""
    nodes, _, ctx, paths = _shape(case)
    tables = s["block_tables"].tolist()
    src, dst = [], []
    for table, n, c, path in zip(tables, nodes, ctx, paths):
        for i, j in enumerate(path):
            src.append(table[(c - n + j) // BLOCK] * BLOCK + (c - n + j) % BLOCK)
            dst.append(table[(c - n + i) // BLOCK] * BLOCK + (c - n + i) % BLOCK)
    src, dst = torch.tensor(src, device="cuda"), torch.tensor(dst, device="cuda")
    out = []
    for pool in _pools(s):
        x = pool.double().transpose(1, 2).flatten(0, 1)
        x[dst] = x[src]
        out.append(x.unflatten(0, (-1, BLOCK)).transpose(1, 2).contiguous())
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "rotate":
        return [_exact_turned(s, s["x"])]
    if case["kind"] == "append":
        return _exact_append(s)
    if case["kind"] == "tree":
        return _exact_tree(case, s)
    if case["kind"] == "verify":
        return _exact_verify(case, s)
    return _exact_compact(case, s)
