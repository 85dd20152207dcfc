"""Whole speculative decoding steps: rotated append, attention of the trees, verification, compaction of the accepted path."""
import random

import pytest
import torch

import speculative_reference as R
from paged_kv_cache_95_gb300 import pagedkv as P

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
VOCAB, HEADS, KV, BLOCKS = 97, 12, 2, 40
SCALE = 128.0 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _lib(built_library):
    P.load_library()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Step:
    """The buffers that a server keeps, and one step on them.  Everything that changes between steps is device data."""

    def __init__(self, fp8, lens, most):
        self.fp8, self.most, self.seqs = fp8, most, len(lens)
        rows = self.seqs * most
        self.held = list(lens)  # cached tokens (the host's copy)
        rng = random.Random(5)
        ids = rng.sample(range(BLOCKS), BLOCKS)
        per = BLOCKS // self.seqs
        self.tables = [ids[b * per:(b + 1) * per] for b in range(self.seqs)]
        self.d_tables = i32(self.tables)
        shape = (BLOCKS, KV, 16, 128)
        g = torch.Generator(device="cuda")
        g.manual_seed(9)
        x = torch.randn(2, *shape, generator=g, device="cuda")
        if fp8:
            self.pools = [(t * 100).clamp(-448, 448).to(F8) for t in x] + [torch.full(shape[:3], 0.01, device="cuda") for _ in "kv"]
        else:
            self.pools = [t.clone() for t in x.bfloat16()]
        self.w, _ = P.rotary_frequencies(128, 10000.0)
        self.q, self.q_out, self.out = (torch.zeros(rows, HEADS, 128, dtype=torch.bfloat16, device="cuda") for _ in range(3))
        self.out = self.out.float()
        self.k, self.v = (torch.zeros(rows, KV, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.positions, self.slots, self.tokens, self.parents = (torch.zeros(rows, dtype=torch.int32, device="cuda")
                                                                 for _ in range(4))
        self.masks = torch.zeros(rows, dtype=torch.int64, device="cuda")
        self.cu, self.ctx = i32([0] * (self.seqs + 1)), i32([0] * self.seqs)
        self.target, self.uniforms = torch.zeros(rows, VOCAB, device="cuda"), torch.zeros(rows, device="cuda")
        self.words, self.path = (torch.zeros(self.seqs, most, dtype=torch.int32, device="cuda") for _ in range(2))
        self.counts = i32([0] * self.seqs)
        desc = P.cache_desc(self.pools[0])
        size = P.paged_attention_tree_workspace_size(self.seqs, HEADS, most, desc)
        self.workspace = torch.zeros(size, dtype=torch.uint8, device="cuda")

    def feed(self, seed):
        """The next step's drafts, as a drafter would leave them."""
        rng, g = random.Random(seed), torch.Generator(device="cuda")
        g.manual_seed(seed)
        n = [rng.choice([1, 2, self.most // 2, self.most]) for _ in range(self.seqs)]
        self.n, self.host = n, dict(cu=[0], parents=[], tokens=[], positions=[], slots=[], masks=[])
        h = self.host
        for b, count in enumerate(n):
            tree = R.random_tree(rng, count, reach=3)
            depth = []
            for up in tree:
                depth.append(depth[up] + 1 if up >= 0 else 0)
            h["cu"].append(h["cu"][-1] + count)
            h["parents"] += tree
            h["tokens"] += [rng.randrange(VOCAB) for _ in tree]
            h["positions"] += [self.held[b] + d for d in depth]
            h["slots"] += [self.tables[b][(self.held[b] + i) // 16] * 16 + (self.held[b] + i) % 16 for i in range(count)]
            h["masks"] += R.ancestors(tree)
        rows = h["cu"][-1]
        for name, to in (("parents", self.parents), ("tokens", self.tokens), ("positions", self.positions)):
            to[:rows] = i32(h[name])
        self.slots.fill_(-1)  # (padding)
        self.slots[:rows] = i32(h["slots"])
        self.masks[:rows] = torch.tensor(R.as_int64(h["masks"]), device="cuda")
        self.cu.copy_(i32(h["cu"]))
        self.ctx.copy_(i32([c + m for c, m in zip(self.held, n)]))
        for t in (self.q, self.k, self.v):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        logits = torch.randn(self.target.shape, generator=g, device="cuda")
        logits[:, :].scatter_add_(1, self.tokens.long().roll(-1)[:, None], torch.full_like(logits[:, :1], 4.0))
        self.target.copy_(torch.softmax(logits, -1))
        self.uniforms.copy_(torch.rand(self.uniforms.shape, generator=g, device="cuda"))

    def append_and_attend(self):
        scales = dict(k_scale=self.pools[2], v_scale=self.pools[3]) if self.fp8 else {}
        call = P.rotary_reshape_and_cache_fp8 if self.fp8 else P.rotary_reshape_and_cache
        call(self.q_out, self.q, self.k, self.v, *self.pools, self.positions, self.slots, self.w)
        P.paged_attention_tree(self.out, self.q_out, self.masks, self.cu, self.most, *self.pools[:2], self.d_tables, self.ctx,
                               SCALE, workspace=self.workspace, **scales)

    def verify_and_compact(self):
        scales = dict(k_scale=self.pools[2], v_scale=self.pools[3]) if self.fp8 else {}
        P.speculative_verify(self.words, self.path, self.counts, self.target, self.tokens, self.cu, self.most, self.uniforms,
                             parents=self.parents)
        P.kv_compact_path(*self.pools[:2], self.d_tables, self.ctx, self.cu, self.path, self.counts, **scales)

    def run(self):
        self.append_and_attend()
        self.verify_and_compact()

    def accept(self):
        self.held = [c + m for c, m in zip(self.held, self.counts.tolist())]

    def dense(self):
        """K and V as the numbers that they stand for."""
        if not self.fp8:
            return [t.double() for t in self.pools]
        return [t.float().double() * s.double()[..., None] for t, s in zip(self.pools[:2], self.pools[2:])]

    def bytes(self):
        return [t.clone().view(torch.uint8) for t in self.pools]


def bound(q, k, v, fp8):
    """As for the attention alone: fp32 sums of 128 products, two bf16 parts of a weight (FP8: fp16 with the value's scale)."""
    most = float(q.double().norm(dim=-1).max()) * float(k.norm(dim=-1).max())
    weight = 2 * most * SCALE * 128 * 2.0 ** -23 + 2.0 ** -15 + 2.0 ** -21 + (2.0 ** -11 if fp8 else 0)
    return 2 * weight * float(v.abs().max()) + 2.0 ** -20


@pytest.mark.parametrize("fp8", [False, True])
def test_steps_in_a_row(fp8):
    s = Step(fp8, [1, 30, 95, 16], 12)
    for seed in range(4):
        s.feed(seed)
        h = s.host
        rows = h["cu"][-1]
        s.append_and_attend()
        k, v = s.dense()
        # the drafts' rows in the pool: turned keys to a step of their type, values as they came
        turned = R.rotate(s.k[:rows], h["positions"], R.frequencies(128, 10000.0)[0], "half")
        step = 2.0 ** -4 if fp8 else 2.0 ** -8
        for row, slot in enumerate(h["slots"]):
            for pool, want in ((k, turned[row]), (v, s.v[row].double().cpu())):
                got = pool[slot // 16, :, slot % 16].cpu()
                # (a pair's rounding goes by its norm, at most sqrt 2 of the row's largest; E4M3 below 2^-6 steps by 2^-9 of 448)
                limit = step * want.abs() * (1 + 2.0 ** -8) + want.abs().amax(-1, keepdim=True) * (2.0 ** -9 / 448 * 4 + 2.0 ** -20)
                assert bool(((got - want).abs() <= limit).all())
        want = R.tree_attention(s.q_out[:rows], h["masks"], h["cu"], k, v, s.tables, s.ctx.tolist(), SCALE)
        limit = bound(s.q_out[:rows], k, v, fp8)
        assert float((s.out[:rows].double().cpu() - want).abs().max()) <= limit
        s.verify_and_compact()
        words, paths, counts = R.verify(s.target, h["tokens"], s.uniforms.tolist(), h["cu"], s.most, h["parents"])
        assert (s.words.tolist(), s.path.tolist(), s.counts.tolist()) == (words, paths, counts)
        # behind the compaction the accepted path is a chain: its last node's attention is that of a plain decode row
        k, v = s.dense()
        leaf = [h["cu"][b] + paths[b][counts[b] - 1] for b in range(s.seqs)]
        ends = [c + m for c, m in zip(s.held, counts)]
        chain = R.tree_attention(s.q_out[leaf], [1] * s.seqs, list(range(s.seqs + 1)), k, v, s.tables, ends, SCALE)
        assert float((s.out[leaf].double().cpu() - chain).abs().max()) <= limit
        s.accept()
    assert int(s.workspace[:4].view(torch.int32)) == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_a_captured_step_follows_the_device_data(fp8):
    lens = [3, 47, 64, 100]
    eager, captured = Step(fp8, lens, 9), Step(fp8, lens, 9)
    captured.feed(0)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    before = captured.bytes()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        captured.run()
    assert all(torch.equal(a, b) for a, b in zip(before, captured.bytes()))
    for seed in range(5):
        for s in (eager, captured):
            s.feed(seed)
        eager.run()
        graph.replay()
        rows = eager.host["cu"][-1]
        assert torch.equal(eager.out[:rows], captured.out[:rows]) and torch.equal(eager.words, captured.words)
        assert all(torch.equal(a, b) for a, b in zip(eager.bytes(), captured.bytes()))
        for s in (eager, captured):
            s.accept()
        assert eager.held == captured.held


@pytest.mark.parametrize("fp8", [False, True])
def test_a_pool_past_32_bits(fp8):
    """The same step, its blocks once in a small pool and once at the end of one of 2.3e9 values."""
    s = Step(fp8, [5, 60], 12)
    s.feed(9)
    s.uniforms.fill_(0)  # every draft stands but the first
    s.uniforms[[c + 1 for c, m in zip(s.host["cu"], s.n) if m > 1]] = 1 - 2.0 ** -24
    blocks = 560_000  # of 2 KV heads x 16 x 128 values
    shift = blocks - BLOCKS
    small, large = s.pools, []
    for t in small:
        x = torch.empty(blocks, *t.shape[1:], dtype=t.dtype, device="cuda")
        x[shift:].view(torch.uint8).copy_(t.view(torch.uint8))
        large.append(x)
    s.run()
    want = [s.out.clone(), s.words.clone(), s.path.clone(), *s.bytes()]
    s.pools, s.d_tables = large, s.d_tables + shift
    s.slots[s.slots >= 0] += shift * 16
    s.run()
    got = [s.out, s.words, s.path, *(t[shift:].view(torch.uint8) for t in large)]
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert any(node > i for path in s.path.tolist() for i, node in enumerate(path))  # (something moved)


def test_two_steps_at_once():
    """Two servers' steps on two streams, each with its own buffers: the bits of each alone."""
    steps = [Step(fp8, [70, 15, 40], 12) for fp8 in (False, True)]
    want = []
    for s in steps:
        s.feed(11)
        s.start = [t.clone() for t in s.pools]
        s.run()
        want.append([s.out.clone(), s.words.clone(), *s.bytes()])
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(10):
        for s in steps:
            s.out.fill_(7)
            s.words.fill_(7)
            for t, x in zip(s.pools, s.start):
                t.view(torch.uint8).copy_(x.view(torch.uint8))
        torch.cuda.synchronize()
        for s, stream in zip(steps, streams):
            with torch.cuda.stream(stream):
                s.run()
        torch.cuda.synchronize()
        for s, w in zip(steps, want):
            rows = s.host["cu"][-1]
            assert torch.equal(s.out[:rows], w[0][:rows]) and torch.equal(s.words, w[1])
            assert all(torch.equal(a, b) for a, b in zip(s.bytes(), w[2:]))
