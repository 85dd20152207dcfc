"""Measured cases of the latent-attention operators.

Latent attention keeps one shared row a token in the paged cache instead of keys
and values per head: a latent vector c (512 values) and a rotated key r (64
values).  The operators are the cache write (bf16, or E4M3 codes with one scale a
token), the read-back of cached rows, the absorbed attention over the paged rows
(decode and multi-token verify) and the expanded attention of a prefill chunk.

``run`` makes one pass: with ``own`` through the library's entry points, without
it in elementary torch operations, in 32 bits, rounded once at the end.
``exact`` computes the same from the definition in 64 bits.
"""
import math
import random

import torch

own = False

LATENT, ROPE, NOPE, VALUE, BLOCK = 512, 64, 128, 128, 16
ROW = LATENT + ROPE
SCALE = 1.0 / math.sqrt(NOPE + ROPE)  # the scale of the expanded head, which the absorbed form keeps
F8 = torch.float8_e4m3fn


def listed():
    return [
        # One decode step of 64 sequences (five of them padding): the smallest call, where the launch counts.
        dict(name="write step bf16", kind="write", fp8=False, tokens=64, padded=5),
        # Prefill of a long chunk into an 8-bit cache, quantised as it is written.
        dict(name="write chunk fp8", kind="write", fp8=True, tokens=16384, padded=0),
        # Ragged cached prefixes read back for the expanded form of a chunked prefill.
        dict(name="gather bf16", kind="gather", fp8=False, seqs=16, lo=200, hi=4096, lens=1),
        # Long prefixes of an 8-bit cache read back to bf16.
        dict(name="gather fp8", kind="gather", fp8=True, seqs=4, lo=16384, hi=32768, lens=2),
        # One sequence of a thousand tokens, few heads: the latency of a lone request.
        dict(name="decode one", kind="decode", fp8=False, seqs=1, lo=1000, hi=1000, lens=3, heads=16, q_per_seq=1),
        # The ragged batch of the library's benchmark (64 sequences of 512 to 4096 tokens, 32 heads).
        dict(name="decode ragged", kind="decode", fp8=False, seqs=64, lo=512, hi=4096, lens=4, heads=32, q_per_seq=1),
        # The long-context batch (8 sequences of 32K tokens, 64 heads).
        dict(name="decode long", kind="decode", fp8=False, seqs=8, lo=32768, hi=32768, lens=5, heads=64, q_per_seq=1),
        # All heads of a wide layer on one GPU: the products weigh as much as the reads.
        dict(name="decode wide", kind="decode", fp8=False, seqs=32, lo=2048, hi=8192, lens=6, heads=128, q_per_seq=1),
        # The ragged batch over an 8-bit cache.
        dict(name="decode ragged fp8", kind="decode", fp8=True, seqs=64, lo=512, hi=4096, lens=4, heads=32, q_per_seq=1),
        # Four draft positions a sequence verified over an 8-bit cache.
        dict(name="verify fp8", kind="decode", fp8=True, seqs=16, lo=4096, hi=16384, lens=7, heads=64, q_per_seq=4),
        # Short ragged chunks behind cached prefixes, as a mixed step of a server has them.
        dict(name="prefill chunks", kind="prefill", seqs=4, lo=33, hi=700, lens=8, prefix=2500, heads=32),
        # One long prompt prefilled whole.
        dict(name="prefill long", kind="prefill", seqs=1, lo=8192, hi=8192, lens=9, prefix=0, heads=32),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    kind = rng.choice(["write", "gather", "decode", "decode", "prefill"])
    if kind == "write":
        tokens = _spread(rng, 1, 16384)
        return dict(kind=kind, fp8=rng.random() < 0.5, tokens=tokens, padded=rng.randint(0, min(5, tokens - 1)))
    if kind == "gather":
        seqs = _spread(rng, 1, 64)
        hi = _spread(rng, 1, 98304 // seqs)
        return dict(kind=kind, fp8=rng.random() < 0.5, seqs=seqs, lo=max(1, hi // rng.randint(1, 8)), hi=hi,
                    lens=rng.randint(1, 1 << 30))
    if kind == "decode":
        heads, q_per_seq = rng.choice([8, 16, 32, 40, 64, 128]), rng.choice([1, 1, 2, 3, 4])
        seqs = _spread(rng, 1, 96)
        hi = _spread(rng, 16, 262144 * 64 // (seqs * max(64, heads * q_per_seq)))
        return dict(kind=kind, fp8=rng.random() < 0.5, seqs=seqs, lo=max(q_per_seq, hi // rng.randint(1, 8)), hi=hi,
                    lens=rng.randint(1, 1 << 30), heads=heads, q_per_seq=q_per_seq)
    heads, seqs = rng.choice([4, 8, 16, 32]), _spread(rng, 1, 8)
    hi = _spread(rng, 1, 4096 // seqs)
    return dict(kind=kind, seqs=seqs, lo=max(1, hi // rng.randint(1, 8)), hi=hi, lens=rng.randint(1, 1 << 30),
                prefix=rng.choice([0, _spread(rng, 1, 4096 // seqs)]), heads=heads)


def _lengths(case):
    """The case's lengths: of the contexts, or of the chunks and of the prefixes before them."""
    rng = random.Random(case["lens"])
    own_len = [rng.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]
    before = [rng.randint(0, case["prefix"]) for _ in own_len] if case.get("prefix") else [0] * len(own_len)
    return own_len, before


def work(case):
    row = LATENT + 2 * ROPE + 4 if case.get("fp8") else 2 * ROW  # a cached row as it is held
    if case["kind"] == "write":
        t = case["tokens"] - case["padded"]
        return dict(bytes=t * (2 * ROW + row) + 4 * case["tokens"], flops=t * LATENT * 3 if case["fp8"] else 0)
    if case["kind"] == "gather":
        t = sum(_lengths(case)[0])
        return dict(bytes=t * (row + 2 * ROW), flops=t * LATENT if case["fp8"] else 0)
    if case["kind"] == "decode":
        lens, k, h = _lengths(case)[0], case["q_per_seq"], case["heads"]
        seen = sum(n - k + 1 + i for n in lens for i in range(k))
        return dict(bytes=sum(lens) * row + len(lens) * k * h * 2 * (ROW + LATENT), flops=2 * h * seen * (ROW + LATENT))
    lens, before = _lengths(case)
    h, tq, tk = case["heads"], sum(lens), sum(lens) + sum(before)
    seen = sum(p * n + n * (n + 1) // 2 for n, p in zip(lens, before))
    return dict(bytes=2 * (tq * h * (NOPE + ROPE + VALUE) + tk * (h * (NOPE + VALUE) + ROPE)),
                flops=2 * h * seen * (NOPE + ROPE + VALUE))


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


def _pool(gen, blocks, fp8):
    """A pool of cached rows: normal latents (they are normalised before they are kept) and rotated keys.  One
    more block lies behind the pool, where the plain form puts padding tokens."""
    s = {}
    if not fp8:
        s["all"] = _normal(gen, blocks + 1, BLOCK, ROW)
        s["cache"] = s["all"][:blocks]
        return s
    x = _normal(gen, blocks + 1, BLOCK, LATENT).float()
    a = x.abs().amax(-1, keepdim=True)
    s["all"] = (x * (448.0 / a)).to(F8)
    s["all_rope"] = _normal(gen, blocks + 1, BLOCK, ROPE)
    s["all_scale"] = (a / 448.0).squeeze(-1).contiguous()
    s["cache"], s["rope_cache"], s["cache_scale"] = (s[n][:blocks] for n in ("all", "all_rope", "all_scale"))
    return s


def _tables(gen, s, lens):
    """Block tables over permuted blocks."""
    need = [-(-n // BLOCK) for n in lens]
    perm = torch.randperm(sum(need), generator=gen, device="cuda").int()
    wide = max(need)
    col = torch.arange(wide, device="cuda")
    at = torch.tensor(_starts(need)[:-1], device="cuda")[:, None] + col
    have = col < torch.tensor(need, device="cuda")[:, None]
    s["block_tables"] = torch.where(have, perm[at.clamp(max=sum(need) - 1)], 0).int().contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    kind = case["kind"]
    if kind == "write":
        t = case["tokens"]
        blocks = -(-t // BLOCK) + 64
        s = _pool(gen, blocks, case["fp8"])
        x = _normal(gen, t, ROW)  # one projection gives both parts: they are slices of its rows
        s["latent"], s["rope"] = x[:, :LATENT], x[:, LATENT:]
        slots = torch.randperm(blocks * BLOCK, generator=gen, device="cuda")[:t].int()
        if case["padded"]:
            slots[t - case["padded"]:] = -1
        s["slots"], s["blocks"] = slots, blocks
    elif kind == "gather":
        lens = _lengths(case)[0]
        s = _pool(gen, sum(-(-n // BLOCK) for n in lens), case["fp8"])
        _tables(gen, s, lens)
        s["cu_lens"] = _i32(_starts(lens))
        s["out"] = torch.empty(sum(lens), ROW, dtype=torch.bfloat16, device="cuda")
    elif kind == "decode":
        lens, k, h = _lengths(case)[0], case["q_per_seq"], case["heads"]
        s = _pool(gen, sum(-(-n // BLOCK) for n in lens), case["fp8"])
        _tables(gen, s, lens)
        s["context_lens"], s["q_per_seq"] = _i32(lens), k
        # The absorbed query comes out of a product over heads: [heads][rows][512] seen as [rows][heads][512].
        s["q_latent"] = _normal(gen, h, len(lens) * k, LATENT).transpose(0, 1)
        s["q_rope"] = _normal(gen, len(lens) * k, h, ROPE)
        s["out"] = torch.empty(len(lens) * k, h, LATENT, dtype=torch.bfloat16, device="cuda")
    else:
        lens, before = _lengths(case)
        whole = [n + p for n, p in zip(lens, before)]
        h = case["heads"]
        s = dict(q=_normal(gen, sum(lens), h, NOPE + ROPE))
        kv = _normal(gen, sum(whole), h, NOPE + VALUE)  # one up-projection gives both
        s["k_nope"], s["v"] = kv[..., :NOPE], kv[..., NOPE:]
        s["k_rope"] = _normal(gen, sum(whole), ROW)[:, LATENT:]  # lies in the rows read back
        s["cu_q_lens"], s["cu_k_lens"] = _i32(_starts(lens)), _i32(_starts(whole))
        s["max_q_len"], s["max_k_len"] = max(lens), max(whole)
        s["out"] = torch.empty(sum(lens), h, VALUE, dtype=torch.bfloat16, device="cuda")
    s["kind"], s["fp8"], s["workspace"] = kind, bool(case.get("fp8")), None
    return s


# ---- one pass -----------------------------------------------------------------------

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from paged_kv_cache_95_gb300 import pagedkv as P
    f8 = dict(rope_cache=s["rope_cache"], cache_scale=s["cache_scale"]) if s["fp8"] else {}
    if s["kind"] == "write":
        if s["fp8"]:
            P.latent_reshape_and_cache_fp8(s["latent"], s["rope"], s["cache"], s["rope_cache"], s["cache_scale"],
                                           s["slots"])
            return [s["cache"], s["rope_cache"], s["cache_scale"]]
        P.latent_reshape_and_cache(s["latent"], s["rope"], s["cache"], s["slots"])
        return [s["cache"]]
    if s["kind"] == "gather":
        P.latent_gather(s["out"], s["cache"], s["block_tables"], s["cu_lens"], **f8)
        return [s["out"]]
    if s["kind"] == "decode":
        s["workspace"] = P.latent_attention_decode(s["out"], s["q_latent"], s["q_rope"], s["cache"], s["block_tables"],
                                                   s["context_lens"], SCALE, workspace=s["workspace"],
                                                   q_per_seq=s["q_per_seq"], **f8)
        return [s["out"]]
    s["workspace"] = P.latent_attention_prefill_chunk(s["out"], s["q"], s["k_nope"], s["v"], s["k_rope"],
                                                      s["cu_q_lens"], s["cu_k_lens"], s["max_q_len"], SCALE,
                                                      workspace=s["workspace"])
    return [s["out"]]


def _run_plain(s):
    return dict(write=_plain_write, gather=_plain_gather, decode=_plain_decode, prefill=_plain_prefill)[s["kind"]](s)


def _plain_write(s):
    at = torch.where(s["slots"] < 0, s["blocks"] * BLOCK, s["slots"]).long()
    if not s["fp8"]:
        s["all"].view(-1, ROW)[at] = torch.cat([s["latent"], s["rope"]], 1)
        return [s["cache"]]
    x = s["latent"].float()
    a = x.abs().amax(-1).clamp(min=2.0 ** -100)
    # E4M3 codes are moved as bytes: indexing has no 8-bit float form.
    most = torch.full_like(a, 448.0)  # a number over a tensor would be a reciprocal and a product
    s["all"].view(torch.uint8).view(-1, LATENT)[at] = (x * (most / a)[:, None]).to(F8).view(torch.uint8)
    s["all_scale"].view(-1)[at] = a / most
    s["all_rope"].view(-1, ROPE)[at] = s["rope"]
    return [s["cache"], s["rope_cache"], s["cache_scale"]]


def _rows(s, at):
    """Cached rows in 32 bits, the latent dequantised."""
    if not s["fp8"]:
        return s["cache"].reshape(-1, ROW)[at].float()
    codes = s["cache"].view(torch.uint8).reshape(-1, LATENT)[at].view(F8).float()
    latent = codes * s["cache_scale"].reshape(-1)[at][..., None]
    return torch.cat([latent, s["rope_cache"].reshape(-1, ROPE)[at].float()], -1)


def _owner(cu, total):
    """Each row's sequence and place in it."""
    r = torch.arange(total, device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), r.int(), right=True)
    return b, r - cu[b].long()


def _plain_gather(s):
    b, pos = _owner(s["cu_lens"], s["out"].shape[0])
    at = s["block_tables"][b, pos // BLOCK].long() * BLOCK + pos % BLOCK
    return [_rows(s, at).bfloat16()]


def _plain_decode(s):
    k, (rows, h, _) = s["q_per_seq"], s["q_latent"].shape
    n = rows // k
    at = s["block_tables"].long()[:, :, None] * BLOCK + torch.arange(BLOCK, device="cuda")
    kv = _rows(s, at.reshape(n, -1))
    q = torch.cat([s["q_latent"], s["q_rope"]], -1).float().reshape(n, k * h, ROW)
    score = torch.bmm(q, kv.transpose(1, 2)) * SCALE
    last = s["context_lens"].long()[:, None] - k + torch.arange(k, device="cuda")  # each row's last visible key
    hide = torch.arange(kv.shape[1], device="cuda") > last[:, :, None]
    score = score.view(n, k, h, -1).masked_fill(hide[:, :, None], -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    out = torch.bmm(p.view(n, k * h, -1), kv[..., :LATENT]) / p.sum(-1).view(n, k * h, 1)
    return [out.view(rows, h, LATENT).bfloat16()]


def _plain_prefill(s):
    cq, ck, lq, lk = s["cu_q_lens"].long(), s["cu_k_lens"].long(), s["max_q_len"], s["max_k_len"]
    tq, h, _ = s["q"].shape
    n, tk = cq.numel() - 1, s["k_nope"].shape[0]
    i, j = torch.arange(lq, device="cuda"), torch.arange(lk, device="cuda")
    q = s["q"][(cq[:-1, None] + i).clamp(max=tq - 1)].float().transpose(1, 2)
    at = (ck[:-1, None] + j).clamp(max=tk - 1)
    key = torch.cat([s["k_nope"][at], s["k_rope"][at][:, :, None].expand(-1, -1, h, -1)], -1).float().transpose(1, 2)
    score = torch.matmul(q, key.transpose(2, 3)) * SCALE
    first = (ck[1:] - ck[:-1]) - (cq[1:] - cq[:-1])  # the position of a chunk's first row
    score.masked_fill_((j > first[:, None, None] + i[:, None])[:, None], -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    out = torch.matmul(p, s["v"][at].float().transpose(1, 2)) / p.sum(-1, keepdim=True)
    b, pos = _owner(s["cu_q_lens"], tq)
    return [out.transpose(1, 2)[b, pos].bfloat16()]


# ---- the definition in 64 bits --------------------------------------------------------

def _exact_pool(s):
    """Every cached row in 64 bits, in slot order."""
    if s["fp8"]:
        latent = s["cache"].double().reshape(-1, LATENT) * s["cache_scale"].double().reshape(-1, 1)
        return torch.cat([latent, s["rope_cache"].double().reshape(-1, ROPE)], 1)
    return s["cache"].double().reshape(-1, ROW)


def _exact_sequence(s, pool, b, length):
    blocks = s["block_tables"][b, : -(-length // BLOCK)].tolist()
    return torch.cat([pool[BLOCK * x: BLOCK * x + BLOCK] for x in blocks])[:length]


def _weigh(score, value):
    e = torch.exp(score - torch.logsumexp(score, -1, keepdim=True))
    return e @ value


def exact(case, seed):
    s = prepare(case, seed)
    if s["kind"] == "write":
        keep = (s["slots"] >= 0).nonzero().flatten()
        at = s["slots"][keep].long()
        if not s["fp8"]:
            pool = s["cache"].double().reshape(-1, ROW)
            pool[at, :LATENT], pool[at, LATENT:] = s["latent"][keep].double(), s["rope"][keep].double()
            return [pool.view(-1, BLOCK, ROW)]
        x = s["latent"][keep].double()
        scale = torch.clamp(x.abs().max(1).values, min=2.0 ** -100) / 448.0
        codes, ropes = s["cache"].double().reshape(-1, LATENT), s["rope_cache"].double().reshape(-1, ROPE)
        scales = s["cache_scale"].double().reshape(-1)
        codes[at], ropes[at], scales[at] = x / scale[:, None], s["rope"][keep].double(), scale
        return [codes.view(-1, BLOCK, LATENT), ropes.view(-1, BLOCK, ROPE), scales.view(-1, BLOCK)]
    lens, before = _lengths(case)
    if s["kind"] == "gather":
        pool = _exact_pool(s)
        return [torch.cat([_exact_sequence(s, pool, b, n) for b, n in enumerate(lens)])]
    if s["kind"] == "decode":
        pool, k, h, out = _exact_pool(s), case["q_per_seq"], case["heads"], []
        for b, n in enumerate(lens):
            c = _exact_sequence(s, pool, b, n)
            for i in range(k):
                seen, r = c[: n - k + 1 + i], b * k + i
                score = s["q_latent"][r].double() @ seen[:, :LATENT].T + s["q_rope"][r].double() @ seen[:, LATENT:].T
                out.append(_weigh(score * SCALE, seen[:, :LATENT]))
        return [torch.stack(out)]
    out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    q0 = k0 = 0
    for n, p in zip(lens, before):
        row, col = torch.arange(n, device="cuda") + p, torch.arange(n + p, device="cuda")
        future = torch.where(col[None] <= row[:, None], 0.0, -math.inf).double()
        r = s["k_rope"][k0:k0 + n + p].double()
        for g in range(case["heads"]):
            q, key = s["q"][q0:q0 + n, g].double(), s["k_nope"][k0:k0 + n + p, g].double()
            score = (q[:, :NOPE] @ key.T + q[:, NOPE:] @ r.T) * SCALE + future
            out[q0:q0 + n, g] = _weigh(score, s["v"][k0:k0 + n + p, g].double())
        q0, k0 = q0 + n, k0 + n + p
    return [out]
