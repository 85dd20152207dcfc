"""Plain 64-bit forms of the latent-attention operators (torch on the CPU), the
inputs of their tests, and the tolerances, derived from the roundings the kernels make.

Rounding a value to a type is off by at most ``finfo(type).eps / 2`` relative to it:
2^-8 for bf16, 2^-24 for fp32, 2^-4 for e4m3.
"""
import torch

LATENT, ROPE, ROW, BLOCK = 512, 64, 576, 16
SCALE = 192.0 ** -0.5
NAN = float("nan")


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def normal(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).bfloat16()


def quantise(x):
    """E4M3 codes and scales of latent rows, each step one fp32 operation (a number over a
    tensor is a reciprocal and a product in torch: hence the tensor of 448)."""
    x = x.float()
    a = x.abs().amax(-1).clamp(min=2.0 ** -100)
    most = torch.full_like(a, 448.0)
    return (x * (most / a)[..., None]).to(torch.float8_e4m3fn), a / most


class Pool:
    """A paged latent pool on the CPU whose unowned slots hold NaN: sequences of `lens`
    tokens over permuted blocks; `rows` are the cached values in 64 bits, in slot order."""

    def __init__(self, seed, lens, fp8=False, spare=3, table_pad=2, latent_scale=1.0):
        g = gen(seed)
        need = [(max(n, 0) + BLOCK - 1) // BLOCK for n in lens]
        self.fp8, self.lens, self.num_blocks = fp8, list(lens), sum(need) + spare
        perm = torch.randperm(self.num_blocks, generator=g)
        self.max_blocks = max(max(need), 1) + table_pad
        self.tables = torch.full((len(lens), self.max_blocks), -7, dtype=torch.int32)  # never read past a length
        owned = torch.zeros(self.num_blocks * BLOCK, dtype=torch.bool)
        at = 0
        for b, n in enumerate(need):
            ids = perm[at:at + n]
            at += n
            self.tables[b, :n] = ids.int()
            slots = (ids[:, None] * BLOCK + torch.arange(BLOCK)).flatten()[:max(lens[b], 0)]
            owned[slots] = True
        total = self.num_blocks * BLOCK
        latent, rope = normal(g, total, LATENT, scale=latent_scale), normal(g, total, ROPE)
        rope[~owned] = NAN
        if fp8:
            codes, scale = quantise(latent)
            codes = codes.view(torch.uint8)
            codes[~owned] = 0x7F  # NaN
            scale[~owned] = NAN
            self.cache = codes.view(self.num_blocks, BLOCK, LATENT)
            self.rope_cache = rope.view(self.num_blocks, BLOCK, ROPE)
            self.cache_scale = scale.view(self.num_blocks, BLOCK)
            latent = codes.view(torch.float8_e4m3fn).double() * scale.double()[:, None]
        else:
            latent[~owned] = NAN
            self.cache = torch.cat([latent, rope], 1).view(self.num_blocks, BLOCK, ROW)
        self.rows = torch.cat([latent.double(), rope.double()], 1)

    def sequence(self, b, n=None):
        n = self.lens[b] if n is None else n
        slots = (self.tables[b].long()[:, None] * BLOCK + torch.arange(BLOCK)).flatten()[:n]
        return self.rows[slots]

    def device(self):
        """Keyword arguments of the entry points: the pool on the GPU."""
        d = dict(cache=self.cache.cuda())
        if self.fp8:
            d.update(rope_cache=self.rope_cache.cuda(), cache_scale=self.cache_scale.cuda())
        return d


def attend(q, keys, values, visible):
    """softmax(q keys^T * SCALE) values over each row's first `visible` keys, and the same
    mean of |values| (the size that a relative error of a weight is multiplied with).
    A key whose row is None-like (not finite) must not be visible."""
    score = (q @ keys.T) * SCALE
    score[torch.arange(keys.shape[0])[None, :] >= visible[:, None]] = -float("inf")
    w = torch.softmax(score, -1)
    return w @ values, w @ values.abs()


def decode(q_latent, q_rope, pool, q_per_seq, skip_blocks=()):
    """The absorbed form: (out, tolerance) [rows, heads, 512].  Blocks of `skip_blocks`
    ((sequence, index) pairs) contribute nothing."""
    rows, heads, _ = q_latent.shape
    out = torch.zeros(rows, heads, LATENT, dtype=torch.float64)
    tol = torch.zeros_like(out)
    q = torch.cat([q_latent.double(), q_rope.double()], -1)
    for b, n in enumerate(pool.lens):
        if n < 1 or n < q_per_seq:
            continue
        bad = {i for s, i in skip_blocks if s == b}
        keep = torch.tensor([j for j in range(n) if j // BLOCK not in bad], dtype=torch.long)
        slots = (pool.tables[b].long()[:, None].clamp(min=0) * BLOCK + torch.arange(BLOCK)).flatten()[:n]
        c = pool.rows[slots[keep]]
        for i in range(q_per_seq):
            r = b * q_per_seq + i
            seen = int((keep <= n - q_per_seq + i).sum())
            if seen == 0:
                continue
            s = c[:seen]
            o, size = attend(q[r], s, s[:, :LATENT], torch.full((heads,), seen))
            out[r] = o
            tol[r] = size * weight_error(q[r], s, pool.fp8)
            if pool.fp8:
                # The weights that multiply the codes, w_j s_j, are pairs of E4M3 codes in which the largest is at
                # least 2^2 and the smallest step is 2^-9: each is off by up to 2^-10 / 2^2 of the largest.
                scale = s[:, :LATENT].abs().amax(1) / 448  # of a row that quantise() made: exact to rounding
                w = torch.softmax((q[r] @ s.T) * SCALE, -1)
                codes = (s[:, :LATENT].abs() / scale.clamp(min=1e-300)[:, None]).sum(0)
                tol[r] += (w * scale).amax(-1)[:, None] * 2.0 ** -12 * 1.01 * codes[None]
    return out, tol


def weight_error(q, keys, fp8=False):
    """Relative error of a row's softmax weights, numerator and sum: each weight rounded to bf16
    (over an FP8 pool: to a pair of E4M3 codes) 2^-8, twice; exponentials 2^-12; scores
    accumulated in fp32 over n products, n 2^-24 of the sum of their sizes, twice; over an
    FP8 pool the query held as a pair of E4M3 codes, the largest above 224, in steps of 2^-9:
    2^-10 / 224 of its largest value."""
    size = SCALE * (q.abs() @ keys.abs().T).amax(-1)
    score = q.shape[-1] * 2.0 ** -24 * size
    if fp8:
        score = score + SCALE * 2.0 ** -10 / 224 * q[:, :LATENT].abs().amax(-1) * keys[:, :LATENT].abs().sum(-1).max()
    return (2 * 2.0 ** -8 + 2.0 ** -12 + 2 * score)[:, None]


def expanded(q, k_nope, v, k_rope, q_lens, k_lens):
    """The expanded form: (out, tolerance) [total_q, heads, 128]."""
    tq, heads, _ = q.shape
    out = torch.zeros(tq, heads, 128, dtype=torch.float64)
    tol = torch.zeros_like(out)
    q0 = k0 = 0
    for lq, lk in zip(q_lens, k_lens):
        if 0 < lq <= lk:
            for h in range(heads):
                key = torch.cat([k_nope[k0:k0 + lk, h], k_rope[k0:k0 + lk]], -1).double()
                qq = q[q0:q0 + lq, h].double()
                o, size = attend(qq, key, v[k0:k0 + lk, h].double(), torch.arange(lq) + lk - lq + 1)
                out[q0:q0 + lq, h] = o
                tol[q0:q0 + lq, h] = size * weight_error(qq, key)
        q0, k0 = q0 + lq, k0 + lk
    return out, tol


def assert_within(got, ref, tol, what=""):
    """|got - ref| <= tol, elementwise; a bf16 result is rounded once more."""
    rounding = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -23
    got = got.detach().cpu().double()
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    over = (got - ref).abs() - (tol * (1 + rounding) + rounding * ref.abs() + 1e-30)
    at = int(over.argmax())
    assert over.max() <= 0, (f"{what}: element {at} is {got.flatten()[at]:.6g}, {ref.flatten()[at]:.6g} +- "
                             f"{tol.flatten()[at]:.3g} expected")
