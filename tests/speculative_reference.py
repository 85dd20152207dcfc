"""A speculative decoding step's operators in 64 bits, written from their definitions."""
import math

import numpy as np
import torch


def frequencies(dim, base, scaling="none", factor=1.0, length=0, low=1.0, high=32.0):
    """Radians a position of each pair, and the magnitude."""
    if scaling == "ntk":
        base = base * factor ** (dim / (dim - 2))
    w = [base ** (-2.0 * i / dim) for i in range(dim // 2)]
    if scaling == "linear":
        w = [x / factor for x in w]
    if scaling == "by_parts":
        def pair(turns):  # the (fractional) pair that turns so often over `length`
            return dim * math.log(length / (2 * math.pi * turns)) / (2 * math.log(base))
        a, b = max(0, math.floor(pair(high))), min(dim - 1, math.ceil(pair(low)))
        for i, x in enumerate(w):
            ramp = min(1.0, max(0.0, (i - a) / max(b - a, 0.001)))
            w[i] = x / factor * ramp + x * (1 - ramp)
    if scaling == "by_wavelength":
        for i, x in enumerate(w):
            turns = length * x / (2 * math.pi)
            if turns < low:
                w[i] = x / factor
            elif turns <= high:
                s = (turns - low) / (high - low)
                w[i] = (1 - s) * x / factor + s * x
    return w, 0.1 * math.log(factor) + 1 if scaling == "by_parts" and factor > 1 else 1.0


def rotate(x, positions, w, layout, magnitude=1.0):
    """x [tokens, heads, dim] (any type) -> float64, positions a list."""
    y = x.double().cpu().clone()
    r = 2 * len(w)
    angle = torch.tensor([[(p * f) % (2 * math.pi) for f in w] for p in positions], dtype=torch.float64)
    cos, sin = (magnitude * f(angle)[:, None] for f in (torch.cos, torch.sin))
    first, second = (slice(0, r // 2), slice(r // 2, r)) if layout == "half" else (slice(0, r, 2), slice(1, r, 2))
    a, b = y[..., first].clone(), y[..., second].clone()
    y[..., first], y[..., second] = a * cos - b * sin, b * cos + a * sin
    return y


def ancestors(parents):
    """Bits of the nodes that each node sees (itself too); parents of one tree, -1 first."""
    out = []
    for j, up in enumerate(parents):
        out.append((out[up] if up >= 0 else 0) | 1 << j)
    return out


def as_int64(bits):
    return [b - (1 << 64) if b >> 63 else b for b in bits]


def tree_attention(q, masks, cu, k, v, tables, ctx, scale):
    """q [rows, heads, 128], k and v pools [blocks, kv, 16, 128] in any type (dequantised), masks a list of bits: float64
    [rows, heads, 128]; a row that sees nothing is zero."""
    q, k, v = (t.double().cpu() for t in (q, k, v))
    heads, kv = q.shape[1], k.shape[1]
    group = heads // kv
    out = torch.zeros_like(q)
    for b, c in enumerate(ctx):
        n = cu[b + 1] - cu[b]
        blocks = [int(x) for x in tables[b][: -(-c // 16)]]
        keys, values = (t[blocks].transpose(0, 1).reshape(kv, -1, 128)[:, :c] for t in (k, v))
        for i in range(n):
            seen = [j for j in range(c) if j < c - n or masks[cu[b] + i] >> (j - c + n) & 1]
            if not seen:
                continue
            for g in range(kv):
                s = q[cu[b] + i, g * group:(g + 1) * group] @ keys[g, seen].T * scale
                out[cu[b] + i, g * group:(g + 1) * group] = torch.softmax(s, -1) @ values[g, seen]
    return out


def verify(target, tokens, uniforms, cu, most, parents=None, draft=None):
    """(tokens_out, path, counts) as lists, from the definition."""
    target = target.double().cpu().numpy()
    target = np.clip(np.nan_to_num(target, nan=0.0, posinf=1.0, neginf=0.0), 0.0, 1.0)
    if draft is not None:
        draft = np.clip(np.nan_to_num(draft.double().cpu().numpy(), nan=0.0, posinf=1.0, neginf=0.0), 0.0, 1.0)
    vocab = target.shape[1]
    words_out, paths, counts = [], [], []
    for b in range(len(cu) - 1):
        row, n = cu[b], cu[b + 1] - cu[b]
        if n == 0:
            words_out.append([-1] * most)
            paths.append([-1] * most)
            counts.append(0)
            continue
        path, words = [0], []
        while True:
            cur, rest, gone, chosen = path[-1], 1.0, [], None
            for j in range(cur + 1, n):
                if (parents[row + j] if parents is not None else j - 1) != cur:
                    continue
                x, p = tokens[row + j], 0.0
                if 0 <= x < vocab and x not in gone:
                    p = target[row + cur, x]
                other = (draft[row + cur, x] if 0 <= x < vocab else 0.0) if draft is not None else rest
                if uniforms[row + j] * other < p:
                    chosen = j
                    break
                gone.append(x)
                rest -= p
            if chosen is None:
                break
            path.append(chosen)
            words.append(tokens[row + chosen])
        p = target[row + path[-1]]
        w = p.copy()
        if draft is None:
            w[[x for x in gone if 0 <= x < vocab]] = 0.0
        elif gone:
            w = np.maximum(p - draft[row + path[-1]], 0.0)
        if w.sum() <= 0:
            w = p
        if w.sum() <= 0:
            words.append(-1)
        else:
            below = np.cumsum(w)
            later = np.nonzero(below > uniforms[row] * below[-1])[0]
            words.append(int(later[0]) if len(later) else int(np.nonzero(w)[0].max()))
        words_out.append(words + [-1] * (most - len(words)))
        paths.append(path + [-1] * (most - len(path)))
        counts.append(len(path))
    return words_out, paths, counts


def random_tree(rng, n, reach=8):
    return [-1] + [rng.randint(max(0, j - reach), j - 1) for j in range(1, n)]
