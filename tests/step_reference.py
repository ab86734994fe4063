"""Plain 64-bit forms of the drafted-token step's operators (numpy, written from
the formulas), with the magnitudes that the tolerances of the tests are made of."""
import math

import numpy as np


def linear(x, qweight, scales, zeros, group):
    """(y, mass): mass[t][i] = sum_k |w[i][k] x[t][k]|, the scale of fp32 summation errors."""
    n = np.empty((qweight.shape[0], 2 * qweight.shape[1]))
    n[:, 0::2], n[:, 1::2] = qweight & 15, qweight >> 4
    z = 8.0 if zeros is None else np.repeat(zeros.astype(np.float64), group, 1)
    w = (n - z) * np.repeat(scales.astype(np.float64), group, 1)
    with np.errstate(all="ignore"):
        return x @ w.T, np.abs(x) @ np.abs(w).T


def rope_table(n_positions, rot_dim, base, scaling=None, factor=1.0, original=1.0, low_freq=1.0, high_freq=1.0):
    """cos and sin [n_positions, rot_dim / 2] in 64 bits."""
    mag = 1.0
    if scaling == "base":
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = []
    for j in range(rot_dim // 2):
        fj = base ** (-2.0 * j / rot_dim)
        if scaling == "linear":
            fj /= factor
        if scaling == "pieces":
            wave = 2 * math.pi / fj
            if wave > original / low_freq:
                fj /= factor
            elif wave >= original / high_freq:
                m = (original / wave - low_freq) / (high_freq - low_freq)
                fj = (1 - m) * fj / factor + m * fj
        if scaling == "yarn":
            def dim_of(turns):
                return rot_dim * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
            lo = max(math.floor(dim_of(high_freq)), 0)
            hi = min(math.ceil(dim_of(low_freq)), rot_dim - 1)
            ramp = min(max((j - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            fj = fj * (1 - ramp) + fj / factor * ramp
            mag = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
        f.append(fj)
    angle = np.arange(n_positions)[:, None] * np.array(f)
    return mag * np.cos(angle), mag * np.sin(angle)


def rope(x, cos, sin, interleaved):
    """(y, mass) of x [tokens, heads, dim] with cos, sin [tokens, rot / 2]; mass = |a| + |b| of the pair."""
    half = cos.shape[1]
    y, mass = x.copy(), np.zeros_like(x)
    i0 = np.arange(half) * 2 if interleaved else np.arange(half)
    i1 = i0 + 1 if interleaved else i0 + half
    a, b, c, s = x[..., i0], x[..., i1], cos[:, None, :], sin[:, None, :]
    y[..., i0], y[..., i1] = a * c - b * s, a * s + b * c
    mass[..., i0] = mass[..., i1] = np.abs(a) + np.abs(b)
    return y, mass


def tree_attention(q, k_cache, v_cache, page_table, ctx, starts, sees_node, scale):
    """(out, lse, mass, reach) for q [tokens, heads, dim]. sees_node(token, i, j): whether node i (row `token`) sees
    node j. mass = sum_p w_p |v_p|; reach = the largest scale * sum |q||k| over the keys a row sees. Rows of no
    request are NaN."""
    tokens, heads, dim = q.shape
    pages, page, kv_heads, _ = k_cache.shape
    out, mass = np.full(q.shape, np.nan), np.zeros(q.shape)
    lse, reach = np.full((tokens, heads), np.nan), np.zeros((tokens, heads))
    for b in range(len(ctx)):
        n = starts[b + 1] - starts[b]
        for i in range(n):
            t = starts[b] + i
            seen = list(range(max(ctx[b], 0))) + [max(ctx[b], 0) + j for j in range(n) if sees_node(t, i, j)]
            seen = [p for p in seen if p // page < page_table.shape[1]]
            where = [(page_table[b, p // page], p % page) for p in seen]
            where = [w for w in where if 0 <= w[0] < pages]
            if not where:
                out[t], lse[t] = 0.0, -np.inf
                continue
            at = tuple(np.array(where).T)
            for h in range(heads):
                g = h // (heads // kv_heads)
                k, v = k_cache[at[0], at[1], g], v_cache[at[0], at[1], g]
                s = scale * (k @ q[t, h])
                top = s.max()
                w = np.exp(s - top)
                lse[t, h] = top + np.log(w.sum())
                w /= w.sum()
                out[t, h], mass[t, h] = w @ v, w @ np.abs(v)
                reach[t, h] = abs(scale) * (np.abs(k) @ np.abs(q[t, h])).max()
    return out, lse, mass, reach


def verify(target, draft, tokens, parents, starts, uniforms, noise, max_path):
    """(path, n_accepted, next_token, margin): the sequential scheme with the residual normalised after every
    rejection. margin[b] = the smallest relative distance of request b's decisions from their other outcome."""
    requests, vocab = len(starts) - 1, target.shape[1]
    path = np.full((requests, max_path), -1, np.int64)
    count, chosen, margin = np.zeros(requests, np.int64), np.full(requests, -1, np.int64), np.full(requests, np.inf)
    for b in range(requests):
        at, n = starts[b], starts[b + 1] - starts[b]
        if n <= 0:
            continue
        node = 0
        while True:
            p = target[at + node]
            left, tried = p.copy(), 0
            went = None
            if count[b] < max_path:
                for c in range(node + 1, n):
                    x = tokens[at + c]
                    if parents[at + c] != node or not 0 <= x < vocab:
                        continue
                    q = draft[at + node] if draft is not None else np.eye(1, vocab, x)[0]
                    u, have = uniforms[at + c] * q[x], left[x]
                    margin[b] = min(margin[b], abs(u - have) / max(u, have, 1e-300))
                    if u < have:
                        went = c
                        break
                    tried += 1
                    if draft is None:
                        left[x] = 0.0
                    else:
                        left = np.maximum(left - q, 0.0)
                    left = left / left.sum() if left.sum() > 0 else left
            if went is None:
                break
            path[b, count[b]] = node = went
            count[b] += 1
        if not left.max() > 0:
            left = p
        if left.max() > 0:
            key = left / noise[b]
            order = np.argsort(-key, kind="stable")
            chosen[b] = order[0]
            if vocab > 1:
                margin[b] = min(margin[b], 1 - key[order[1]] / key[order[0]])
    return path, count, chosen, margin
