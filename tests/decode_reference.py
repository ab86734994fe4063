"""Plain 64-bit forms of a decoding step's operators (numpy, written from the formulas), with the magnitudes that the
tolerances of the tests are made of."""
import numpy as np

from tests import step_reference as ref


def norm_rope(x, weight, cos, sin, interleaved, eps):
    """(y, mass) of x [tokens, heads, dim], weight [dim], [heads, dim] or None; mass as step_reference.rope gives it, of
    the normed rows, and their magnitude past the turned part."""
    with np.errstate(all="ignore"):
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    y = y if weight is None else y * weight
    out, mass = ref.rope(y, cos, sin, interleaved)
    mass[..., 2 * cos.shape[1]:] = np.abs(y[..., 2 * cos.shape[1]:])
    return out, mass


def prefix_attention(q, k_cache, v_cache, prefix_table, prefix_lens, group_starts, page_table, ctx, starts, sees_node,
                     scale):
    """(out, lse, mass, reach) as step_reference.tree_attention gives them; rows of no request are NaN."""
    tokens, heads, dim = q.shape
    pages, page, kv_heads, _ = k_cache.shape
    out, mass = np.full(q.shape, np.nan), np.zeros(q.shape)
    lse, reach = np.full((tokens, heads), np.nan), np.zeros((tokens, heads))

    def places(table, seen):
        at = [(table[p // page], p % page) for p in seen if p // page < len(table)]
        return [w for w in at if 0 <= w[0] < pages]
    for b in range(len(ctx)):
        shared = []
        for g in range(len(prefix_lens)):
            if group_starts[g] <= b < group_starts[g + 1]:
                shared = places(prefix_table[g], range(max(prefix_lens[g], 0)))
        c, n = max(ctx[b], 0), starts[b + 1] - starts[b]
        for i in range(n):
            t = starts[b] + i
            where = shared + places(page_table[b], list(range(c)) + [c + j for j in range(n) if sees_node(t, i, j)])
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


def sample(logits, noise, temperature, top_k, top_p, min_p):
    """(tokens, logprobs, tol, margin) of finite logits [rows, vocab]. tol = what fp32 may be off in logprobs in units of
    2^-24; margin = the smallest relative distance of a row's decisions from their other outcome."""
    rows, vocab = logits.shape
    tokens, logprobs = np.zeros(rows, np.int64), np.zeros(rows)
    tol, margin = np.zeros(rows), np.full(rows, np.inf)
    for r in range(rows):
        t = 1.0 if temperature is None else float(temperature[r])
        greedy = not t > 0
        z = (logits[r] - logits[r].max()) / (1.0 if greedy else t)
        p = np.exp(z)
        total = p.sum()
        order = np.argsort(-logits[r], kind="stable")
        n = vocab
        front = np.cumsum(p[order]) - p[order]
        mass_edge = p_edge = np.full(vocab, np.inf)
        if top_k is not None and top_k[r] > 0:
            n = min(n, int(top_k[r]))
        if top_p is not None and float(top_p[r]) < 1:
            edge = float(top_p[r]) * total
            n = min(n, max(1, int((front < edge).sum())))
            mass_edge = np.abs(front - edge) / total
        if min_p is not None and float(min_p[r]) > 0:
            n = min(n, max(1, int((p[order] >= float(min_p[r])).sum())))
            p_edge = np.abs(p[order] - float(min_p[r])) / p[order]
        if greedy:
            n = 1
        key = (p / noise[r])[order]
        kept = np.argsort(-key[:n] + 0.0, kind="stable")
        best = kept[0]
        same = kept[key[kept] == key[best]]
        best = same[np.argmin(order[same])]
        tokens[r] = order[best]
        if n > 1:
            others = np.delete(key[:n], best)
            margin[r] = min(margin[r], 1 - others.max() / key[best]) if not greedy else margin[r]
        # the tokens that would win if they were kept, and the winner itself: how far from the border
        decisive = (key >= key[best]) & (np.arange(vocab) > 0)
        if decisive.any() and not greedy:
            margin[r] = min(margin[r], np.minimum(mass_edge, p_edge)[decisive].min())
        logprobs[r] = z[tokens[r]] - np.log(total)
        tol[r] = 8 + 4 * abs(z[tokens[r]]) + 4 * (p / total) @ np.abs(z)
    return tokens, logprobs, tol, margin
