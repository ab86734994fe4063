"""Cases of a decoding step's operators: norms of the query and key heads with
the rotary positions and the cache append, attention of requests that share a
prefix, and the draw of the next token under temperature, top-k, top-p and min-p.

``run`` computes a case in plain torch (32 bits, rounded once; sums along the
sorted vocabulary in 64) where ``own`` is false and calls
rank_adapter_apply_gb300.operators where it is true.
"""
import math

import numpy as np
import torch

own = False

_ops = None


def _framework():
    global _ops
    if _ops is None:
        from rank_adapter_apply_gb300 import operators
        _ops = operators
    return _ops


DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ---- cases ---------------------------------------------------------------------------
def listed():
    return [
        # a small decode step: eight tokens of q, k, v with norms of q and k; k and v go to the cache
        {"name": "norm 8 tokens", "op": "norm", "tokens": 8, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128,
         "interleaved": False, "each": False, "positions": 8192, "page": 64, "dtype": "bf16"},
        # a weight for each head, part of the head turned, interleaved, 32 bits, odd counts
        {"name": "norm 1021 part f32", "op": "norm", "tokens": 1021, "heads": 28, "kv_heads": 4, "dim": 80, "rot": 64,
         "interleaved": True, "each": True, "positions": 32768, "page": 16, "dtype": "f32"},
        # the prefill of several prompts with long positions
        {"name": "norm 16384 tokens", "op": "norm", "tokens": 16384, "heads": 64, "kv_heads": 8, "dim": 128,
         "rot": 128, "interleaved": False, "each": False, "positions": 131072, "page": 64, "dtype": "bf16"},
        # three requests at the start of their answers behind one short prompt: latency
        {"name": "prefix 3x1 of 777", "op": "prefix", "requests": 3, "nodes": 1, "groups": 1, "prefix": 777, "ctx": 40,
         "lone": False, "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "dtype": "bf16"},
        # two tenants' instructions before 64 conversations of ragged lengths
        {"name": "prefix 64x1 of 8192", "op": "prefix", "requests": 64, "nodes": 1, "groups": 2, "prefix": 8192,
         "ctx": 1000, "lone": False, "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "dtype": "bf16"},
        # drafted trees of up to seven nodes behind three prefixes, some requests without one; small pages, odd head size
        {"name": "prefix 37x7 of 3001", "op": "prefix", "requests": 37, "nodes": 7, "groups": 4, "prefix": 3001,
         "ctx": 700, "lone": True, "heads": 28, "kv_heads": 4, "dim": 96, "page": 16, "dtype": "bf16"},
        # a large batch over one long document
        {"name": "prefix 256x1 of 32768", "op": "prefix", "requests": 256, "nodes": 1, "groups": 1, "prefix": 32768,
         "ctx": 1024, "lone": False, "heads": 64, "kv_heads": 8, "dim": 128, "page": 64, "dtype": "bf16"},
        # 32 bits, as a small model or a check would run it
        {"name": "prefix 24x2 of 1024 f32", "op": "prefix", "requests": 24, "nodes": 2, "groups": 2, "prefix": 1024,
         "ctx": 200, "lone": False, "heads": 16, "kv_heads": 4, "dim": 64, "page": 32, "dtype": "f32"},
        # the next token of one request: latency
        {"name": "sample 1 v32000", "op": "sample", "rows": 1, "vocab": 32000, "filters": "mixed", "dtype": "f32"},
        # a batch whose tenants ask for different filters, an odd vocabulary, bf16 logits
        {"name": "sample 32 v100003", "op": "sample", "rows": 32, "vocab": 100003, "filters": "mixed", "dtype": "bf16"},
        # top-k alone over a ragged vocabulary
        {"name": "sample 77 v65537", "op": "sample", "rows": 77, "vocab": 65537, "filters": "top_k", "dtype": "bf16"},
        # a large batch over a large vocabulary, top-p alone
        {"name": "sample 256 v131072", "op": "sample", "rows": 256, "vocab": 131072, "filters": "top_p",
         "dtype": "f32"},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "prefix", "prefix", "sample"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "norm":
        dim = rng.choice([64, 80, 96, 128, 256])
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.randint(1, 8)
        most = 16384 * 10240 // ((heads + 2 * kv) * dim)
        return {"op": op, "tokens": _log(rng, 1, min(16384, most) if dtype == "bf16" else min(8192, most // 2)),
                "heads": heads, "kv_heads": kv, "dim": dim, "rot": rng.choice([dim, dim // 2]),
                "interleaved": rng.random() < 0.5, "each": rng.random() < 0.3,
                "positions": rng.choice([4096, 32768, 131072]), "page": rng.choice([16, 32, 64]), "dtype": dtype}
    if op == "prefix":
        requests = _log(rng, 1, 256)
        kv = rng.choice([2, 4, 8])
        nodes = rng.choice([1, 1, rng.randint(2, 16)])
        keys = 256 * 32768 // (requests * nodes)
        return {"op": op, "requests": requests, "nodes": nodes, "groups": min(requests, rng.choice([1, 1, 2, 3, 5])),
                "prefix": min(_log(rng, 16, 32768 if dtype == "bf16" else 4096), keys),
                "ctx": rng.choice([0, _log(rng, 1, 1024)]), "lone": rng.random() < 0.3, "heads": kv * rng.choice([1, 2, 4, 8]),
                "kv_heads": kv, "dim": rng.choice([64, 96, 128]), "page": rng.choice([16, 32, 64, 128]), "dtype": dtype}
    rows = _log(rng, 1, 256)
    return {"op": op, "rows": rows, "vocab": _log(rng, 1000, min(200000, 256 * 131072 // rows)),
            "filters": rng.choice(["plain", "top_k", "top_p", "mixed", "mixed"]), "dtype": rng.choice(["f32", "bf16"])}


def work(case):
    eb = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        t, hq, hk, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        table = min(t, case["positions"]) * case["rot"] * 4
        weights = eb * d * (hq + hk if case["each"] else 2)
        return {"bytes": 2 * eb * t * d * (hq + 2 * hk) + table + weights + 12 * t,
                "flops": t * (hq + hk) * (4 * d + 3 * case["rot"])}
    if case["op"] == "prefix":
        prefix, ctx, nodes, starts = _lengths(case)
        hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
        of_group = np.add.reduceat(nodes, starts[:-1])
        keys = int(prefix.sum() + ctx.sum() + nodes.sum())            # a group's prefix is read once
        pairs = int((prefix * of_group).sum() + (ctx * nodes).sum() + (nodes * (nodes + 1) // 2).sum())
        rows = int(nodes.sum())
        return {"bytes": 2 * eb * keys * hk * d + rows * hq * (2 * eb * d + 4), "flops": 4 * pairs * hq * d}
    rows, v = case["rows"], case["vocab"]
    # a row's noise is needed for every token where neither top-k, min-p nor a temperature of zero leaves few tokens
    noisy = sum(_kind(case, i) in ("plain", "top_p") for i in range(rows))
    return {"bytes": v * (rows * eb + noisy * 4) + 24 * rows, "flops": 4 * rows * v}


# ---- inputs --------------------------------------------------------------------------
def _lengths(case):
    """Prefix lengths of the groups; own context lengths and nodes of the requests; first request of each group."""
    b, g, c, n, p = case["requests"], case["groups"], case["ctx"], case["nodes"], case["prefix"]
    i, j = np.arange(b), np.arange(g)
    prefix = p - (j * 1237) % max(1, p // 2)
    if case["lone"]:
        prefix[-1] = 0                                                # the last group's requests share nothing
    ctx = c - (i * 7919) % max(1, c)
    nodes = np.where(i == 0, n, np.maximum(1, n - (i * 3) % max(1, n // 2 + 1)))
    return prefix.astype(np.int64), ctx.astype(np.int64), nodes.astype(np.int64), np.arange(g + 1) * b // g


def _kind(case, row):
    """The filters of a row: "plain", "top_k", "top_p", or by turns in a mixed batch."""
    if case["filters"] != "mixed":
        return case["filters"]
    return ("both", "top_p", "min_p", "greedy")[row % 4]


def _parents(b, n, r):
    """Parents [b, n] of random trees: a node's is one of the three nodes before it, the root's is -1."""
    back = r.randint(1, 4, size=(b, n))
    return np.maximum(np.arange(n) - back, np.minimum(np.arange(n) - 1, 0)).astype(np.int64)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    r = np.random.RandomState(seed % (1 << 31))
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    def on_gpu(a):
        return torch.from_numpy(np.ascontiguousarray(a)).to(dev)

    s = {"case": case}
    if case["op"] == "norm":
        t, hq, hk, d, rot, page = (case[k] for k in ("tokens", "heads", "kv_heads", "dim", "rot", "page"))
        qkv = (normal(t, (hq + 2 * hk) * d) * (0.2 + 3.0 * torch.rand((t, 1), generator=g, device=dev))).to(dt)
        s["q"] = qkv[:, :hq * d].view(t, hq, d)                       # one fused projection's rows, split
        s["k"] = qkv[:, hq * d:(hq + hk) * d].view(t, hk, d)
        s["v"] = qkv[:, (hq + hk) * d:].view(t, hk, d)
        s["q_weight"] = (1.0 + 0.3 * normal(*((hq, d) if case["each"] else (d,)))).to(dt)
        s["k_weight"] = (1.0 + 0.3 * normal(*((hk, d) if case["each"] else (d,)))).to(dt)
        s["positions"] = on_gpu(r.randint(0, case["positions"], size=t).astype(np.int32))
        freq = 500000.0 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)
        angle = torch.arange(case["positions"], device=dev, dtype=torch.float64)[:, None] * freq
        s["table"] = torch.cat([angle.cos(), angle.sin()], dim=1).float()
        pages = (t + page - 1) // page + 2
        s["k_cache"] = normal(pages, page, hk, d).to(dt)
        s["v_cache"] = normal(pages, page, hk, d).to(dt)
        s["slots"] = on_gpu(r.permutation(pages * page)[:t].astype(np.int64))
        return s
    if case["op"] == "prefix":
        hq, hk, d, page = (case[k] for k in ("heads", "kv_heads", "dim", "page"))
        prefix, ctx, nodes, groups = _lengths(case)
        b, total, most = len(ctx), int(nodes.sum()), int(nodes.max())
        shared = max(1, -(-int(prefix.max()) // page))
        per = max(1, -(-int((ctx + nodes).max()) // page))
        pages = r.permutation(len(prefix) * shared + b * per).astype(np.int32)
        s["q"] = normal(total, hq, d).to(dt)
        s["k_cache"] = normal(len(pages), page, hk, d).to(dt)
        s["v_cache"] = normal(len(pages), page, hk, d).to(dt)
        s["prefix_table"] = on_gpu(pages[:len(prefix) * shared].reshape(len(prefix), shared))
        s["page_table"] = on_gpu(pages[len(prefix) * shared:].reshape(b, per))
        s["prefix_lens"] = on_gpu(prefix.astype(np.int32))
        s["group_starts"] = on_gpu(groups.astype(np.int32))
        s["ctx_lens"] = on_gpu(ctx.astype(np.int32))
        s["node_starts"] = on_gpu(np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32))
        parents = _parents(b, most, r)
        seen = np.zeros((b, most), np.int64)                          # bit j: node j is the node or above it
        for i in range(most):
            up = np.where(parents[:, i] < 0, 0, seen[np.arange(b), np.maximum(parents[:, i], 0)])
            seen[:, i] = up | (1 << i)
        keep = np.arange(most)[None, :] < nodes[:, None]
        s["tree_mask"] = on_gpu(seen[keep].reshape(total, 1))
        return s
    rows, v = case["rows"], case["vocab"]
    # a bulk of unlikely tokens, some likely ones, rows of different sharpness
    logits = normal(rows, v) * 2.0
    first = torch.randint(0, v, (rows, 1), generator=g, device=dev)
    likely = (first + torch.arange(64, device=dev) * (v // 64)) % v
    logits.scatter_(1, likely, 4.0 + 8.0 * torch.rand((rows, 64), generator=g, device=dev))
    s["logits"] = (logits * (0.5 + torch.rand((rows, 1), generator=g, device=dev))).to(dt)
    s["noise"] = torch.empty((rows, v), device=dev).exponential_(generator=g).clamp_min_(1e-30)
    kinds = [_kind(case, i) for i in range(rows)]
    hot = r.uniform(0.6, 1.2, size=rows)
    k = np.minimum(r.choice([1, 20, 50, 200, 1000], size=rows), v)
    s["temperature"] = on_gpu(np.where([x == "greedy" for x in kinds], 0.0, hot).astype(np.float32))
    s["top_k"] = on_gpu(np.where([x in ("top_k", "both") for x in kinds], k, 0).astype(np.int32))
    s["top_p"] = on_gpu(np.where([x in ("top_p", "both") for x in kinds], r.uniform(0.7, 0.98, size=rows),
                                 1.0).astype(np.float32))
    s["min_p"] = on_gpu(np.where([x == "min_p" for x in kinds], 0.05, 0.0).astype(np.float32))
    for name in ("top_k", "top_p", "min_p"):                          # a filter that no row asks for is not passed
        if case["filters"] not in (name, "mixed"):
            s[name] = None
    return s


# ---- the operators ---------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if op == "norm":
        return _norm_own(state) if own else _norm_plain(state)
    if op == "prefix":
        return _prefix_own(state) if own else _prefix_plain(state)
    return _sample_own(state) if own else _sample_plain(state)


def _norm_own(s):
    q = _framework().norm_rope_append(s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], s["positions"], s["table"],
                                      s["k_cache"], s["v_cache"], s["slots"], eps=EPS,
                                      interleaved=s["case"]["interleaved"])
    return q, s["k_cache"], s["v_cache"]


def _prefix_own(s):
    return _framework().prefix_attention(s["q"], s["k_cache"], s["v_cache"], s["prefix_table"], s["prefix_lens"],
                                         s["group_starts"], s["page_table"], s["ctx_lens"], s["node_starts"],
                                         s["tree_mask"])


def _sample_own(s):
    return _framework().sample_tokens(s["logits"], s["noise"], s["temperature"], s["top_k"], s["top_p"], s["min_p"])


def _normed(x, weight, cos, sin, interleaved):
    rot = 2 * cos.shape[-1]
    x32 = x.float()
    y = x32 * torch.rsqrt(x32.square().mean(-1, keepdim=True) + EPS) * weight.float()
    a, b = y[..., :rot].unflatten(-1, (-1, 2) if interleaved else (2, -1)).unbind(-1 if interleaved else -2)
    turned = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1 if interleaved else -2).flatten(-2)
    return torch.cat([turned, y[..., rot:]], dim=-1).to(x.dtype)


def _norm_plain(s):
    cos, sin = s["table"][s["positions"].long()][:, None, :].chunk(2, dim=-1)
    way = s["case"]["interleaved"]
    q = _normed(s["q"], s["q_weight"], cos, sin, way)
    s["k_cache"].flatten(0, 1)[s["slots"]] = _normed(s["k"], s["k_weight"], cos, sin, way)
    s["v_cache"].flatten(0, 1)[s["slots"]] = s["v"]
    return q, s["k_cache"], s["v_cache"]


def _part(q, k, v, sees, scale):
    """Maximum, sum and weighted values of q [b, n, kv, g, d] over k, v [b, l, kv, d], where sees [b, n, l]."""
    score = torch.einsum("bnkgd,blkd->bnkgl", q, k) * scale
    score = score.masked_fill(~sees[:, :, None, None, :], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    p = (score - top).exp()
    return top, p.sum(-1, keepdim=True), torch.einsum("bnkgl,blkd->bnkgd", p, v)


def _prefix_plain(s):
    q, case = s["q"], s["case"]
    total, heads, dim = q.shape
    page, kv = s["k_cache"].shape[1:3]
    dev, scale = q.device, 1.0 / math.sqrt(dim)
    starts, ctx, groups = s["node_starts"].long(), s["ctx_lens"].long(), s["group_starts"].long()

    def gathered(cache, table):
        return cache[table.long()].flatten(1, 2).float()              # [b, keys, kv, dim]

    def rows_of(first, last, most):
        """Places [b, most] of the rows first .. last, and which of them there are."""
        at = first[:, None] + torch.arange(most, device=dev)
        return at.clamp(max=total - 1), at < last[:, None]

    q32 = q.float().view(total, kv, heads // kv, dim)
    # the prefixes, for all rows of a group at once
    _, _, nodes, first = _lengths(case)
    most_rows = int(np.add.reduceat(nodes, first[:-1]).max())
    at, real = rows_of(starts[groups[:-1]], starts[groups[1:]], most_rows)
    k = gathered(s["k_cache"], s["prefix_table"])
    sees = torch.arange(k.shape[1], device=dev)[None, None, :] < s["prefix_lens"].long()[:, None, None]
    shared = [x[real] for x in _part(q32[at], k, gathered(s["v_cache"], s["prefix_table"]),
                                     sees.expand(-1, most_rows, -1), scale)]
    # each request's own keys: its context, then its tree
    most = case["nodes"]
    at, real = rows_of(starts[:-1], starts[1:], most)
    k = gathered(s["k_cache"], s["page_table"])
    node = torch.arange(k.shape[1], device=dev)[None, :] - ctx[:, None]
    bit = (s["tree_mask"][at, 0][:, :, None] >> node.clamp(0, 63)[:, None, :]) & 1
    own_nodes = (starts[1:] - starts[:-1])[:, None]
    sees = (node < 0)[:, None, :] | ((node >= 0) & (node < own_nodes))[:, None, :] & (bit == 1)
    alone = [x[real] for x in _part(q32[at], k, gathered(s["v_cache"], s["page_table"]), sees, scale)]
    top = torch.maximum(shared[0], alone[0])
    f, h = (shared[0] - top).exp(), (alone[0] - top).exp()
    sums = shared[1] * f + alone[1] * h
    out = (shared[2] * f + alone[2] * h) / sums
    return out.reshape(total, heads, dim).to(q.dtype), (sums.log() + top).reshape(total, heads)


def _sample_plain(s):
    x = s["logits"].float()
    rows, v = x.shape
    t = s["temperature"][:, None]
    greedy = t <= 0
    z = (x - x.amax(1, keepdim=True)) * (1.0 / torch.where(greedy, 1.0, t))
    p = z.exp()
    by_value = x.sort(dim=1, descending=True, stable=True).indices        # of equal logits the lowest index first
    p_sorted = p.gather(1, by_value).double()
    before = p_sorted.cumsum(1) - p_sorted                            # mass of the tokens in front
    total = p_sorted.sum(1, keepdim=True)
    rank = torch.arange(v, device=x.device)[None, :]
    keep = torch.ones_like(p, dtype=torch.bool)
    if s["top_k"] is not None:
        k = s["top_k"][:, None]
        keep &= (rank < k) | (k <= 0)
    if s["top_p"] is not None:
        most = s["top_p"].double()[:, None]
        keep &= (before < most * total) | (most >= 1)
    if s["min_p"] is not None:
        keep &= p_sorted >= s["min_p"][:, None]
    keep &= ~greedy
    keep[:, 0] = True
    keep = torch.zeros_like(keep).scatter(1, by_value, keep)
    race = torch.where(keep, p / s["noise"], -1.0)
    token = torch.where(race == race.amax(1, keepdim=True), rank, v).amin(1)
    logprob = z.gather(1, token[:, None])[:, 0] - total[:, 0].log()
    return token.int(), logprob.float()


# ---- the definitions in 64 bits ----------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        half = case["rot"] // 2
        rows = s["table"].double()[s["positions"].long()]
        turn = torch.complex(rows[:, :half], rows[:, half:])[:, None, :]

        def turned(x, weight):
            y = x.double()
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / case["dim"] + EPS) * weight.double()
            if case["interleaved"]:
                z = torch.complex(y[..., 0:2 * half:2], y[..., 1:2 * half:2]) * turn
                y[..., 0:2 * half:2], y[..., 1:2 * half:2] = z.real, z.imag
            else:
                z = torch.complex(y[..., :half], y[..., half:2 * half]) * turn
                y[..., :half], y[..., half:2 * half] = z.real, z.imag
            return y
        k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
        where = (s["slots"] // case["page"], s["slots"] % case["page"])
        k_cache[where] = turned(s["k"], s["k_weight"])
        v_cache[where] = s["v"].double()
        return turned(s["q"], s["q_weight"]), k_cache, v_cache
    if case["op"] == "prefix":
        prefix, ctx, nodes, groups = _lengths(case)
        first = np.concatenate([[0], np.cumsum(nodes)])
        per_kv, dim, dev = case["heads"] // case["kv_heads"], case["dim"], s["q"].device
        out = torch.empty(s["q"].shape, dtype=torch.float64, device=dev)
        lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device=dev)

        def keys(cache, pages, count, h):
            return cache[:, :, h][pages.long()].flatten(0, 1)[:count].double()
        for j in range(len(prefix)):
            lo, hi = int(first[groups[j]]), int(first[groups[j + 1]])
            for h in range(case["kv_heads"]):
                q = s["q"][lo:hi, h * per_kv:(h + 1) * per_kv].double() / math.sqrt(dim)
                kp = keys(s["k_cache"], s["prefix_table"][j], int(prefix[j]), h)
                vp = keys(s["v_cache"], s["prefix_table"][j], int(prefix[j]), h)
                of_prefix = q.reshape(-1, dim) @ kp.t()                # [rows, prefix]
                own_scores, own_values, all_lse = [], [], torch.logsumexp(of_prefix, 1) if len(kp) else \
                    torch.full((of_prefix.shape[0],), -math.inf, dtype=torch.float64, device=dev)
                all_lse = all_lse.view(hi - lo, per_kv)
                for b in range(int(groups[j]), int(groups[j + 1])):
                    n, c, at = int(nodes[b]), int(ctx[b]), int(first[b])
                    kb = keys(s["k_cache"], s["page_table"][b], c + n, h)
                    score = (q[at - lo:at - lo + n].reshape(-1, dim) @ kb.t()).view(n, per_kv, c + n)
                    shown = torch.ones((n, c + n), dtype=torch.bool, device=dev)
                    bits = s["tree_mask"][at:at + n]
                    shown[:, c:] = ((bits >> torch.arange(n, device=dev)[None, :]) % 2) != 0
                    score = torch.where(shown[:, None, :], score, -math.inf)
                    own_scores.append(score)
                    own_values.append(keys(s["v_cache"], s["page_table"][b], c + n, h))
                    all_lse[at - lo:at - lo + n] = torch.logaddexp(all_lse[at - lo:at - lo + n], torch.logsumexp(score, -1))
                o = (torch.exp(of_prefix - all_lse.view(-1, 1)) @ vp).view(hi - lo, per_kv, dim)
                for b, score, values in zip(range(int(groups[j]), int(groups[j + 1])), own_scores, own_values):
                    at = int(first[b]) - lo
                    n = score.shape[0]
                    weight = torch.exp(score - all_lse[at:at + n, :, None])
                    o[at:at + n] += (weight.reshape(n * per_kv, -1) @ values).view(n, per_kv, dim)
                out[lo:hi, h * per_kv:(h + 1) * per_kv] = o
                lse[lo:hi, h * per_kv:(h + 1) * per_kv] = all_lse
        return out, lse
    tokens, logprobs = [], []
    for i in range(case["rows"]):
        x = s["logits"][i].double()
        t = float(s["temperature"][i])
        log_p = torch.log_softmax(x / (t if t > 0 else 1.0), 0)
        order = torch.argsort(-x, stable=True)
        n = case["vocab"]
        if t <= 0:
            n = 1
        if s["top_k"] is not None and int(s["top_k"][i]) > 0:
            n = min(n, int(s["top_k"][i]))
        sorted_p = log_p[order].exp()
        if s["top_p"] is not None and float(s["top_p"][i]) < 1:
            n = min(n, 1 + int((sorted_p.cumsum(0)[:-1] < float(s["top_p"][i])).sum()))
        if s["min_p"] is not None:
            n = min(n, max(1, int((sorted_p >= float(s["min_p"][i]) * sorted_p[0]).sum())))
        kept = order[:n].sort().values
        token = kept[(log_p[kept] - s["noise"][i].double()[kept].log()).argmax()]
        tokens.append(token)
        logprobs.append(log_p[token])
    return torch.stack(tokens).int(), torch.stack(logprobs)
