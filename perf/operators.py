"""Cases of the drafted-token step's operators: the 4-bit base product, rotary
positions with the cache append, attention of drafted trees over the paged
cache, and the verification of the drafts.

``run`` computes a case in plain torch (32 bits, rounded once) where ``own`` is
false and calls rank_adapter_apply_gb300.operators where it is true.
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


# ---- cases ---------------------------------------------------------------------------
def listed():
    return [
        # one token of one request through a 4096-wide projection: latency
        {"name": "linear 1x4096x4096", "op": "linear", "tokens": 1, "d_in": 4096, "d_out": 4096, "group": 128,
         "zeros": False, "dtype": "bf16"},
        # one request's tree of 17 nodes through a down projection, asymmetric groups of 32
        {"name": "linear 17x14336x4096", "op": "linear", "tokens": 17, "d_in": 14336, "d_out": 4096, "group": 32,
         "zeros": True, "dtype": "bf16"},
        # eight requests of eight nodes through a 5120-wide model's q projection
        {"name": "linear 64x5120x8192", "op": "linear", "tokens": 64, "d_in": 5120, "d_out": 8192, "group": 64,
         "zeros": False, "dtype": "bf16"},
        # a small decode step: eight single tokens of q, k, v; k and v go to the cache
        {"name": "rope 8 tokens", "op": "rope", "tokens": 8, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128,
         "interleaved": False, "positions": 8192, "page": 64, "dtype": "bf16"},
        # part of the head, interleaved, 32 bits, odd counts
        {"name": "rope 1021 part f32", "op": "rope", "tokens": 1021, "heads": 28, "kv_heads": 4, "dim": 80, "rot": 64,
         "interleaved": True, "positions": 32768, "page": 16, "dtype": "f32"},
        # the prefill of several prompts with long positions
        {"name": "rope 16384 tokens", "op": "rope", "tokens": 16384, "heads": 64, "kv_heads": 8, "dim": 128,
         "rot": 128, "interleaved": False, "positions": 131072, "page": 64, "dtype": "bf16"},
        # one request, a tree of eight nodes, a short context: latency
        {"name": "tree 1x8 ctx 777", "op": "tree", "requests": 1, "nodes": 8, "ctx": 777, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 64, "dtype": "bf16"},
        # a batch of requests with ragged contexts, 16 drafted nodes at most for each
        {"name": "tree 32x16 ctx 4096", "op": "tree", "requests": 32, "nodes": 16, "ctx": 4096, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 64, "dtype": "bf16"},
        # few requests with wide trees over long contexts
        {"name": "tree 4x64 ctx 32768", "op": "tree", "requests": 4, "nodes": 64, "ctx": 32768, "heads": 64,
         "kv_heads": 8, "dim": 128, "page": 64, "dtype": "bf16"},
        # one request, a chain of four drafted tokens
        {"name": "verify 1x5 v32000", "op": "verify", "requests": 1, "nodes": 5, "children": 1, "vocab": 32000,
         "drafts": True, "dtype": "f32"},
        # a batch of trees with up to three candidates at a node, an odd vocabulary, bf16 probabilities
        {"name": "verify 32x13 v100003", "op": "verify", "requests": 32, "nodes": 13, "children": 3, "vocab": 100003,
         "drafts": True, "dtype": "bf16"},
        # a large batch of short trees over a large vocabulary
        {"name": "verify 256x8 v131072", "op": "verify", "requests": 256, "nodes": 8, "children": 2, "vocab": 131072,
         "drafts": True, "dtype": "f32"},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["linear", "rope", "tree", "verify"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "linear":
        group = rng.choice([32, 64, 128])
        return {"op": op, "tokens": _log(rng, 1, 64), "d_in": group * max(1, _log(rng, 512, 14336) // group),
                "d_out": _log(rng, 256, 14336), "group": group, "zeros": rng.random() < 0.5, "dtype": dtype}
    if op == "rope":
        dim = rng.choice([64, 80, 96, 128])
        kv = rng.choice([1, 2, 4, 8])
        return {"op": op, "tokens": _log(rng, 1, 16384 if dtype == "bf16" else 8192), "heads": kv * rng.randint(1, 8),
                "kv_heads": kv, "dim": dim, "rot": rng.choice([dim, dim // 2]), "interleaved": rng.random() < 0.5,
                "positions": rng.choice([4096, 32768, 131072]), "page": rng.choice([16, 32, 64]), "dtype": dtype}
    if op == "tree":
        requests = _log(rng, 1, 64)
        kv = rng.choice([2, 4, 8])
        return {"op": op, "requests": requests, "nodes": rng.choice([1, rng.randint(2, 64)]),
                "ctx": min(_log(rng, 16, 32768), 131072 // requests if dtype == "bf16" else 32768 // requests),
                "heads": kv * rng.choice([1, 2, 4, 8]), "kv_heads": kv, "dim": rng.choice([64, 96, 128]),
                "page": rng.choice([16, 32, 64, 128]), "dtype": dtype}
    requests = _log(rng, 1, 256)
    nodes = rng.randint(1, 16)
    return {"op": op, "requests": requests, "nodes": nodes, "children": rng.randint(1, 4),
            "vocab": min(_log(rng, 1000, 131072), 268435456 // (requests * nodes)), "drafts": rng.random() < 0.75,
            "dtype": rng.choice(["f32", "bf16"])}


def work(case):
    eb = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "linear":
        t, di, do = case["tokens"], case["d_in"], case["d_out"]
        groups = do * di // case["group"]
        return {"bytes": do * di / 2 + groups * (eb + (1 if case["zeros"] else 0)) + eb * t * (di + do),
                "flops": 2 * t * di * do}
    if case["op"] == "rope":
        t, hq, hk, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        table = min(t, case["positions"]) * case["rot"] * 4
        return {"bytes": 2 * eb * t * d * (hq + 2 * hk) + table + 16 * t, "flops": 3 * t * case["rot"] * (hq + hk)}
    if case["op"] == "tree":
        ctx, nodes = _tree_lengths(case)
        hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
        keys = int(ctx.sum() + nodes.sum())
        pairs = int((ctx * nodes).sum() + (nodes * (nodes + 1) // 2).sum())
        rows = int(nodes.sum())
        return {"bytes": 2 * eb * keys * hk * d + rows * hq * (2 * eb * d + 4), "flops": 4 * pairs * hq * d}
    b, n, v = case["requests"], case["nodes"], case["vocab"]
    rows = 2 if case["drafts"] else 1
    # the row that the next token is drawn from, for each request, and two values for each drafted token
    return {"bytes": b * v * (rows * eb + 4) + b * n * (2 * eb + 12), "flops": 4 * b * v}


# ---- inputs --------------------------------------------------------------------------
def _tree_lengths(case):
    """Context lengths and node counts of the requests: the largest first, then ragged ones."""
    b, n, c = case["requests"], case["nodes"], case["ctx"]
    i = np.arange(b)
    ctx = np.where(i == 0, c, c - (i * 7919) % max(1, c // 2))
    nodes = np.where(i == 0, n, np.maximum(1, n - (i * 3) % max(1, n // 2)))
    return ctx.astype(np.int64), nodes.astype(np.int64)


def _parents(b, n, children, r):
    """Parents [b, n] of random trees: a node's is one of the `children` nodes before it, the root's is -1."""
    back = r.randint(1, children + 1, size=(b, n))
    return np.maximum(np.arange(n) - back, np.minimum(np.arange(n) - 1, 0)).astype(np.int32)


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
    if case["op"] == "linear":
        t, di, do, group = case["tokens"], case["d_in"], case["d_out"], case["group"]
        s["x"] = normal(t, di).to(dt)
        s["qweight"] = torch.randint(0, 256, (do, di // 2), generator=g, device=dev, dtype=torch.uint8)
        s["scales"] = ((0.5 + torch.rand((do, di // group), generator=g, device=dev)) / (4.6 * math.sqrt(di))).to(dt)
        s["zeros"] = torch.randint(4, 13, (do, di // group), generator=g, device=dev, dtype=torch.uint8) \
            if case["zeros"] else None
        return s
    if case["op"] == "rope":
        t, hq, hk, d, rot, page = (case[k] for k in ("tokens", "heads", "kv_heads", "dim", "rot", "page"))
        qkv = normal(t, (hq + 2 * hk) * d).to(dt)                     # one fused projection's rows, split below
        s["q"] = qkv[:, :hq * d].view(t, hq, d)
        s["k"] = qkv[:, hq * d:(hq + hk) * d].view(t, hk, d)
        s["v"] = qkv[:, (hq + hk) * d:].view(t, hk, d)
        s["positions"] = on_gpu(r.randint(0, case["positions"], size=t).astype(np.int32))
        freq = 500000.0 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)
        angle = torch.arange(case["positions"], device=dev, dtype=torch.float64)[:, None] * freq
        s["table"] = torch.cat([angle.cos(), angle.sin()], dim=1).float()
        pages = (t + page - 1) // page + 2
        s["k_cache"] = normal(pages, page, hk, d).to(dt)
        s["v_cache"] = normal(pages, page, hk, d).to(dt)
        s["slots"] = on_gpu(r.permutation(pages * page)[:t].astype(np.int64))
        return s
    if case["op"] == "tree":
        hq, hk, d, page = (case[k] for k in ("heads", "kv_heads", "dim", "page"))
        ctx, nodes = _tree_lengths(case)
        b, total, most = len(ctx), int(nodes.sum()), int(nodes.max())
        per = -(-int((ctx + nodes).max()) // page)
        s["q"] = normal(total, hq, d).to(dt)
        s["k_cache"] = normal(b * per, page, hk, d).to(dt)
        s["v_cache"] = normal(b * per, page, hk, d).to(dt)
        s["page_table"] = on_gpu(r.permutation(b * per).reshape(b, per).astype(np.int32))
        s["ctx_lens"] = on_gpu(ctx.astype(np.int32))
        starts = np.concatenate([[0], np.cumsum(nodes)])
        s["node_starts"] = on_gpu(starts.astype(np.int32))
        parents = _parents(b, most, 4, r)
        seen = np.zeros((b, most), np.uint64)                         # bit j: node j is the node or above it
        for i in range(most):
            up = np.where(parents[:, i] < 0, np.uint64(0), seen[np.arange(b), np.maximum(parents[:, i], 0)])
            seen[:, i] = up | np.uint64(1 << i)
        keep = np.arange(most)[None, :] < nodes[:, None]
        s["tree_mask"] = on_gpu(seen[keep].view(np.int64).reshape(total, 1))
        return s
    b, n, v = case["requests"], case["nodes"], case["vocab"]
    target = normal(b * n, v) * 2.0
    draft = target + normal(b * n, v) * 0.7
    s["target"] = torch.softmax(target, 1).to(dt)
    draft = torch.softmax(draft, 1).to(dt)
    parents = _parents(b, n, case["children"], r)
    s["parents"] = on_gpu(parents.reshape(-1))
    s["node_starts"] = on_gpu((np.arange(b + 1) * n).astype(np.int32))
    above = on_gpu((np.arange(b)[:, None] * n + np.maximum(parents, 0)).reshape(-1).astype(np.int64))
    if case["drafts"]:                                                # each drafted token is a draw of its parent's row
        race = torch.empty((b * n, v), device=dev).exponential_(generator=g)
        s["tokens"] = (draft.float()[above] / race).argmax(1).to(torch.int32)
        s["draft"] = draft
        del race
    else:                                                             # the draft's likeliest tokens
        best = draft.float().topk(case["children"], 1).indices
        turn = on_gpu(r.randint(0, case["children"], size=b * n).astype(np.int64))
        s["tokens"] = best[above, turn].to(torch.int32)
        s["draft"] = None
    s["uniforms"] = torch.rand((b * n,), generator=g, device=dev)
    s["noise"] = torch.empty((b, v), device=dev).exponential_(generator=g).clamp_min_(1e-30)
    return s


# ---- the operators ---------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if op == "linear":
        return _linear_own(state) if own else _linear_plain(state)
    if op == "rope":
        return _rope_own(state) if own else _rope_plain(state)
    if op == "tree":
        return _tree_own(state) if own else _tree_plain(state)
    return _verify_own(state) if own else _verify_plain(state)


def _linear_own(s):
    return _framework().base_linear(s["x"], s["qweight"], s["scales"], s["zeros"])


def _rope_own(s):
    q = _framework().rope_append(s["q"], s["k"], s["v"], s["positions"], s["table"], s["k_cache"], s["v_cache"],
                                 s["slots"], interleaved=s["case"]["interleaved"])
    return q, s["k_cache"], s["v_cache"]


def _tree_own(s):
    return _framework().tree_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["ctx_lens"],
                                       s["node_starts"], s["tree_mask"])


def _verify_own(s):
    return _framework().verify_drafts(s["target"], s["draft"], s["tokens"], s["parents"], s["node_starts"],
                                      s["uniforms"], s["noise"], s["case"]["nodes"])


def _linear_plain(s):
    w, scales = s["qweight"], s["scales"].float()
    n = torch.stack([w & 15, w >> 4], dim=2).view(scales.shape[0], scales.shape[1], -1).float()
    zero = 8.0 if s["zeros"] is None else s["zeros"].float()[:, :, None]
    weight = ((n - zero) * scales[:, :, None]).view(w.shape[0], -1)
    return (s["x"].float() @ weight.t()).to(s["x"].dtype)


def _rotate(x, cos, sin, interleaved):
    rot = 2 * cos.shape[-1]
    x32 = x.float()
    pairs = x32[..., :rot].unflatten(-1, (-1, 2) if interleaved else (2, -1))
    a, b = pairs.unbind(-1 if interleaved else -2)
    turned = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1 if interleaved else -2).flatten(-2)
    return torch.cat([turned, x32[..., rot:]], dim=-1).to(x.dtype)


def _rope_plain(s):
    cos, sin = s["table"][s["positions"].long()][:, None, :].chunk(2, dim=-1)
    way = s["case"]["interleaved"]
    q = _rotate(s["q"], cos, sin, way)
    s["k_cache"].flatten(0, 1)[s["slots"]] = _rotate(s["k"], cos, sin, way)
    s["v_cache"].flatten(0, 1)[s["slots"]] = s["v"]
    return q, s["k_cache"], s["v_cache"]


def _tree_plain(s):
    q, starts, ctx = s["q"], s["node_starts"].long(), s["ctx_lens"].long()
    total, heads, dim = q.shape
    b, page, kv = ctx.shape[0], s["k_cache"].shape[1], s["k_cache"].shape[2]
    keys = s["page_table"].shape[1] * page
    k = s["k_cache"][s["page_table"].long()].view(b, keys, kv, dim).float()
    v = s["v_cache"][s["page_table"].long()].view(b, keys, kv, dim).float()
    most = s["case"]["nodes"]
    at = (starts[:-1, None] + torch.arange(most, device=q.device)).clamp(max=total - 1)
    node = torch.arange(keys, device=q.device)[None, :] - ctx[:, None]                  # a key's place in the tree
    bit = (s["tree_mask"][at, 0][:, :, None] >> node.clamp(0, 63)[:, None, :]) & 1
    own_nodes = (starts[1:] - starts[:-1])[:, None]
    sees = (node < 0)[:, None, :] | ((node >= 0) & (node < own_nodes))[:, None, :] & (bit == 1)
    q32 = q[at].float().view(b, most, kv, heads // kv, dim)
    score = torch.einsum("bnkgd,blkd->bkgnl", q32, k) / math.sqrt(dim)
    score = score.masked_fill(~sees[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    p = (score - top).exp()
    sums = p.sum(-1, keepdim=True)
    out = torch.einsum("bkgnl,blkd->bnkgd", p / sums.clamp(min=1e-37), v).reshape(b, most, heads, dim)
    lse = (sums.log() + top).squeeze(-1).permute(0, 3, 1, 2).reshape(b, most, heads)
    real = torch.arange(most, device=q.device)[None, :] < own_nodes
    return out[real].to(q.dtype), lse[real]


def _verify_plain(s):
    case, parents = s["case"], s["parents"].long()
    b, n = case["requests"], case["nodes"]
    p = s["target"].float()
    above = parents.clamp(min=0) + torch.arange(b, device=p.device).repeat_interleave(n) * n
    drafted = parents >= 0
    tokens = s["tokens"].long()
    # a node's turn among its parent's children, and the node that each row tries at a turn
    same = (above.view(b, n, 1) == above.view(b, 1, n)) & drafted.view(b, n, 1) & drafted.view(b, 1, n)
    turn = same.tril(-1).sum(-1).view(-1)
    here = torch.arange(b * n, device=p.device)
    left, rest, open_ = p, torch.ones(b * n, device=p.device), torch.ones(b * n, dtype=torch.bool, device=p.device)
    taken = torch.zeros(b * n, dtype=torch.bool, device=p.device)
    a = torch.zeros(b * n, device=p.device)
    one_hot = s["draft"] is None
    q = None if one_hot else s["draft"].float()
    for t in range(min(case["children"], n - 1)):                     # the siblings are tried one after another
        child = torch.full((b * n,), -1, device=p.device)
        child[above[drafted & (turn == t)]] = here[drafted & (turn == t)]
        tried = (child >= 0) & open_
        at = child.clamp(min=0)
        x = tokens[at][:, None]
        q_x = torch.ones_like(rest) if one_hot else q.gather(1, x)[:, 0]
        yes = tried & (s["uniforms"][at] * (q_x * rest) < left.gather(1, x)[:, 0])
        taken[at[yes]] = True
        open_ = open_ & ~yes
        no = tried & ~yes
        a = torch.where(no, a + rest, a)
        if one_hot:
            next_left = left.scatter(1, x, 0.0)
        else:
            next_left = (p - a[:, None] * q).clamp(min=0.0)
        left = torch.where(no[:, None], next_left, left)
        rest = torch.where(no, left.sum(1), rest)
    # the accepted path: nodes whose every node above them was accepted, too
    reach = torch.zeros((b, n, n), device=p.device)
    reach[torch.arange(b, device=p.device)[:, None], torch.arange(n, device=p.device)[None, :],
          (above.view(b, n) - torch.arange(b, device=p.device)[:, None] * n)] = \
        (drafted & taken).view(b, n).float()
    reach[:, 0, 0] = 1.0
    for _ in range(max(1, (n - 1).bit_length())):                     # paths of 2, 4, 8 .. steps to the root
        reach = reach @ reach
    on_path = (reach[:, :, 0] > 0) & (torch.arange(n, device=p.device) > 0)
    count = on_path.sum(1)
    order = torch.where(on_path, torch.arange(n, device=p.device), n).sort(1).values
    path = torch.where(order < n, order, -1)
    last = torch.where(count > 0, order.gather(1, (count - 1).clamp(min=0)[:, None])[:, 0], 0)
    row = torch.arange(b, device=p.device) * n + last
    final = torch.where((left[row].amax(1, keepdim=True) > 0), left[row], p[row])
    return path.int(), count.int(), (final / s["noise"]).argmax(1).int()


# ---- the definitions in 64 bits ----------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        w = s["qweight"].long()
        n = torch.empty((w.shape[0], 2 * w.shape[1]), dtype=torch.float64, device=w.device)
        n[:, 0::2], n[:, 1::2] = (w % 16).double(), (w // 16).double()
        spread = s["scales"].double().repeat_interleave(case["group"], 1)
        zero = torch.full_like(spread, 8.0) if s["zeros"] is None else \
            s["zeros"].double().repeat_interleave(case["group"], 1)
        return torch.matmul((n - zero) * spread, s["x"].double().t()).t().contiguous()
    if case["op"] == "rope":
        half = case["rot"] // 2
        rows = s["table"].double()[s["positions"].long()]
        turn = torch.complex(rows[:, :half], rows[:, half:])[:, None, :]

        def turned(x):
            y = x.double().clone()
            if case["interleaved"]:
                z = torch.complex(y[..., 0:2 * half:2], y[..., 1:2 * half:2]) * turn
                y[..., 0:2 * half:2], y[..., 1:2 * half:2] = z.real, z.imag
            else:
                z = torch.complex(y[..., :half], y[..., half:2 * half]) * turn
                y[..., :half], y[..., half:2 * half] = z.real, z.imag
            return y
        k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
        page = case["page"]
        where = (s["slots"] // page, s["slots"] % page)
        k_cache[where] = turned(s["k"])
        v_cache[where] = s["v"].double()
        return turned(s["q"]), k_cache, v_cache
    if case["op"] == "tree":
        ctx, nodes = _tree_lengths(case)
        outs, lses, at = [], [], 0
        group = case["heads"] // case["kv_heads"]
        for b in range(case["requests"]):
            n, c = int(nodes[b]), int(ctx[b])
            pages = s["page_table"][b].long()
            k = s["k_cache"][pages].flatten(0, 1)[:c + n].double()
            v = s["v_cache"][pages].flatten(0, 1)[:c + n].double()
            bits = s["tree_mask"][at:at + n, 0].cpu().numpy().view(np.uint64)
            sees = np.ones((n, c + n), bool)
            sees[:, c:] = (bits[:, None] >> np.arange(n, dtype=np.uint64)) & np.uint64(1)
            sees = torch.from_numpy(sees).to(k.device)
            one_o, one_l = [], []
            for h in range(case["kv_heads"]):
                q = s["q"][at:at + n, h * group:(h + 1) * group].double()
                score = (q.reshape(-1, case["dim"]) @ k[:, h].t() / math.sqrt(case["dim"])).view(n, group, -1)
                score = torch.where(sees[:, None, :], score, -math.inf)
                one_l.append(torch.logsumexp(score, -1))
                one_o.append((torch.softmax(score, -1).view(n * group, -1) @ v[:, h]).view(n, group, -1))
            outs.append(torch.cat(one_o, 1))
            lses.append(torch.cat(one_l, 1))
            at += n
        return torch.cat(outs), torch.cat(lses)
    b, n = case["requests"], case["nodes"]
    parents = s["parents"].view(b, n).tolist()
    tokens = s["tokens"].view(b, n).tolist()
    uniforms = s["uniforms"].double().view(b, n).tolist()
    path = torch.full((b, n), -1, dtype=torch.int32)
    count, chosen = torch.zeros(b, dtype=torch.int32), torch.zeros(b, dtype=torch.int32)
    for i in range(b):
        node, steps = 0, 0
        while True:
            p = s["target"][i * n + node].double()
            left = p.clone()
            went = None
            for child in [c for c in range(1, n) if parents[i][c] == node]:
                x = tokens[i][child]
                q = s["draft"][i * n + node].double() if case["drafts"] else \
                    torch.nn.functional.one_hot(torch.tensor(x), case["vocab"]).double().to(p.device)
                if uniforms[i][child] * float(q[x]) < float(left[x]):
                    went = child
                    break
                if case["drafts"]:
                    left = (left - q).clamp(min=0)
                    left = left / left.sum().clamp(min=1e-300)
                else:
                    left[x] = 0
                    left = left / left.sum().clamp(min=1e-300)
            if went is None:
                break
            path[i, steps] = went
            node, steps = went, steps + 1
        final = left if float(left.max()) > 0 else p
        count[i], chosen[i] = steps, int((final / s["noise"][i].double()).argmax())
    dev = s["target"].device
    return path.to(dev), count.to(dev), chosen.to(dev)
