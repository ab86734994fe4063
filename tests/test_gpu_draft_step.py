"""The drafted-token step as a whole (draft_step.py): two steps of a small fp32 model with adapters, against the same
model in 64 bits that recomputes every sequence from its tokens, without a cache, trees or adapters apart.

Tolerance: the step is about 20 fp32 operators deep, each within a few 2^-22 of its inputs' size, and the norms keep
sizes near one: probabilities within 2^-12 relative (a wrong mask, position, slot or cache row is off by far more)."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _dequantise(w, group):
    q, s, z = [t.double().cpu().numpy() if t.dtype != np.uint8 else t for t in w]
    q = w[0].cpu().numpy()
    n = np.empty((q.shape[0], 2 * q.shape[1]))
    n[:, 0::2], n[:, 1::2] = q & 15, q >> 4
    return (n - np.repeat(z, group, 1)) * np.repeat(s, group, 1)


class Plain:
    """The model in 64 bits: the probabilities after the last of a sequence of tokens, with one adapter merged in."""

    def __init__(self, model, adapters, rank, alpha):
        from rank_adapter_apply_gb300.draft_step import LAYER_NAMES
        cfg = model.cfg
        self.cfg, self.names = cfg, LAYER_NAMES
        self.emb = model.embedding.double().cpu().numpy()
        self.head = _dequantise(model.head, cfg.group)
        self.merged = []
        for A, Bm in adapters:
            flat = [w for layer in model.weights for w in layer]
            self.merged.append([_dequantise(w, cfg.group) + alpha / rank * Bm[i].double().numpy() @ A[i].double().numpy()
                                for i, w in enumerate(flat)])

    def probabilities(self, tokens, adapter):
        cfg = self.cfg
        W = self.merged[adapter]
        n, d = len(tokens), cfg.head_dim
        f = cfg.rope_base ** (-2.0 * np.arange(d // 2) / d)
        ang = np.arange(n)[:, None] * f
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]

        def turn(x):
            a, b = x[..., :d // 2], x[..., d // 2:]
            return np.concatenate([a * c - b * s, a * s + b * c], -1)

        def norm(x):
            return x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-5)
        x = self.emb[tokens]
        for layer in range(cfg.layers):
            w = dict(zip(self.names, W[layer * 7:layer * 7 + 7]))
            h = norm(x)
            q = turn((h @ w["q"].T).reshape(n, cfg.heads, d))
            k = turn((h @ w["k"].T).reshape(n, cfg.kv_heads, d))
            v = (h @ w["v"].T).reshape(n, cfg.kv_heads, d)
            att = np.zeros((n, cfg.heads, d))
            for hd in range(cfg.heads):
                g = hd // (cfg.heads // cfg.kv_heads)
                sc = q[:, hd] @ k[:, g].T / math.sqrt(d)
                sc[np.triu_indices(n, 1)] = -np.inf
                e = np.exp(sc - sc.max(1, keepdims=True))
                att[:, hd] = (e / e.sum(1, keepdims=True)) @ v[:, g]
            x = x + att.reshape(n, -1) @ w["o"].T
            h = norm(x)
            gate, up = h @ w["gate"].T, h @ w["up"].T
            x = x + (gate / (1 + np.exp(-gate)) * up) @ w["down"].T
        z = norm(x[-1]) @ self.head.T
        e = np.exp(z - z.max())
        return e / e.sum()


def test_two_steps_of_drafted_trees():
    import torch
    from rank_adapter_apply_gb300 import binding as B
    from rank_adapter_apply_gb300 import build
    build.build()
    from rank_adapter_apply_gb300.draft_step import DraftBatch, DraftConfig, DraftModel, step
    cfg = DraftConfig(hidden=256, heads=4, kv_heads=2, head_dim=64, ffn=384, layers=2, vocab=500, group=64,
                      positions=256, page_size=8, pages=40, max_loras=3, max_lora_rank=16, max_tokens=64,
                      rope_base=10000.0, dtype=torch.float32)
    model = DraftModel(cfg, seed=5)
    try:
        plain = Plain(model, model.load_adapters(3, 8, alpha=16.0), 8, 16.0)
        r = np.random.default_rng(3)
        pages = r.permutation(40).reshape(4, 10).tolist()
        adapters = [0, 2, 1, 0]
        # the first step reads the prompts: chains whose drafts are taken as they are (u = 0 accepts what is possible)
        prompts = [r.integers(0, 500, n).tolist() for n in (9, 1, 5, 14)]
        known, ctx = [list(p) for p in prompts], [0, 0, 0, 0]
        trees = [(p, [-1] + list(range(len(p) - 1))) for p in prompts]
        for turn in range(2):
            batch = DraftBatch.make(trees, ctx, pages, adapters, cfg.page_size)
            nodes = batch.tokens.shape[0]
            u = torch.zeros(nodes, device="cuda") if turn == 0 else torch.rand(nodes, device="cuda") * 0.02
            noise = torch.ones((4, 500), device="cuda")
            path, count, token, target = step(model, batch, None, u, noise, 16)
            model.slots.compute.synchronize()
            got, path, count, token = target.double().cpu().numpy(), path.tolist(), count.tolist(), token.tolist()
            starts = batch.node_starts.tolist()
            for b, (toks, pars) in enumerate(trees):
                before = known[b][:ctx[b]]
                for i in range(len(toks)):
                    line, j = [], i
                    while j >= 0:
                        line.append(toks[j])
                        j = pars[j]
                    want = plain.probabilities(before + line[::-1], adapters[b])
                    p = got[starts[b] + i]
                    assert np.abs(p - want).max() <= 2.0 ** -12 * want.max() and \
                        np.abs(np.log(p / want)).max() <= 2.0 ** -10, (turn, b, i, np.abs(p - want).max())
                # u so small that every first child with u < p is taken: follow the path
                node = 0
                for step_at in range(count[b]):
                    assert pars[path[b][step_at]] == node
                    node = path[b][step_at]
                assert path[b][count[b]:] == [-1] * (16 - count[b])
                if turn == 0:
                    assert count[b] == len(toks) - 1
                last = got[starts[b] + node].copy()
                assert token[b] == int(last.argmax()) or turn == 1
                if turn == 0:
                    known[b] = before + toks
                    ctx[b] = len(known[b])
            # the next step: trees that fork, after the token that the step gave
            trees = []
            for b in range(4):
                n = [12, 3, 1, 7][b]
                pars = [-1] + [int(r.integers(max(0, i - 3), i)) for i in range(1, n)]
                trees.append(([token[b]] + r.integers(0, 500, n - 1).tolist(), pars))
        assert B.lora_step_wait_timeouts() == 0
    finally:
        model.close()


def test_accepted_nodes_stay_in_the_cache():
    """After a step over a forking tree, the cache holds the accepted path's rows behind the context: a further step
    from there gives the probabilities of the sequence without any cache."""
    import torch
    from rank_adapter_apply_gb300.draft_step import DraftBatch, DraftConfig, DraftModel, step
    cfg = DraftConfig(hidden=128, heads=2, kv_heads=1, head_dim=64, ffn=256, layers=2, vocab=300, group=32,
                      positions=128, page_size=4, pages=20, max_loras=1, max_lora_rank=8, max_tokens=64,
                      rope_base=10000.0, dtype=torch.float32)
    model = DraftModel(cfg, seed=9)
    try:
        plain = Plain(model, model.load_adapters(1, 8, alpha=8.0), 8, 8.0)
        pages = [list(range(19, 0, -1))]
        tree = ([7, 11, 12, 13, 14, 15], [-1, 0, 0, 2, 2, 4])     # the path 2, 4, 5 is the one to take
        batch = DraftBatch.make([tree], [0], pages, [0], cfg.page_size)
        u = torch.tensor([0, 1, 0, 1, 0, 0], dtype=torch.float32, device="cuda")
        noise = torch.ones((1, 300), device="cuda")
        path, count, token, _ = step(model, batch, None, u, noise, 6)
        model.slots.compute.synchronize()
        assert path.tolist() == [[2, 4, 5, -1, -1, -1]] and count.tolist() == [3]
        batch = DraftBatch.make([([int(token[0])], [-1])], [4], pages, [0], cfg.page_size)
        _, _, _, target = step(model, batch, None, u[:1], noise, 6)
        model.slots.compute.synchronize()
        want = plain.probabilities([7, 12, 14, 15, int(token[0])], 0)
        p = target.double().cpu().numpy()[0]
        assert np.abs(np.log(p / want)).max() <= 2.0 ** -10
    finally:
        model.close()


def test_command_runs(capsys):
    from rank_adapter_apply_gb300 import draft_step
    draft_step.main(["--requests", "3", "--nodes", "4", "--steps", "2", "--layers", "1"])
    assert "2 steps of 3 requests" in capsys.readouterr().out
