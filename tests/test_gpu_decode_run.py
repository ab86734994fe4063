"""Decoding steps as they would be run (draft_step.py): head norms, prefixes that requests share, drafted trees behind them
and sampled tokens, against the same model in 64 bits that recomputes every sequence from its tokens.

Tolerances as in test_gpu_draft_step.py: an fp32 model's probabilities within 2^-12 of their largest."""
import math

import numpy as np
import pytest

from tests.test_gpu_draft_step import Plain

pytestmark = pytest.mark.gpu


class NormedPlain(Plain):
    """Plain with the heads of q and k normed before the rotation."""

    def __init__(self, model, adapters, rank, alpha):
        super().__init__(model, adapters, rank, alpha)
        self.norms = [[w.double().cpu().numpy() for w in pair] for pair in model.norms]

    def probabilities(self, tokens, adapter):
        cfg, W = self.cfg, self.merged[adapter]
        n, d = len(tokens), cfg.head_dim
        ang = np.arange(n)[:, None] * cfg.rope_base ** (-2.0 * np.arange(d // 2) / d)
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]

        def norm(x, eps=1e-5):
            return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)

        def turn(x, weight):
            x = norm(x, 1e-6) * weight
            a, b = x[..., :d // 2], x[..., d // 2:]
            return np.concatenate([a * c - b * s, a * s + b * c], -1)
        x = self.emb[tokens]
        for layer in range(cfg.layers):
            w = dict(zip(self.names, W[layer * 7:layer * 7 + 7]))
            h = norm(x)
            q = turn((h @ w["q"].T).reshape(n, cfg.heads, d), self.norms[layer][0])
            k = turn((h @ w["k"].T).reshape(n, cfg.kv_heads, d), self.norms[layer][1])
            v = (h @ w["v"].T).reshape(n, cfg.kv_heads, d)
            each = cfg.heads // cfg.kv_heads
            sc = np.einsum("ihd,jhd->hij", q, np.repeat(k, each, 1)) / math.sqrt(d)
            sc[:, np.triu(np.ones((n, n), bool), 1)] = -np.inf
            e = np.exp(sc - sc.max(-1, keepdims=True))
            att = np.einsum("hij,jhd->ihd", e / e.sum(-1, keepdims=True), np.repeat(v, each, 1))
            x = x + att.reshape(n, -1) @ w["o"].T
            h = norm(x)
            gate, up = h @ w["gate"].T, h @ w["up"].T
            x = x + (gate / (1 + np.exp(-gate)) * up) @ w["down"].T
        z = norm(x[-1]) @ self.head.T
        e = np.exp(z - z.max())
        return e / e.sum()


def _softmax(z):
    e = np.exp(z - z.max(-1, keepdims=True))
    return e / e.sum(-1, keepdims=True)


def _same(p, want, where):
    assert np.abs(p - want).max() <= 2.0 ** -12 * want.max() and np.abs(np.log(p / want)).max() <= 2.0 ** -10, where


def test_decoding_behind_shared_prefixes():
    import torch
    from rank_adapter_apply_gb300 import binding as B
    from rank_adapter_apply_gb300 import build
    build.build()
    from rank_adapter_apply_gb300.draft_step import DraftBatch, DraftConfig, DraftModel, sample_step, step
    cfg = DraftConfig(hidden=256, heads=4, kv_heads=2, head_dim=64, ffn=384, layers=2, vocab=500, group=64,
                      positions=256, page_size=8, pages=60, max_loras=3, max_lora_rank=16, max_tokens=128,
                      rope_base=10000.0, dtype=torch.float32, head_norms=True)
    model = DraftModel(cfg, seed=6)
    try:
        plain = NormedPlain(model, model.load_adapters(3, 8, alpha=16.0), 8, 16.0)
        r = np.random.default_rng(4)
        ids = r.permutation(60)
        shared = [r.integers(0, 500, 50).tolist(), r.integers(0, 500, 17).tolist()]
        prefix_pages = [ids[:7].tolist(), ids[7:10].tolist()]
        pages = ids[10:].reshape(5, 10).tolist()
        adapters = [1, 1, 1, 2, 0]                       # two groups, and a request of none
        in_front = [shared[0]] * 3 + [shared[1]] + [[]]
        prefixes = [(3, prefix_pages[0], 50), (1, prefix_pages[1], 17)]
        chain = lambda t: (t, list(range(-1, len(t) - 1)))  # noqa: E731

        def noise_of(rows):
            return torch.from_numpy(r.standard_exponential((rows, 500)).astype(np.float32)).cuda()
        # the prefixes' keys; their probabilities are those of the sequence
        batch = DraftBatch.make([chain(t) for t in shared], [0, 0], [prefix_pages[0], prefix_pages[1] + [0] * 4], [1, 2],
                                cfg.page_size)
        _, _, logits = sample_step(model, batch, noise_of(67))
        got = _softmax(logits.double().cpu().numpy())
        for row, (t, adapter) in {49: (shared[0], 1), 66: (shared[1], 2), 20: (shared[0][:21], 1)}.items():
            _same(got[row], plain.probabilities(t, adapter), row)
        # plain decoding steps; the first reads prompts of one to four tokens
        known = [[] for _ in range(5)]
        new = [r.integers(0, 500, n).tolist() for n in (1, 4, 2, 3, 1)]
        dev = lambda v, t=torch.float32: torch.tensor(v, dtype=t, device="cuda")  # noqa: E731
        for turn in range(3):
            batch = DraftBatch.make([chain(t) for t in new], [len(k) for k in known], pages, adapters, cfg.page_size, prefixes)
            ends = (batch.node_starts[1:] - 1).tolist()
            rows = ends[-1] + 1
            noise = noise_of(rows)
            t, k, p = [0.7] * rows, [0] * rows, [1.0] * rows
            t[ends[1]], k[ends[2]], p[ends[3]], k[ends[4]], p[ends[4]] = 0.0, 5, 0.6, 40, 0.9
            token, logprob, logits = sample_step(model, batch, noise, dev(t), dev(k, torch.int32), dev(p))
            z, noise = logits.double().cpu().numpy(), noise.double().cpu().numpy()
            for b, e in enumerate(ends):
                _same(_softmax(z[e]), plain.probabilities(in_front[b] + known[b] + new[b], adapters[b]), (turn, b))
                probs = _softmax(z[e] / (t[e] or 1.0))
                order = np.argsort(-probs, kind="stable")
                n = len(order) if k[e] == 0 else k[e]
                if p[e] < 1:
                    n = min(n, int((np.cumsum(probs[order]) - probs[order] < p[e]).sum()))
                kept = order[:1 if t[e] == 0 else n]
                want = kept[np.argmax(probs[kept] / noise[e][kept])]
                assert token[e].item() == want, (turn, b)
                assert abs(logprob[e].item() - math.log(probs[want])) <= 2.0 ** -18
            known = [k + n for k, n in zip(known, new)]
            new = [[int(token[e])] for e in ends]
        # drafted trees behind the same prefixes
        trees = [([t[0]] + r.integers(0, 500, n - 1).tolist(), [-1] + [int(r.integers(max(0, i - 2), i)) for i in range(1, n)])
                 for t, n in zip(new, (9, 1, 30, 4, 6))]
        batch = DraftBatch.make(trees, [len(k) for k in known], pages, adapters, cfg.page_size, prefixes)
        nodes = batch.tokens.shape[0]
        path, count, _, target = step(model, batch, None, torch.zeros(nodes, device="cuda"), torch.ones((5, 500), device="cuda"), 30)
        got = target.double().cpu().numpy()
        for b, (toks, pars) in enumerate(trees):
            for i in range(len(toks)):
                line, j = [], i
                while j >= 0:
                    line.append(toks[j])
                    j = pars[j]
                _same(got[int(batch.node_starts[b]) + i], plain.probabilities(in_front[b] + known[b] + line[::-1], adapters[b]), (b, i))
        # and a step from the accepted path
        path, count = path.tolist(), count.tolist()
        known = [k + [t[0][0]] + [t[0][j] for j in path[b][:count[b]]] for b, (k, t) in enumerate(zip(known, trees))]
        batch = DraftBatch.make([chain([3 + b]) for b in range(5)], [len(k) for k in known], pages, adapters, cfg.page_size, prefixes)
        _, _, logits = sample_step(model, batch, noise_of(5))
        got = _softmax(logits.double().cpu().numpy())
        for b in range(5):
            _same(got[b], plain.probabilities(in_front[b] + known[b] + [3 + b], adapters[b]), b)
        assert B.lora_step_wait_timeouts() == 0
    finally:
        model.close()


def test_command_of_plain_decoding():
    from rank_adapter_apply_gb300 import draft_step
    draft_step.main(["--requests", "3", "--steps", "2", "--layers", "1", "--sample", "--prefix", "100", "--head-norms"])
