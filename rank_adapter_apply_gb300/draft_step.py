"""One verification step of drafted tokens for many tenants: a small decoder whose base weights are in 4 bits, with an
adapter for each request, run with the framework's calls from the tokens to the verified path.

    python -m rank_adapter_apply_gb300.draft_step            # a few steps of a random model, tokens accepted and time
    python -m rank_adapter_apply_gb300.draft_step --sample --prefix 256 --head-norms     # plain decoding, one adapter

Per layer: base_linear (q, k, v) + the adapters' deltas, rope_append into the paged cache, tree_attention, base_linear
(o) + deltas, then the gated feed-forward the same way; at the end the target's probabilities after every node, and
verify_drafts. Weights are random: the step, not the model, is the point. Norms, activation and softmax are torch's.

A model with head_norms takes norm_rope_append in rope_append's place, and a batch whose requests share prefixes
prefix_attention in tree_attention's; a step without drafts (sample_step) ends with sample_tokens.
"""
from __future__ import annotations

import argparse
import contextlib
import dataclasses
import itertools
import math
import time

import torch

from . import binding as B
from . import operators as ops
from .slots import LoraSlots

LAYER_NAMES = ("q", "k", "v", "o", "gate", "up", "down")


@dataclasses.dataclass
class DraftConfig:
    hidden: int = 4096
    heads: int = 32
    kv_heads: int = 8
    head_dim: int = 128
    ffn: int = 14336
    layers: int = 2
    vocab: int = 32000
    group: int = 128
    rope_base: float = 500000.0
    positions: int = 32768
    page_size: int = 64
    pages: int = 512
    max_loras: int = 8
    max_lora_rank: int = 16
    max_tokens: int = 256
    dtype: torch.dtype = torch.bfloat16
    head_norms: bool = False     # every head of q and k is normed before the rotation

    def shapes(self):
        """(d_in, d_out) of a layer's linear layers, in LAYER_NAMES' order."""
        q, kv = self.heads * self.head_dim, self.kv_heads * self.head_dim
        h, f = self.hidden, self.ffn
        return [(h, q), (h, kv), (h, kv), (q, h), (h, f), (h, f), (f, h)]


class DraftModel:
    """Random weights, the paged cache and the adapter slots."""

    def __init__(self, cfg: DraftConfig, seed=0):
        self.cfg = cfg
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.slots = LoraSlots(cfg.shapes() * cfg.layers, cfg.max_loras, cfg.max_lora_rank, cfg.max_tokens,
                               dtype=cfg.dtype, max_layers_per_call=3)
        # made on the stream that reads them; the caller's stream may read them, too
        with torch.cuda.stream(self.slots.compute):
            self.weights = [[self._quantised(i, o) for i, o in cfg.shapes()] for _ in range(cfg.layers)]
            self.head = self._quantised(cfg.hidden, cfg.vocab)
            self.embedding = self._normal(cfg.vocab, cfg.hidden)
            self.table = ops.rope_table(cfg.positions, cfg.head_dim, base=cfg.rope_base)
            shape = (cfg.layers, cfg.pages, cfg.page_size, cfg.kv_heads, cfg.head_dim)
            self.k_cache = torch.zeros(shape, dtype=cfg.dtype, device="cuda")
            self.v_cache = torch.zeros(shape, dtype=cfg.dtype, device="cuda")
            # weights of q's and k's heads
            self.norms = [[self._normal(cfg.head_dim) * 0.2 + 1 for _ in "qk"]
                          for _ in range(cfg.layers)] if cfg.head_norms else None
        torch.cuda.current_stream().wait_stream(self.slots.compute)

    def _normal(self, *shape):
        return torch.randn(shape, generator=self.gen, device="cuda", dtype=torch.float32).to(self.cfg.dtype)

    def _quantised(self, d_in, d_out):
        """(qweight, scales, zeros) of a random layer whose outputs keep its inputs' size."""
        q = torch.randint(0, 256, (d_out, d_in // 2), generator=self.gen, device="cuda", dtype=torch.uint8)
        s = torch.rand((d_out, d_in // self.cfg.group), generator=self.gen, device="cuda") + 0.5
        z = torch.randint(6, 10, s.shape, generator=self.gen, device="cuda", dtype=torch.uint8)
        return q, (s / (4.7 * math.sqrt(d_in))).to(self.cfg.dtype), z

    def load_adapters(self, n, rank, alpha=32.0, seed=1):
        """Random adapters in slots 0..n-1; returns their host tensors (per slot: A list, B list)."""
        gen = torch.Generator().manual_seed(seed)
        made = []
        for slot in range(n):
            A = [(torch.randn((rank, i), generator=gen) / math.sqrt(i)).to(self.cfg.dtype).pin_memory()
                 for i, _ in self.slots.layers]
            Bm = [(torch.randn((o, rank), generator=gen) * 0.1).to(self.cfg.dtype).pin_memory()
                  for _, o in self.slots.layers]
            self.slots.load_slot(slot, A, Bm, rank, alpha)
            made.append((A, Bm))
        self.slots.sync_uploads()
        return made

    def _norm(self, x):
        x32 = x.float()
        return (x32 * torch.rsqrt(x32.square().mean(-1, keepdim=True) + 1e-5)).to(x.dtype)

    def _linear(self, layer, names, x, slot_idx):
        """The named layers' products of x with the adapters' deltas added."""
        at = [LAYER_NAMES.index(n) for n in names]
        ys = [ops.base_linear(x, *self.weights[layer][i]) for i in at]
        self.slots.apply_multi([layer * len(LAYER_NAMES) + i for i in at], [x] * len(at), ys, slot_idx)
        return ys

    def logits(self, batch):
        """The target's logits after every node; the nodes' keys and values are appended to the cache.
        To be called with the slots' compute stream as the current one, after the batch is there (step() sees to both)."""
        cfg = self.cfg
        tokens = batch.tokens.shape[0]
        x = self.embedding[batch.tokens.long()]
        for layer in range(cfg.layers):
            h = self._norm(x)
            q, k, v = self._linear(layer, ("q", "k", "v"), h, batch.slot_idx)
            q = q.view(tokens, cfg.heads, cfg.head_dim)
            k, v = (t.view(tokens, cfg.kv_heads, cfg.head_dim) for t in (k, v))
            cache = self.k_cache[layer], self.v_cache[layer]
            if self.norms:
                q = ops.norm_rope_append(q, k, v, *self.norms[layer], batch.positions, self.table, *cache, batch.places, out=q)
            else:
                q = ops.rope_append(q, k, v, batch.positions, self.table, *cache, batch.places, out=q)
            if batch.prefix_table is not None:
                attended, _ = ops.prefix_attention(q, *cache, batch.prefix_table, batch.prefix_lens, batch.group_starts,
                                                   batch.page_table, batch.ctx_lens, batch.node_starts, batch.tree_mask)
            else:
                attended, _ = ops.tree_attention(q, *cache, batch.page_table, batch.ctx_lens, batch.node_starts,
                                                 batch.tree_mask)
            o, = self._linear(layer, ("o",), attended.view(tokens, -1), batch.slot_idx)
            x = x + o
            gate, up = self._linear(layer, ("gate", "up"), self._norm(x), batch.slot_idx)
            down, = self._linear(layer, ("down",), torch.nn.functional.silu(gate) * up, batch.slot_idx)
            x = x + down
        return ops.base_linear(self._norm(x), *self.head)

    def probabilities(self, batch):
        """The target's probabilities after every node (fp32); else as logits."""
        return torch.softmax(self.logits(batch).float(), dim=-1)

    def keep(self, batch, path, count):
        """Move the accepted nodes' cache rows behind the root's, where the next step expects them."""
        accepted = path >= 0                                              # [requests, max_path]
        request, step = accepted.nonzero(as_tuple=True)
        ctx = batch.ctx_lens.long()[request]
        source, target = ctx + path[request, step], ctx + 1 + step
        table, page = batch.page_table.long(), self.cfg.page_size
        at = (table[request, source // page], source % page)
        to = (table[request, target // page], target % page)
        for cache in (self.k_cache, self.v_cache):
            cache[:, to[0], to[1]] = cache[:, at[0], at[1]]               # all read before any is written

    def close(self):
        self.slots.close()


@dataclasses.dataclass
class DraftBatch:
    """The drafted trees of a step, on the device. Node 0 of a request is its last token."""
    tokens: torch.Tensor        # int32 [nodes]
    parents: torch.Tensor       # int32 [nodes], within the request
    node_starts: torch.Tensor   # int32 [requests + 1]
    ctx_lens: torch.Tensor      # int32 [requests], tokens in the cache
    positions: torch.Tensor     # int32 [nodes]: (prefix +) context + depth
    places: torch.Tensor        # int64 [nodes]: cache slot of context + node
    tree_mask: torch.Tensor     # int64 [nodes, 1]
    page_table: torch.Tensor    # int32 [requests, pages]
    slot_idx: torch.Tensor      # int32 [nodes]: the request's adapter slot
    # of requests that share prefixes, which ctx_lens and page_table then do not contain
    prefix_table: torch.Tensor | None = None    # int32 [groups, pages]
    prefix_lens: torch.Tensor | None = None     # int32 [groups]
    group_starts: torch.Tensor | None = None    # int32 [groups + 1], requests

    @staticmethod
    def make(trees, ctx_lens, page_table, slots, page_size, prefixes=None):
        """trees: per request (tokens, parents) of up to 64 nodes; page_table: list of page ids per request. prefixes: list
        of (requests, page ids, length), in the requests' order; requests behind the last one have none. The keys of a
        prefix are those of the adapter it was run with: a group's requests have that one."""
        tokens, parents, positions, places, masks, slot_idx, starts = [], [], [], [], [], [], [0]
        in_front = [length for n, _, length in prefixes or [] for _ in range(n)]
        in_front += [0] * (len(trees) - len(in_front))
        for (toks, pars), ctx, pages, slot, shared in zip(trees, ctx_lens, page_table, slots, in_front):
            depth, seen = [], []
            for i, p in enumerate(pars):
                depth.append(0 if i == 0 else depth[p] + 1)
                seen.append((0 if i == 0 else seen[p]) | 1 << i)
                at = ctx + i
                places.append(pages[at // page_size] * page_size + at % page_size)
            tokens += toks
            parents += pars
            positions += [shared + ctx + d for d in depth]
            masks += [s - (1 << 64) if s >> 63 else s for s in seen]
            slot_idx += [slot] * len(toks)
            starts.append(len(tokens))

        def dev(v, dtype):
            return torch.tensor(v, dtype=dtype).cuda()
        groups = [None] * 3
        if prefixes:
            wide = max(len(pages) for _, pages, _ in prefixes)
            table = [list(pages) + [-1] * (wide - len(pages)) for _, pages, _ in prefixes]
            counts = [0] + list(itertools.accumulate(n for n, _, _ in prefixes))
            groups = [dev(table, torch.int32), dev([n for _, _, n in prefixes], torch.int32), dev(counts, torch.int32)]
        return DraftBatch(dev(tokens, torch.int32), dev(parents, torch.int32), dev(starts, torch.int32),
                          dev(list(ctx_lens), torch.int32), dev(positions, torch.int32), dev(places, torch.int64),
                          dev(masks, torch.int64).view(-1, 1), dev([list(p) for p in page_table], torch.int32),
                          dev(slot_idx, torch.int32), *groups)


@contextlib.contextmanager
def _on_slots_stream(model, inputs):
    """The slots' compute stream as the current one, behind what the caller's stream holds so far; the caller's stream in
    turn waits for the work, and gets the results that are put into the list. Inputs may be dropped right after."""
    caller, compute, results = torch.cuda.current_stream(), model.slots.compute, []
    compute.wait_stream(caller)
    for t in inputs:
        if t is not None:
            t.record_stream(compute)
    with torch.no_grad(), torch.cuda.stream(compute):
        yield results
    caller.wait_stream(compute)
    for t in results:
        t.record_stream(caller)


def step(model: DraftModel, batch: DraftBatch, draft, uniforms, noise, max_path):
    """One step: probabilities, verification, cache rows of the accepted nodes. draft: the rows the children were drawn
    from (fp32) or None. Returns (path, n_accepted, next_token, probabilities).

    The work runs on the slots' compute stream, behind what the caller's current stream holds so far; the current stream
    in turn waits for the results. Inputs may be dropped right after the call."""
    with _on_slots_stream(model, (*vars(batch).values(), draft, uniforms, noise)) as results:
        target = model.probabilities(batch)
        path, count, token = ops.verify_drafts(target, draft, batch.tokens, batch.parents, batch.node_starts, uniforms,
                                               noise, max_path)
        model.keep(batch, path, count)
        results += [path, count, token, target]
    return path, count, token, target


def sample_step(model: DraftModel, batch: DraftBatch, noise, temperature=None, top_k=None, top_p=None, min_p=None):
    """One step without drafts: a token after every node, with the filters and the noise [nodes, vocab] of sample_tokens.
    Returns (tokens, logprobs, logits). Nodes that are a prompt's, or a prefix's, leave their keys in the cache, and the
    last one's token is the next. Streams as in step()."""
    filters = (temperature, top_k, top_p, min_p)
    with _on_slots_stream(model, (*vars(batch).values(), noise, *filters)) as results:
        logits = model.logits(batch)
        token, logprob = ops.sample_tokens(logits, noise, *filters)
        results += [token, logprob, logits]
    return token, logprob, logits


def _chain(tokens):
    return list(tokens), list(range(-1, len(tokens) - 1))


def _main_sample(model, a):
    """Plain decoding steps, all requests behind one prefix with the adapter of slot 0."""
    cfg = model.cfg
    gen = torch.Generator(device="cuda").manual_seed(2)
    shared = list(range(-(-a.prefix // cfg.page_size)))
    per = (cfg.pages - len(shared)) // a.requests
    pages = [list(range(len(shared) + r * per, len(shared) + (r + 1) * per)) for r in range(a.requests)]

    def run(batch, temperature=0.8, top_p=0.95):
        rows = batch.tokens.shape[0]
        noise = torch.empty((rows, cfg.vocab), device="cuda").exponential_(generator=gen)
        full = lambda v: torch.full((rows,), v, device="cuda")  # noqa: E731
        return sample_step(model, batch, noise, full(temperature), None, full(top_p), None)
    for at in range(0, a.prefix, 64):                   # the prefix's keys, as one request's chains
        chain = _chain([(7 * t + 1) % cfg.vocab for t in range(at, min(at + 64, a.prefix))])
        run(DraftBatch.make([chain], [at], [shared], [0], cfg.page_size))
    ctx, last, spent = 0, [1 + r for r in range(a.requests)], 0.0
    for s in range(a.steps + 1):
        batch = DraftBatch.make([_chain([t]) for t in last], [ctx] * a.requests, pages, [0] * a.requests, cfg.page_size,
                                [(a.requests, shared, a.prefix)] if a.prefix else None)
        torch.cuda.synchronize()
        t = time.perf_counter()
        token, _, _ = run(batch)
        torch.cuda.synchronize()
        spent += time.perf_counter() - t if s > 0 else 0.0      # the first step loads device code
        ctx, last = ctx + 1, token.tolist()
    print(f"{a.steps} steps of {a.requests} requests behind a prefix of {a.prefix}, {cfg.layers} layers: "
          f"{spent / a.steps * 1e3:.3f} ms a step, waits given up: {B.lora_step_wait_timeouts()}")


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--nodes", type=int, default=8)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--head-norms", action="store_true", help="norm the heads of q and k")
    ap.add_argument("--sample", action="store_true", help="steps without drafts, behind a shared prefix of --prefix tokens")
    ap.add_argument("--prefix", type=int, default=0)
    a = ap.parse_args(argv)
    cfg = DraftConfig(layers=a.layers, max_tokens=max(256, a.requests * a.nodes), head_norms=a.head_norms)
    own = (cfg.pages - -(-a.prefix // cfg.page_size)) // a.requests * cfg.page_size
    if a.sample and (a.prefix < 0 or a.steps >= own or a.prefix + a.steps >= cfg.positions):
        ap.error(f"the cache holds {cfg.pages} pages of {cfg.page_size} and {cfg.positions} positions")
    model = DraftModel(cfg)
    model.load_adapters(cfg.max_loras, cfg.max_lora_rank)
    if a.sample:
        _main_sample(model, a)
        return model.close()
    per = cfg.pages // a.requests
    pages = [list(range(r * per, (r + 1) * per)) for r in range(a.requests)]
    ctx, last = [0] * a.requests, [1 + r for r in range(a.requests)]
    gen = torch.Generator(device="cuda").manual_seed(2)
    total, began = 0, 0.0
    for s in range(a.steps + 1):
        # drafts: chains of the tokens that a flat draft row gives
        nodes = a.requests * a.nodes
        drafted = torch.randint(0, cfg.vocab, (a.requests, a.nodes), generator=gen, device="cuda")
        draft = torch.full((1, cfg.vocab), 1.0 / cfg.vocab, device="cuda").expand(nodes, -1)
        uniforms = torch.rand((nodes,), generator=gen, device="cuda")
        noise = torch.empty((a.requests, cfg.vocab), device="cuda").exponential_(generator=gen)
        trees = [([last[r]] + drafted[r, 1:].tolist(), [-1] + list(range(a.nodes - 1))) for r in range(a.requests)]
        batch = DraftBatch.make(trees, ctx, pages, [r % cfg.max_loras for r in range(a.requests)], cfg.page_size)
        torch.cuda.synchronize()
        t = time.perf_counter()
        path, count, token, _ = step(model, batch, draft, uniforms, noise, a.nodes - 1)
        torch.cuda.synchronize()
        if s > 0:                                       # the first step loads device code
            began += time.perf_counter() - t
            total += int(count.sum()) + a.requests
        ctx = [c + 1 + n for c, n in zip(ctx, count.tolist())]
        last = token.tolist()
    print(f"{a.steps} steps of {a.requests} requests, {a.nodes} nodes each, {cfg.layers} layers: {total} tokens, "
          f"{began / a.steps * 1e3:.3f} ms a step, waits given up: {B.lora_step_wait_timeouts()}")
    model.close()


if __name__ == "__main__":
    main()
