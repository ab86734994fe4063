"""The drafted-token step as a whole against the model in 64 bits, in both types and over the kernels that sizes choose:
prompts as chains, forking trees, single tokens, a batch of two tokens; requests with and without an adapter.

Tolerance of ln p. fp32 as in test_gpu_draft_step.py: 2^-10. bf16: some 15 values of a layer are rounded to 2^-9 (0.0008 in
the mean), 30 of them come to sqrt(30) * 0.0008 = 0.0045 of the last hidden vector and of the logits, which are of size
one: 0.02 at 4.2 sigma, the largest of 30000, and 2^-9 of logits up to 4.5 for their own rounding: 0.03. 2^-3 is allowed at
most and 2^-6 in the mean; a wrong mask, position, adapter or cache row is off by about one."""
import numpy as np
import pytest

from tests.test_gpu_draft_step import Plain, _dequantise

pytestmark = pytest.mark.gpu

MOST, MEAN = {"bf16": 2.0 ** -3, "f32": 2.0 ** -10}, {"bf16": 2.0 ** -6, "f32": 2.0 ** -13}


class PlainWithBase(Plain):
    """Slot -1 (the last entry): no adapter."""

    def __init__(self, model, *args):
        super().__init__(model, *args)
        self.merged.append([_dequantise(w, model.cfg.group) for layer in model.weights for w in layer])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,kv_heads,head_dim,group", [(8, 2, 64, 64), (4, 4, 128, 128)])
def test_turns_of_a_batch(heads, kv_heads, head_dim, group, dtype):
    import torch
    from rank_adapter_apply_gb300 import binding as B
    from rank_adapter_apply_gb300 import build
    build.build()
    from rank_adapter_apply_gb300.draft_step import DraftBatch, DraftConfig, DraftModel, step
    cfg = DraftConfig(hidden=256, heads=heads, kv_heads=kv_heads, head_dim=head_dim, ffn=384, layers=2, vocab=500,
                      group=group, positions=256, page_size=8, pages=60, max_loras=3, max_lora_rank=16, max_tokens=128,
                      rope_base=10000.0, dtype={"bf16": torch.bfloat16, "f32": torch.float32}[dtype])
    model = DraftModel(cfg, seed=heads)
    try:
        plain = PlainWithBase(model, model.load_adapters(3, 8, alpha=16.0), 8, 16.0)
        r = np.random.default_rng(heads)
        pages = r.permutation(60).reshape(4, 15).tolist()
        adapters, known, ctx = [0, -1, 2, 1], [[], [], [], []], [0, 0, 0, 0]
        last = [int(t) for t in r.integers(0, 500, 4)]

        def tree(first, n, fork):
            pars = [-1] + [int(r.integers(max(0, i - fork), i)) for i in range(1, n)]
            return [first] + [int(t) for t in r.integers(0, 500, n - 1)], pars
        # (requests, nodes of each, how far back a parent may be)
        turns = [([0, 1, 2, 3], [30, 1, 9, 14], 1), ([0, 1, 2, 3], [12, 20, 9, 17], 3), ([0, 1, 2, 3], [3, 2, 1, 4], 2),
                 ([0, 1, 2, 3], [1] * 4, 1), ([1, 2], [1, 1], 1), ([3], [1], 1)]
        for turn, (who, sizes, fork) in enumerate(turns):
            trees = [tree(last[b], n, fork) for b, n in zip(who, sizes)]
            batch = DraftBatch.make(trees, [ctx[b] for b in who], [pages[b] for b in who], [adapters[b] for b in who],
                                    cfg.page_size)
            u = torch.zeros(batch.tokens.shape[0], device="cuda")             # a node's first child is accepted
            path, count, token, target = step(model, batch, None, u, torch.ones((len(who), 500), device="cuda"), 32)
            got, at, errors = target.double().cpu().numpy(), 0, []
            for j, (b, (toks, pars)) in enumerate(zip(who, trees)):
                assert np.abs(got[at:at + len(toks)].sum(1) - 1).max() < 1e-5
                for i in range(len(toks)):
                    line, up = [], i
                    while up >= 0:
                        line.append(toks[up])
                        up = pars[up]
                    errors.append(np.abs(np.log(got[at + i] / plain.probabilities(known[b] + line[::-1], adapters[b]))))
                node, steps = 0, []
                while node in pars:
                    node = pars.index(node)
                    steps.append(node)
                assert path[j].tolist() == steps + [-1] * (32 - len(steps)) and int(count[j]) == len(steps)
                assert int(token[j]) == int(got[at + node].argmax())
                known[b] = known[b] + [toks[0]] + [toks[s] for s in steps]
                ctx[b], last[b] = len(known[b]), int(token[j])
                at += len(toks)
            errors = np.array(errors)
            assert errors.max() <= MOST[dtype] and errors.mean() <= MEAN[dtype], (turn, errors.max(), errors.mean())
        assert B.lora_step_wait_timeouts() == 0
    finally:
        model.close()
