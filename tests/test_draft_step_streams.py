"""Streams of draft_step.step: its work runs on the slots' stream, between the caller's stream before and after it. On the
CPU with stand-ins for the streams that note what waits for what; on the GPU with inputs that come late."""
import contextlib
import types

import pytest


class _Stream:
    def __init__(self, name, log):
        self.name, self.log = name, log

    def wait_stream(self, other):
        self.log.append((self.name, "waits for", other.name))


class _Tensor:
    def __init__(self, name, log):
        self.name, self.log = name, log

    def record_stream(self, stream):
        self.log.append((self.name, "used on", stream.name))


def test_order_of_a_step(monkeypatch):
    """Nothing runs before the caller's work is waited for, the caller's stream waits for everything that ran, inputs are
    recorded on the slots' stream before their use and results on the caller's."""
    from rank_adapter_apply_gb300 import build
    build.build()
    from rank_adapter_apply_gb300 import draft_step
    log = []
    caller, compute = _Stream("caller", log), _Stream("compute", log)

    @contextlib.contextmanager
    def entered(stream):
        log.append(("enter", stream.name))
        yield
        log.append(("leave", stream.name))
    monkeypatch.setattr(draft_step.torch.cuda, "current_stream", lambda *a: caller)
    monkeypatch.setattr(draft_step.torch.cuda, "stream", entered)
    results = [_Tensor(n, log) for n in ("path", "count", "token")]
    target = _Tensor("target", log)
    monkeypatch.setattr(draft_step.ops, "verify_drafts", lambda *a: log.append("verify") or tuple(results))
    model = types.SimpleNamespace(slots=types.SimpleNamespace(compute=compute),
                                  probabilities=lambda b: log.append("probabilities") or target,
                                  keep=lambda *a: log.append("keep"))
    names = [f.name for f in draft_step.dataclasses.fields(draft_step.DraftBatch)]
    batch = draft_step.DraftBatch(*[_Tensor(n, log) for n in names])
    uniforms, noise = _Tensor("uniforms", log), _Tensor("noise", log)
    for draft in (None, _Tensor("draft", log)):
        log.clear()
        assert draft_step.step(model, batch, draft, uniforms, noise, 3) == (*results, target)
        first, last = log.index("probabilities"), log.index("keep")
        assert log.index(("compute", "waits for", "caller")) < log.index(("enter", "compute")) < first
        assert last < log.index(("leave", "compute")) < log.index(("caller", "waits for", "compute"))
        for name in names + ["uniforms", "noise"] + (["draft"] if draft else []):
            assert (name, "used on", "compute") in log
        for name in ("path", "count", "token", "target"):
            assert log.index((name, "used on", "caller")) > last


@pytest.mark.gpu
def test_inputs_that_come_late():
    """Uniforms and noise that the caller's stream writes only after a while, and drops right after the call: the step
    uses them, and the caller's stream sees the step's results without a wait of its own."""
    import torch
    from rank_adapter_apply_gb300 import build
    build.build()
    from rank_adapter_apply_gb300.draft_step import DraftBatch, DraftConfig, DraftModel, step
    cfg = DraftConfig(hidden=128, heads=2, kv_heads=1, head_dim=64, ffn=256, layers=1, vocab=300, group=32,
                      positions=128, page_size=4, pages=20, max_loras=1, max_lora_rank=8, max_tokens=64,
                      rope_base=10000.0, dtype=torch.float32)
    model = DraftModel(cfg, seed=9)
    try:
        model.load_adapters(1, 8, alpha=8.0)
        # every child is accepted with u = 0 and none with u = 1
        tree = ([7, 11, 12, 13], [-1, 0, 1, 2])
        batch = DraftBatch.make([tree], [0], [list(range(19, 0, -1))], [0], cfg.page_size)
        for u_value, accepted in ((0.0, 3), (1.0, 0), (0.0, 3)):
            u, noise = torch.full((4,), 1.0 - u_value, device="cuda"), torch.zeros((1, 300), device="cuda")
            torch.cuda.synchronize()
            torch.cuda._sleep(100_000_000)
            u.fill_(u_value)
            noise.fill_(1.0)
            noise[0, 42] = 1e-30                                   # the race's winner
            path, count, token, target = step(model, batch, None, u, noise, 3)
            del u, noise
            again = [torch.full((4,), 0.5, device="cuda"), torch.full((1, 300), 7.0, device="cuda")]
            assert count.tolist() == [accepted] and token.tolist() == [42] and len(again) == 2
            assert path.tolist() == [list(range(1, accepted + 1)) + [-1] * (3 - accepted)]
            assert abs(target.sum().item() - 4) < 1e-4
    finally:
        model.close()
