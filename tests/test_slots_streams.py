"""LoraSlots: the pools' zeros are written before anything of the context's own streams. On the CPU with stand-ins."""
import types

from rank_adapter_apply_gb300 import slots as slots_mod


class _Stream:
    def __init__(self, name, log):
        self.name, self.log, self.cuda_stream = name, log, 0

    def wait_stream(self, other):
        self.log.append((self.name, other.name))


def test_streams_wait_for_the_zeroed_pools(monkeypatch):
    log = []
    tensor = types.SimpleNamespace(data_ptr=lambda: 256)
    compute, upload, current = (_Stream(n, log) for n in ("compute", "upload", "current"))
    monkeypatch.setattr(slots_mod.torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(slots_mod.torch.cuda, "current_stream", lambda *a: current)
    for name in ("zeros", "empty"):
        monkeypatch.setattr(slots_mod.torch, name, lambda *a, **kw: log.append("made") or tensor)
    monkeypatch.setattr(slots_mod.B, "load", lambda: None)
    monkeypatch.setattr(slots_mod.B, "lora_workspace_bytes", lambda *a: 1024)
    monkeypatch.setattr(slots_mod.B, "lora_slots_init", lambda *a: log.append("init"))
    slots_mod.LoraSlots([(64, 64)], 2, 16, 8, compute_stream=compute, upload_stream=upload)
    last_made = len(log) - 1 - log[::-1].index("made")
    for stream in ("compute", "upload"):
        assert last_made < log.index((stream, "current")) < log.index("init")
