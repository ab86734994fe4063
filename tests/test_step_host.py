"""CPU tests of the drafted-token step's calls: every refusal comes before any CUDA call, with a message, and counts
of zero are accepted without one. Pointers here are addresses that nothing reads."""
import ctypes

import pytest

from rank_adapter_apply_gb300 import binding as B
from rank_adapter_apply_gb300 import build as build_mod

P = 0x10000


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load()


def _linear(**kw):
    f = dict(x=P, x_stride=64, qweight=P, scales=P, zeros=None, y=P, y_stride=8, n_tokens=2, d_in=64, d_out=8,
             group=32, dtype=B.LORA_DTYPE_BF16)
    f.update(kw)
    return B.LoraBaseLinearDesc(**f)


def _rope(**kw):
    f = dict(q=P, q_token=64, q_head=16, q_out=P, q_out_token=64, q_out_head=16, k=P, k_token=16, k_head=16, v=P,
             v_token=16, v_head=16, k_cache=P, v_cache=P, cache_page=256, cache_slot=16, cache_head=16, slots=P,
             n_pages=2, positions=P, table=P, n_positions=10, page_size=16, n_tokens=3, n_heads=4, n_kv_heads=1,
             head_dim=16, rot_dim=16, interleaved=0, inverse=0, dtype=B.LORA_DTYPE_BF16)
    f.update(kw)
    return B.LoraRopeDesc(**f)


def _tree(**kw):
    f = dict(q=P, q_token=64, q_head=16, k_cache=P, v_cache=P, cache_page=256, cache_slot=16, cache_head=16, n_pages=2,
             page_table=P, table_stride=2, ctx_lens=P, node_starts=P, tree_mask=P, out=P, out_token=64, out_head=16,
             lse=P, workspace=P, workspace_bytes=1 << 40, scale=0.25, page_size=16, table_pages=2, mask_words=1,
             n_requests=1, n_tokens=3, n_heads=4, n_kv_heads=1, head_dim=16, dtype=B.LORA_DTYPE_BF16)
    f.update(kw)
    return B.LoraTreeAttentionDesc(**f)


def _verify(**kw):
    f = dict(target=P, target_row=100, draft=P, draft_row=100, tokens=P, parents=P, node_starts=P, uniforms=P,
             noise=P, noise_row=100, path=P, n_accepted=P, next_token=P, max_path=3, n_requests=1, n_nodes=4,
             vocab=100, dtype=B.LORA_DTYPE_F32)
    f.update(kw)
    return B.LoraVerifyDesc(**f)


REFUSED = [
    ("lora_base_linear", _linear, [
        dict(dtype=2), dict(group=16), dict(group=0), dict(group=256), dict(d_in=48), dict(d_in=0), dict(d_out=0),
        dict(n_tokens=-1), dict(n_tokens=1 << 20), dict(x=None), dict(qweight=None), dict(scales=None), dict(y=None),
        dict(qweight=P + 8), dict(x_stride=63), dict(y_stride=7)]),
    ("lora_rope", _rope, [
        dict(dtype=-1), dict(n_tokens=-1), dict(n_heads=-1), dict(n_kv_heads=-1), dict(head_dim=1), dict(rot_dim=0),
        dict(rot_dim=15), dict(rot_dim=18), dict(n_positions=-1), dict(page_size=0), dict(n_pages=-1), dict(q=None),
        dict(q_out=None), dict(k=None), dict(v=None), dict(k_cache=None), dict(v_cache=None), dict(slots=None),
        dict(positions=None), dict(table=None), dict(n_pages=1 << 62), dict(n_tokens=1 << 30, n_heads=60000)]),
    ("lora_tree_attention", _tree, [
        dict(dtype=7), dict(n_requests=-1), dict(n_tokens=-1), dict(n_heads=0), dict(n_kv_heads=0), dict(n_kv_heads=3),
        dict(head_dim=0), dict(head_dim=12), dict(head_dim=136), dict(page_size=0), dict(table_pages=-1),
        dict(n_pages=-1), dict(mask_words=-1), dict(mask_words=0), dict(scale=float("nan")),
        dict(scale=float("inf")), dict(q=None), dict(out=None), dict(ctx_lens=None), dict(node_starts=None),
        dict(page_table=None), dict(k_cache=None), dict(v_cache=None), dict(q=P + 2), dict(k_cache=P + 8),
        dict(v_cache=P + 4), dict(out=P + 2), dict(q_token=63), dict(q_head=12), dict(cache_page=255),
        dict(cache_slot=20), dict(cache_head=9), dict(out_token=65), dict(out_head=17), dict(workspace=None),
        dict(workspace=P + 16), dict(workspace_bytes=0)]),
    ("lora_verify_drafts", _verify, [
        dict(dtype=3), dict(n_requests=-1), dict(n_nodes=-1), dict(vocab=0), dict(max_path=-1), dict(target=None),
        dict(tokens=None), dict(parents=None), dict(node_starts=None), dict(uniforms=None), dict(noise=None),
        dict(path=None), dict(n_accepted=None), dict(next_token=None)]),
]


@pytest.mark.parametrize("name,make,change", [(n, m, c) for n, m, cs in REFUSED for c in cs])
def test_refused(lib, name, make, change):
    d = make(**change)
    assert getattr(lib, name)(ctypes.byref(d), None) == B.LORA_ERR_ARG
    assert name[5:] in B.last_error()
    with pytest.raises(B.LoraError):
        getattr(B, name)(ctypes.byref(d), None)


def test_wait_timeouts_needs_a_place(lib):
    assert lib.lora_step_wait_timeouts(None) == B.LORA_ERR_ARG
    assert b"step_wait_timeouts" in lib.lora_last_error()


def test_null_descriptors(lib):
    for name, _, _ in REFUSED:
        assert getattr(lib, name)(None, None) == B.LORA_ERR_ARG


@pytest.mark.parametrize("args", [
    (-1, 64, 0, 1e4, 1, 1, 1, 2), (4, 63, 0, 1e4, 1, 1, 1, 2), (4, 0, 0, 1e4, 1, 1, 1, 2), (4, 514, 0, 1e4, 1, 1, 1, 2),
    (4, 64, 5, 1e4, 1, 1, 1, 2), (4, 64, -1, 1e4, 1, 1, 1, 2), (4, 64, 0, 1.0, 1, 1, 1, 2),
    (4, 64, 0, float("nan"), 1, 1, 1, 2), (4, 64, 1, 1e4, 0.5, 1, 1, 2), (4, 64, 1, 1e4, float("inf"), 1, 1, 2),
    (4, 2, 2, 1e4, 2, 1, 1, 2), (4, 64, 3, 1e4, 2, 0, 1, 2), (4, 64, 3, 1e4, 2, 100, 2, 2), (4, 64, 4, 1e4, 2, 100, 0, 2),
])
def test_rope_table_refused(lib, args):
    assert lib.lora_rope_table(P, *args, None) == B.LORA_ERR_ARG
    assert "rope_table" in B.last_error()
    assert lib.lora_rope_table(None, 4, 64, 0, 1e4, 1, 1, 1, 2, None) == B.LORA_ERR_ARG


def test_nothing_to_do(lib):
    """Counts of zero: accepted, and nothing is queued (there is no device here)."""
    assert lib.lora_base_linear(ctypes.byref(_linear(n_tokens=0, x=None, y=None)), None) == B.LORA_OK
    assert lib.lora_rope(ctypes.byref(_rope(n_tokens=0, q=None, k=None, v=None, q_out=None, slots=None)),
                         None) == B.LORA_OK
    assert lib.lora_tree_attention(ctypes.byref(_tree(n_tokens=0, q=None, out=None)), None) == B.LORA_OK
    assert lib.lora_tree_attention(ctypes.byref(_tree(n_requests=0)), None) == B.LORA_OK
    assert lib.lora_verify_drafts(ctypes.byref(_verify(n_requests=0)), None) == B.LORA_OK
    assert lib.lora_rope_table(None, 0, 64, 0, 1e4, 1, 1, 1, 2, None) == B.LORA_OK


def test_workspace_sizes(lib):
    size = B.lora_tree_attention_workspace_bytes
    assert size(4, 64, 32, 8, 128, B.LORA_DTYPE_BF16) > 0
    for bad in [(-1, 64, 32, 8, 128, 1), (4, -1, 32, 8, 128, 1), (4, 64, 32, 5, 128, 1), (4, 64, 32, 8, 132, 1),
                (4, 64, 32, 8, 256, 1), (4, 64, 32, 8, 128, 9)]:
        assert size(*bad) == 0


def test_tensor_form_refuses_host_tensors():
    import torch
    from rank_adapter_apply_gb300 import operators as ops
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ops.base_linear(x, torch.zeros((8, 32), dtype=torch.uint8), torch.zeros((8, 2), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        ops.rope(x.view(2, 1, 64), torch.zeros(2, dtype=torch.int32), torch.zeros((4, 64)))
    with pytest.raises(ValueError):
        ops.rope_table(4, 64, scaling="cubic")
    with pytest.raises(ValueError):
        ops.rope_table(4, 64, scaling="yarn", factor=2.0)
    with pytest.raises(ValueError):
        ops.base_linear(x.half(), None, None)
