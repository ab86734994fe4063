"""CPU tests of a decoding step's calls: every refusal comes before any CUDA call, with a message, and counts of zero are
accepted without one. Pointers here are addresses that nothing reads."""
import ctypes

import pytest

from rank_adapter_apply_gb300 import binding as B
from tests.test_step_host import REFUSED as STEP
from tests.test_step_host import P, _rope, _tree, lib  # noqa: F401
from tests.test_step_host_edges import OVERLAPS

OF = {name: cases for name, _, cases in STEP}
APART = {name: cases for name, _, cases in OVERLAPS}


def _norm(**kw):
    own = {k: kw.pop(k) for k in list(kw) if k in ("q_weight", "k_weight", "q_weight_head", "k_weight_head", "eps")}
    f = dict(q_weight=P, k_weight=P, q_weight_head=0, k_weight_head=0, eps=1e-6)
    f.update(own)
    return B.LoraNormRopeDesc(rope=_rope(**kw), **f)


def _prefix(**kw):
    own = {k: kw.pop(k) for k in list(kw)
           if k in ("prefix_table", "prefix_stride", "prefix_lens", "group_starts", "n_groups", "prefix_pages")}
    f = dict(prefix_table=P, prefix_stride=2, prefix_lens=P, group_starts=P, n_groups=1, prefix_pages=2)
    f.update(own)
    return B.LoraPrefixAttentionDesc(tree=_tree(**kw), **f)


def _sample(**kw):
    f = dict(logits=P, logits_row=100, noise=P, noise_row=100, temperature=P, top_k=P, top_p=P, min_p=P, tokens=P,
             logprobs=P, n_rows=2, vocab=100, dtype=B.LORA_DTYPE_F32)
    f.update(kw)
    return B.LoraSampleDesc(**f)


REFUSED = [
    ("lora_norm_rope", _norm, OF["lora_rope"] + APART["lora_rope"] + [
        dict(inverse=1), dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")), dict(q_weight_head=-1),
        dict(k_weight_head=-16)]),
    ("lora_prefix_attention", _prefix, OF["lora_tree_attention"] + APART["lora_tree_attention"] + [
        dict(n_groups=-1), dict(n_groups=2 ** 31 - 1, n_requests=2), dict(prefix_pages=-1), dict(prefix_stride=-1),
        dict(prefix_table=None), dict(prefix_lens=None), dict(group_starts=None),
        dict(workspace_bytes=B.lora_tree_attention_workspace_bytes(1, 3, 4, 1, 16, B.LORA_DTYPE_BF16))]),
    ("lora_sample_tokens", _sample, [
        dict(dtype=5), dict(n_rows=-1), dict(n_rows=(1 << 27) + 1), dict(vocab=0), dict(vocab=-3), dict(logits=None),
        dict(noise=None), dict(tokens=None), dict(logits_row=-1), dict(noise_row=-100)]),
]


@pytest.mark.parametrize("name,make,change", [(n, m, c) for n, m, cs in REFUSED for c in cs])
def test_refused(lib, name, make, change):  # noqa: F811
    d = make(**dict(change))
    assert getattr(lib, name)(ctypes.byref(d), None) == B.LORA_ERR_ARG
    assert B.last_error().startswith(name[5:] + ":")
    with pytest.raises(B.LoraError):
        getattr(B, name)(ctypes.byref(d), None)


def test_null_descriptors(lib):  # noqa: F811
    for name, _, _ in REFUSED:
        assert getattr(lib, name)(None, None) == B.LORA_ERR_ARG


def test_nothing_to_do(lib):  # noqa: F811
    """Counts of zero: accepted, and nothing is queued (there is no device here)."""
    for name, d in [("lora_norm_rope", _norm(n_tokens=0, q=None, k=None, v=None, q_out=None, slots=None)),
                    ("lora_prefix_attention", _prefix(n_tokens=0, q=None, out=None)),
                    ("lora_prefix_attention", _prefix(n_requests=0, n_groups=0, prefix_lens=None, group_starts=None)),
                    ("lora_sample_tokens", _sample(n_rows=0, logits=None, noise=None, tokens=None))]:
        assert getattr(lib, name)(ctypes.byref(d), None) == B.LORA_OK, name


def test_workspace_sizes(lib):  # noqa: F811
    size = B.lora_prefix_attention_workspace_bytes
    bf16 = B.LORA_DTYPE_BF16
    assert size(4, 2, 64, 32, 8, 128, bf16) >= 2 * B.lora_tree_attention_workspace_bytes(4, 64, 32, 8, 128, bf16)
    assert size(4, 0, 64, 32, 8, 128, bf16) == size(4, 9, 64, 32, 8, 128, bf16)
    assert size(4, 2, 1 << 20, 64, 8, 128, bf16) > 1072 << 26            # does not wrap around
    for bad in [(-1, 1, 64, 32, 8, 128, 1), (4, -1, 64, 32, 8, 128, 1), (4, 1, -1, 32, 8, 128, 1),
                (4, 1, 64, 32, 5, 128, 1), (4, 1, 64, 32, 8, 132, 1), (4, 1, 64, 32, 8, 256, 1), (4, 1, 64, 32, 8, 128, 9),
                (4, 1, 1 << 26, 32, 8, 128, 1)]:
        assert size(*bad) == 0


def test_tensor_form_refuses_host_tensors():
    import torch
    from rank_adapter_apply_gb300 import operators as ops
    x = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    pos = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        ops.norm_rope(x, None, pos, torch.zeros((4, 64)))
    with pytest.raises(ValueError):
        ops.norm_rope_append(x, x, x, None, None, pos, torch.zeros((4, 64)), x, x, pos.long())
    with pytest.raises(ValueError):
        ops.prefix_attention(x, x, x, pos, pos, pos, pos, pos, pos)
    with pytest.raises(ValueError):
        ops.sample_tokens(torch.zeros((2, 9)), torch.ones((2, 9)))
    with pytest.raises(ValueError):
        ops.sample_tokens([1.0], None)
