"""Torch-tensor form of the calls of a decoding step and of a step over drafted tokens.

Around the adapters' delta (``LoraSlots.apply_multi``) a step over drafted tokens
needs the base model's product with 4-bit weights (``base_linear``), rotary
positions with the append to a paged cache (``rope``, ``rope_append``; with norms of
the query and key heads in front ``norm_rope``, ``norm_rope_append``), attention
of the drafted trees over that cache (``tree_attention``; of requests that share
prefixes ``prefix_attention``) and the verification of the drafts
(``verify_drafts``), a plain decoding step the draw of the next token
(``sample_tokens``). Formulas, layouts and what happens to entries out
of range stand in include/rank_adapter_apply.h.

The checks, descriptors and allocations are native (csrc/tensor_calls.cpp): a small
call's time is the host's. Every function checks its tensors (``ValueError``; what the
library refuses raises ``binding.LoraError``), queues its kernels on torch's current stream of the current
device and returns without waiting. Outputs and workspace come from torch's
allocator on that stream. A tensor made on another stream needs the caller's own
ordering (an event or ``wait_stream``), as for any kernel. No gradient is recorded: a
tensor that requires one, or has a forward-mode tangent, is refused. What a call writes
in place (``out``, the caches) has a new version afterwards.
"""
from __future__ import annotations

import importlib.machinery
import importlib.util
import os

import torch

from . import binding as B
from .build import TENSOR_CALLS


def _load():
    if not os.path.exists(TENSOR_CALLS):
        raise RuntimeError(f"{TENSOR_CALLS} is missing (run `python -m rank_adapter_apply_gb300.build`)")
    lib = B.load()
    loader = importlib.machinery.ExtensionFileLoader("_tensor_calls", TENSOR_CALLS)
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_tensor_calls", loader))
    loader.exec_module(module)
    import ctypes
    names = ("lora_base_linear", "lora_rope", "lora_tree_attention", "lora_tree_attention_workspace_bytes",
             "lora_verify_drafts", "lora_norm_rope", "lora_prefix_attention", "lora_prefix_attention_workspace_bytes",
             "lora_sample_tokens")
    module.bind(*[ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in names], B.check)
    return module


_calls = _load()
_base_linear, _rope, _rope_append = _calls.base_linear, _calls.rope, _calls.rope_append
_tree_attention, _verify_drafts = _calls.tree_attention, _calls.verify_drafts
_norm_rope, _norm_rope_append = _calls.norm_rope, _calls.norm_rope_append
_prefix_attention, _sample_tokens = _calls.prefix_attention, _calls.sample_tokens


def base_linear(x, qweight, scales, zeros=None, out=None):
    """y = x W^T with 4-bit weights, W[i][k] = scales[i][k // group] * (n[i][k] - zeros[i][k // group]).

    x [tokens, d_in] (rows may be strided), qweight uint8 [d_out, d_in // 2] (column 2j in the low four bits of
    byte j), scales [d_out, d_in // group] of x's dtype, group 32, 64 or 128, zeros uint8 like scales or None (8).
    Returns ``out`` or a new [tokens, d_out]."""
    return _base_linear(x, qweight, scales, zeros, out)


_SCALING = {None: B.LORA_ROPE_PLAIN, "linear": B.LORA_ROPE_LINEAR, "base": B.LORA_ROPE_BASE,
            "pieces": B.LORA_ROPE_PIECES, "yarn": B.LORA_ROPE_YARN}


def rope_table(n_positions, rot_dim, base=10000.0, scaling=None, factor=1.0, original=None, low_freq=None,
               high_freq=None, device="cuda"):
    """The fp32 table [n_positions, rot_dim] (cosines, then sines) that rope reads.

    scaling: None, "linear" (positions / factor), "base" (a larger base), "pieces" (by wavelength; low_freq 1,
    high_freq 4 by default) or "yarn" (by turns; low_freq 1, high_freq 32): the last two take ``original``, the
    positions the model was trained on."""
    if scaling not in _SCALING:
        raise ValueError(f"scaling {scaling!r}: one of {list(_SCALING)} is needed")
    if scaling in ("pieces", "yarn") and original is None:
        raise ValueError(f"scaling {scaling!r} needs original")
    device = torch.device(device)
    if device.type != "cuda" or (device.index is not None and device.index != torch.cuda.current_device()):
        raise ValueError(f"device {device}: the current CUDA device is needed")
    table = torch.empty((n_positions, rot_dim), dtype=torch.float32, device=device)
    high = 32.0 if scaling == "yarn" else 4.0
    B.lora_rope_table(table.data_ptr() or None, n_positions, rot_dim, _SCALING[scaling], float(base), float(factor),
                      float(1.0 if original is None else original), float(1.0 if low_freq is None else low_freq),
                      float(high if high_freq is None else high_freq), torch.cuda.current_stream().cuda_stream)
    return table


def rope(x, positions, table, interleaved=False, inverse=False, out=None):
    """Rotate the first table.shape[1] elements of every head of x [tokens, heads, head_dim].

    positions int32 [tokens]; inverse=True turns by the negative angle: the gradient of the forward rotation (its undoing
    only where the table's magnitude is 1, so not with "yarn" and a factor above 1). ``out`` may be x."""
    return _rope(x, positions, table, interleaved, inverse, out)


def rope_append(q, k, v, positions, table, k_cache, v_cache, slots, interleaved=False, out=None):
    """Rotate q and k, and write k and v to the paged cache. Returns the rotated q (``out``, which may be q).

    q [tokens, heads, head_dim], k and v [tokens, kv_heads, head_dim], caches [pages, page_size, kv_heads, head_dim],
    slots int64 [tokens]: token t goes to place slots[t] % page_size of page slots[t] // page_size."""
    return _rope_append(q, k, v, positions, table, k_cache, v_cache, slots, interleaved, out)


def norm_rope(x, weight, positions, table, eps=1e-6, interleaved=False, out=None):
    """Norm every head of x [tokens, heads, head_dim] and rotate it as rope does, in one pass.

    y = x / sqrt(mean(x^2) + eps) * weight over a head's elements, weight [head_dim], [heads, head_dim] or None (ones), of
    x's dtype. ``out`` may be x."""
    return _norm_rope(x, weight, positions, table, eps, interleaved, out)


def norm_rope_append(q, k, v, q_weight, k_weight, positions, table, k_cache, v_cache, slots, eps=1e-6,
                     interleaved=False, out=None):
    """rope_append with norm_rope's norm of the heads of q and k in front. Returns the rotated q (``out``, which may be q)."""
    return _norm_rope_append(q, k, v, q_weight, k_weight, positions, table, k_cache, v_cache, slots, eps, interleaved, out)


def tree_attention(q, k_cache, v_cache, page_table, ctx_lens, node_starts, tree_mask=None, scale=None, out=None):
    """Attention of drafted trees over the paged cache. Returns (out like q, lse fp32 [tokens, heads]).

    q [tokens, heads, head_dim]; page_table int32 [requests, pages of a request]; ctx_lens int32 [requests];
    node_starts int32 [requests + 1]: request b owns the rows node_starts[b] .. node_starts[b + 1], and its node j is
    key ctx_lens[b] + j of the cache; tree_mask int64 [tokens, words] (bit j % 64 of word j // 64: the row sees node
    j), None: node i sees nodes 0..i. scale: head_dim ** -0.5 by default."""
    return _tree_attention(q, k_cache, v_cache, page_table, ctx_lens, node_starts, tree_mask, scale, out)


def prefix_attention(q, k_cache, v_cache, prefix_table, prefix_lens, group_starts, page_table, ctx_lens, node_starts,
                     tree_mask=None, scale=None, out=None):
    """tree_attention of requests that share prefixes. Returns (out like q, lse fp32 [tokens, heads]).

    Group g is the requests group_starts[g] .. group_starts[g + 1] (int32 [groups + 1]); they see the prefix_lens[g]
    (int32 [groups]) keys on the pages prefix_table[g] (int32 [groups, pages of a prefix]), in front of what tree_attention
    shows them: ctx_lens and page_table do not contain the prefix. It is read once for each tile of up to 128 rows of the
    group; a page size that is not a multiple of 8 leaves tiles of 16."""
    return _prefix_attention(q, k_cache, v_cache, prefix_table, prefix_lens, group_starts, page_table, ctx_lens, node_starts,
                             tree_mask, scale, out)


def sample_tokens(logits, noise, temperature=None, top_k=None, top_p=None, min_p=None):
    """Draw a token for every row of logits [rows, vocab]. Returns (tokens int32 [rows], logprobs fp32 [rows]).

    noise fp32 [rows, vocab], exponentially distributed; temperature, top_p, min_p fp32 [rows] and top_k int32 [rows], or
    None. Each filter is taken of the softmax at the row's temperature, and a token stays if all keep it; temperature 0 is
    the likeliest token. logprobs: of the token at the temperature (1 where it is 0), before the filters."""
    return _sample_tokens(logits, noise, temperature, top_k, top_p, min_p)


def verify_drafts(target, draft, tokens, parents, node_starts, uniforms, noise, max_path):
    """Verify drafted trees. Returns int32 (path [requests, max_path], n_accepted [requests], next_token [requests]).

    target [nodes, vocab]: the target's probabilities after each node; draft the same for the rows the children were
    drawn from, or None (drafts chosen without chance); tokens, parents int32 [nodes]; node_starts int32
    [requests + 1]; uniforms fp32 [nodes] from U[0, 1); noise fp32 [requests, vocab], exponentially distributed."""
    return _verify_drafts(target, draft, tokens, parents, node_starts, uniforms, noise, max_path)
