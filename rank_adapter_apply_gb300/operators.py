"""Torch-tensor form of the drafted-token step's calls.

Around the adapters' delta (``LoraSlots.apply_multi``) a step over drafted tokens
needs the base model's product with 4-bit weights (``base_linear``), rotary
positions with the append to a paged cache (``rope``, ``rope_append``), attention
of the drafted trees over that cache (``tree_attention``) and the verification of
the drafts (``verify_drafts``). Formulas, layouts and what happens to entries out
of range stand in include/rank_adapter_apply.h.

Every function checks its tensors (``ValueError``; what the library refuses raises
``binding.LoraError``), queues its kernels on torch's current stream of the current
device and returns without waiting. Outputs and workspace come from torch's
allocator on that stream. A tensor made on another stream needs the caller's own
ordering (an event or ``wait_stream``), as for any kernel.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding as B

_CODE = {torch.bfloat16: B.LORA_DTYPE_BF16, torch.float32: B.LORA_DTYPE_F32}
_byref = ctypes.byref
_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _fail(text):
    raise ValueError(text)


def _start(first, **others):
    """dtype code and raw stream; every tensor given has to be on the current device."""
    code = _CODE.get(first.dtype)
    if code is None:
        _fail(f"dtype {first.dtype}: bfloat16 or float32 is needed")
    device = first.device
    if device.type != "cuda":
        _fail(f"tensors on {device}: a CUDA device is needed")
    for name, t in others.items():
        if t is not None and t.device != device:
            _fail(f"{name} is on {t.device}, not on {device}")
    if device.index != torch.cuda.current_device():
        _fail(f"tensors on {device}, which is not the current device")
    return code, _stream(device.index)


def _typed(t, dtype, name):
    if t.dtype is not dtype:
        _fail(f"{name} has dtype {t.dtype}: {dtype} is needed")


def base_linear(x, qweight, scales, zeros=None, out=None):
    """y = x W^T with 4-bit weights, W[i][k] = scales[i][k // group] * (n[i][k] - zeros[i][k // group]).

    x [tokens, d_in] (rows may be strided), qweight uint8 [d_out, d_in // 2] (column 2j in the low four bits of
    byte j), scales [d_out, d_in // group] of x's dtype, group 32, 64 or 128, zeros uint8 like scales or None (8).
    Returns ``out`` or a new [tokens, d_out]."""
    code, stream = _start(x, qweight=qweight, scales=scales, zeros=zeros, out=out)
    if x.dim() != 2 or qweight.dim() != 2 or scales.dim() != 2:
        _fail("x, qweight and scales have two dimensions")
    tokens, d_in = x.shape
    d_out, groups = scales.shape
    _typed(qweight, torch.uint8, "qweight")
    _typed(scales, x.dtype, "scales")
    if groups < 1 or d_in % groups or qweight.shape != (d_out, d_in // 2):
        _fail(f"x {tuple(x.shape)}, qweight {tuple(qweight.shape)}, scales {tuple(scales.shape)} do not fit")
    if not qweight.is_contiguous() or not scales.is_contiguous() or (tokens and x.stride(1) != 1):
        _fail("qweight and scales are contiguous, and x has unit stride along a row")
    if zeros is not None:
        _typed(zeros, torch.uint8, "zeros")
        if zeros.shape != scales.shape or not zeros.is_contiguous():
            _fail("zeros is contiguous and has the shape of scales")
    if out is None:
        out = torch.empty((tokens, d_out), dtype=x.dtype, device=x.device)
    else:
        _typed(out, x.dtype, "out")
        if out.shape != (tokens, d_out) or (tokens and d_out > 1 and out.stride(1) != 1):
            _fail(f"out {tuple(out.shape)} with unit stride along a row: {(tokens, d_out)} is needed")
    d = B.LoraBaseLinearDesc(x.data_ptr(), x.stride(0), qweight.data_ptr(), scales.data_ptr(),
                             None if zeros is None else zeros.data_ptr(), out.data_ptr(), out.stride(0), tokens, d_in,
                             d_out, d_in // groups, code)
    B.lora_base_linear(_byref(d), stream)
    return out


_SCALING = {None: B.LORA_ROPE_PLAIN, "linear": B.LORA_ROPE_LINEAR, "base": B.LORA_ROPE_BASE,
            "pieces": B.LORA_ROPE_PIECES, "yarn": B.LORA_ROPE_YARN}


def rope_table(n_positions, rot_dim, base=10000.0, scaling=None, factor=1.0, original=None, low_freq=None,
               high_freq=None, device="cuda"):
    """The fp32 table [n_positions, rot_dim] (cosines, then sines) that rope reads.

    scaling: None, "linear" (positions / factor), "base" (a larger base), "pieces" (by wavelength; low_freq 1,
    high_freq 4 by default) or "yarn" (by turns; low_freq 1, high_freq 32): the last two take ``original``, the
    positions the model was trained on."""
    if scaling not in _SCALING:
        _fail(f"scaling {scaling!r}: one of {list(_SCALING)} is needed")
    if scaling in ("pieces", "yarn") and original is None:
        _fail(f"scaling {scaling!r} needs original")
    device = torch.device(device)
    if device.type != "cuda" or (device.index is not None and device.index != torch.cuda.current_device()):
        _fail(f"device {device}: the current CUDA device is needed")
    table = torch.empty((n_positions, rot_dim), dtype=torch.float32, device=device)
    B.lora_rope_table(table.data_ptr() or None, n_positions, rot_dim, _SCALING[scaling], float(base), float(factor),
                      float(original or 1.0), float(low_freq or 1.0),
                      float(high_freq or (32.0 if scaling == "yarn" else 4.0)),
                      _stream(torch.cuda.current_device()))
    return table


def _rope_common(q, positions, table, out):
    if q.dim() != 3 or (q.numel() and q.stride(2) != 1):
        _fail("q is [tokens, heads, head_dim] with unit stride along a head")
    _typed(positions, torch.int32, "positions")
    _typed(table, torch.float32, "table")
    if positions.shape != (q.shape[0],) or not positions.is_contiguous():
        _fail(f"positions {tuple(positions.shape)}: one contiguous int32 for each of {q.shape[0]} tokens is needed")
    if table.dim() != 2 or not table.is_contiguous():
        _fail("table is a contiguous [n_positions, rot_dim]")
    if out is None:
        return torch.empty(q.shape, dtype=q.dtype, device=q.device)
    _typed(out, q.dtype, "out")
    if out.shape != q.shape or (out.numel() and out.stride(2) != 1):
        _fail(f"out {tuple(out.shape)} with unit stride along a head: {tuple(q.shape)} is needed")
    return out


def rope(x, positions, table, interleaved=False, inverse=False, out=None):
    """Rotate the first table.shape[1] elements of every head of x [tokens, heads, head_dim].

    positions int32 [tokens]; inverse=True turns back (the gradient of the forward rotation). ``out`` may be x."""
    code, stream = _start(x, positions=positions, table=table, out=out)
    out = _rope_common(x, positions, table, out)
    tokens, heads, dim = x.shape
    d = B.LoraRopeDesc(x.data_ptr(), x.stride(0), x.stride(1), out.data_ptr(), out.stride(0), out.stride(1), None, 0,
                       0, None, 0, 0, None, None, 0, 0, 0, None, 0, positions.data_ptr(), table.data_ptr(),
                       table.shape[0], 1, tokens, heads, 0, dim, table.shape[1], interleaved, inverse, code)
    B.lora_rope(_byref(d), stream)
    return out


def _cache(k_cache, v_cache, like, kv_heads, dim):
    _typed(k_cache, like.dtype, "k_cache")
    _typed(v_cache, like.dtype, "v_cache")
    if k_cache.dim() != 4 or k_cache.shape[2:] != (kv_heads, dim):
        _fail(f"k_cache {tuple(k_cache.shape)}: [pages, page_size, {kv_heads}, {dim}] is needed")
    if v_cache.shape != k_cache.shape or v_cache.stride() != k_cache.stride() or k_cache.stride(3) != 1:
        _fail("k_cache and v_cache have one shape and one set of strides, unit along a head")


def rope_append(q, k, v, positions, table, k_cache, v_cache, slots, interleaved=False, out=None):
    """Rotate q and k, and write k and v to the paged cache. Returns the rotated q (``out``, which may be q).

    q [tokens, heads, head_dim], k and v [tokens, kv_heads, head_dim], caches [pages, page_size, kv_heads, head_dim],
    slots int64 [tokens]: token t goes to place slots[t] % page_size of page slots[t] // page_size."""
    code, stream = _start(q, k=k, v=v, positions=positions, table=table, k_cache=k_cache, v_cache=v_cache,
                          slots=slots, out=out)
    out = _rope_common(q, positions, table, out)
    tokens, heads, dim = q.shape
    _typed(k, q.dtype, "k")
    _typed(v, q.dtype, "v")
    _typed(slots, torch.int64, "slots")
    if k.dim() != 3 or k.shape[0] != tokens or k.shape[2] != dim or v.shape != k.shape:
        _fail(f"k {tuple(k.shape)}, v {tuple(v.shape)}: [{tokens}, kv_heads, {dim}] is needed")
    if k.numel() and (k.stride(2) != 1 or v.stride(2) != 1):
        _fail("k and v have unit stride along a head")
    kv_heads = k.shape[1]
    _cache(k_cache, v_cache, q, kv_heads, dim)
    if slots.shape != (tokens,) or not slots.is_contiguous():
        _fail(f"slots {tuple(slots.shape)}: one contiguous int64 for each of {tokens} tokens is needed")
    cp, cs, ch, _ = k_cache.stride()
    d = B.LoraRopeDesc(q.data_ptr(), q.stride(0), q.stride(1), out.data_ptr(), out.stride(0), out.stride(1),
                       k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0), v.stride(1),
                       k_cache.data_ptr(), v_cache.data_ptr(), cp, cs, ch, slots.data_ptr(), k_cache.shape[0],
                       positions.data_ptr(), table.data_ptr(), table.shape[0], k_cache.shape[1], tokens, heads,
                       kv_heads, dim, table.shape[1], interleaved, 0, code)
    B.lora_rope(_byref(d), stream)
    return out


def tree_attention(q, k_cache, v_cache, page_table, ctx_lens, node_starts, tree_mask=None, scale=None, out=None):
    """Attention of drafted trees over the paged cache. Returns (out like q, lse fp32 [tokens, heads]).

    q [tokens, heads, head_dim]; page_table int32 [requests, pages of a request]; ctx_lens int32 [requests];
    node_starts int32 [requests + 1]: request b owns the rows node_starts[b] .. node_starts[b + 1], and its node j is
    key ctx_lens[b] + j of the cache; tree_mask int64 [tokens, words] (bit j % 64 of word j // 64: the row sees node
    j), None: node i sees nodes 0..i. scale: head_dim ** -0.5 by default."""
    code, stream = _start(q, k_cache=k_cache, v_cache=v_cache, page_table=page_table, ctx_lens=ctx_lens,
                          node_starts=node_starts, tree_mask=tree_mask, out=out)
    if q.dim() != 3 or (q.numel() and q.stride(2) != 1):
        _fail("q is [tokens, heads, head_dim] with unit stride along a head")
    tokens, heads, dim = q.shape
    if k_cache.dim() != 4:
        _fail("k_cache is [pages, page_size, kv_heads, head_dim]")
    n_pages, page_size, kv_heads, _ = k_cache.shape
    _cache(k_cache, v_cache, q, kv_heads, dim)
    _typed(page_table, torch.int32, "page_table")
    _typed(ctx_lens, torch.int32, "ctx_lens")
    _typed(node_starts, torch.int32, "node_starts")
    requests = ctx_lens.numel()
    if page_table.dim() != 2 or page_table.shape[0] != requests or (page_table.numel() and page_table.stride(1) != 1):
        _fail(f"page_table {tuple(page_table.shape)}: {requests} rows with unit stride are needed")
    if node_starts.shape != (requests + 1,) or ctx_lens.dim() != 1 or not node_starts.is_contiguous() \
            or not ctx_lens.is_contiguous():
        _fail(f"node_starts {tuple(node_starts.shape)}: {requests + 1} contiguous entries are needed")
    words = 0
    if tree_mask is not None:
        _typed(tree_mask, torch.int64, "tree_mask")
        if tree_mask.dim() != 2 or tree_mask.shape[0] != tokens or not tree_mask.is_contiguous():
            _fail(f"tree_mask {tuple(tree_mask.shape)}: a contiguous [{tokens}, words] is needed")
        words = tree_mask.shape[1]
    if out is None:
        out = torch.empty((tokens, heads, dim), dtype=q.dtype, device=q.device)
    else:
        _typed(out, q.dtype, "out")
        if out.shape != q.shape or (out.numel() and out.stride(2) != 1):
            _fail(f"out {tuple(out.shape)} with unit stride along a head: {tuple(q.shape)} is needed")
    lse = torch.empty((tokens, heads), dtype=torch.float32, device=q.device)
    size = B.lora_tree_attention_workspace_bytes(requests, tokens, heads, kv_heads, dim, code)
    workspace = torch.empty(size, dtype=torch.uint8, device=q.device)
    cp, cs, ch, _ = k_cache.stride()
    d = B.LoraTreeAttentionDesc(q.data_ptr(), q.stride(0), q.stride(1), k_cache.data_ptr(), v_cache.data_ptr(), cp, cs,
                                ch, n_pages, page_table.data_ptr(), page_table.stride(0), ctx_lens.data_ptr(),
                                node_starts.data_ptr(), None if tree_mask is None else tree_mask.data_ptr(),
                                out.data_ptr(), out.stride(0), out.stride(1), lse.data_ptr(), workspace.data_ptr(),
                                size, dim ** -0.5 if scale is None else scale, page_size, page_table.shape[1], words,
                                requests, tokens, heads, kv_heads, dim, code)
    B.lora_tree_attention(_byref(d), stream)
    return out, lse


def verify_drafts(target, draft, tokens, parents, node_starts, uniforms, noise, max_path):
    """Verify drafted trees. Returns int32 (path [requests, max_path], n_accepted [requests], next_token [requests]).

    target [nodes, vocab]: the target's probabilities after each node; draft the same for the rows the children were
    drawn from, or None (drafts chosen without chance); tokens, parents int32 [nodes]; node_starts int32
    [requests + 1]; uniforms fp32 [nodes] from U[0, 1); noise fp32 [requests, vocab], exponentially distributed."""
    code, stream = _start(target, draft=draft, tokens=tokens, parents=parents, node_starts=node_starts,
                          uniforms=uniforms, noise=noise)
    if target.dim() != 2 or (target.numel() and target.stride(1) != 1):
        _fail("target is [nodes, vocab] with unit stride along a row")
    nodes, vocab = target.shape
    if draft is not None:
        _typed(draft, target.dtype, "draft")
        if draft.shape != target.shape or (draft.numel() and draft.stride(1) != 1):
            _fail(f"draft {tuple(draft.shape)}: {tuple(target.shape)} with unit stride along a row is needed")
    _typed(tokens, torch.int32, "tokens")
    _typed(parents, torch.int32, "parents")
    _typed(node_starts, torch.int32, "node_starts")
    _typed(uniforms, torch.float32, "uniforms")
    _typed(noise, torch.float32, "noise")
    requests = node_starts.numel() - 1
    if tokens.shape != (nodes,) or parents.shape != (nodes,) or uniforms.shape != (nodes,) or requests < 0 \
            or node_starts.dim() != 1:
        _fail(f"tokens, parents and uniforms hold one entry for each of {nodes} nodes, node_starts requests + 1")
    if not (tokens.is_contiguous() and parents.is_contiguous() and uniforms.is_contiguous()
            and node_starts.is_contiguous()):
        _fail("tokens, parents, uniforms and node_starts are contiguous")
    if noise.shape != (requests, vocab) or (noise.numel() and noise.stride(1) != 1):
        _fail(f"noise {tuple(noise.shape)}: {(requests, vocab)} with unit stride along a row is needed")
    path = torch.empty((requests, max_path), dtype=torch.int32, device=target.device)
    result = torch.empty((2, requests), dtype=torch.int32, device=target.device)
    d = B.LoraVerifyDesc(target.data_ptr(), target.stride(0), None if draft is None else draft.data_ptr(),
                         0 if draft is None else draft.stride(0), tokens.data_ptr(), parents.data_ptr(),
                         node_starts.data_ptr(), uniforms.data_ptr(), noise.data_ptr(), noise.stride(0),
                         path.data_ptr(), result.data_ptr(), result.data_ptr() + 4 * requests, max_path, requests,
                         nodes, vocab, code)
    B.lora_verify_drafts(_byref(d), stream)
    return path, result[0], result[1]
