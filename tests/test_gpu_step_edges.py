"""What the drafted-token step's calls make of values, tensors and streams out of the ordinary, on the GPU."""
import numpy as np
import pytest

from tests import step_reference as ref
from tests.test_gpu_step import (ROUND, _check_linear, _check_tree, _check_verify, _close, _dev, _dt, _linear_inputs,  # noqa: F401
                                 _np, _rope_inputs, _run_tree, _run_verify, _tree_case, _verify_case, ops)

pytestmark = pytest.mark.gpu


# ---- tree_attention: rows that see keys, but no finite score -----------------------------------
# Rows of a request (nodes times query heads of a key/value head) choose the kernel: up to 16, up to 32, more. A context of
# 20 is one tile of keys, whose rows a block writes itself; 3000 are joined from parts.
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nodes", [3, 7, 40])
@pytest.mark.parametrize("ctx", [0, 20, 3000])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_tree_attention_query_row_not_finite(ops, value, ctx, nodes, dtype):  # noqa: F811
    """A NaN in a query row makes every score of the row NaN, an infinity makes some +inf or NaN: its output is NaN and
    its lse not finite, and no other row's changes by more than their tolerance."""
    import torch
    c = _tree_case([ctx], [nodes], 8, 2, 64, 16, dtype, seed=3)
    c["kc"][:, :, :, 5] = c["kc"][:, :, :, 5].abs() * (1.0 if value > 0 else -1.0)    # infinite scores are +inf
    want = _run_tree(ops, c)
    _check_tree(c, *want)
    c["q"][1, 2, 5] = value
    c["q"][nodes - 1, 7, 5] = value
    out, lse = _run_tree(ops, c)
    keep = torch.ones_like(lse, dtype=torch.bool)
    keep[1, 2] = keep[nodes - 1, 7] = False
    assert torch.isnan(out[~keep]).all() and not torch.isneginf(lse[~keep]).any() and not torch.isfinite(lse[~keep]).any()
    tol = 2.0 ** -6 if dtype == "bf16" else 2.0 ** -18      # both within their tolerance of the same values
    assert ((out - want[0]).abs()[keep] <= tol * (1 + want[0].abs()[keep])).all()
    assert ((lse - want[1]).abs()[keep] <= 2.0 ** -16 * (1 + want[1].abs()[keep])).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nodes", [3, 7, 40, 64])
def test_tree_attention_one_visible_key_nan(ops, nodes, dtype):  # noqa: F811
    """Nodes that see themselves alone, without context: the one whose key is NaN is NaN, the others see one key and
    are its value, and a node that sees nothing is 0 with lse = -inf."""
    import torch
    c = _tree_case([0], [nodes], 8, 2, 64, 16, dtype, seed=4)
    mask = np.zeros((nodes, 64), bool)
    mask[np.arange(nodes), np.arange(nodes)] = True
    mask[2] = False
    c["mask"], c["bits"] = mask, _dev(np.packbits(mask, axis=1, bitorder="little").view(np.int64).reshape(nodes, 1))
    c["kc"][int(c["table"][0, 0]), 1, 1, 9] = float("nan")
    out, lse = _run_tree(ops, c)
    assert torch.isnan(out[1, 4:]).all() and torch.isnan(lse[1, 4:]).all()
    assert torch.isfinite(out[1, :4]).all() and torch.isfinite(lse[1, :4]).all()
    assert not out[2].any() and torch.isneginf(lse[2]).all()
    for i in [i for i in range(nodes) if i not in (1, 2)]:
        v = c["vc"][int(c["table"][0, i // 16]), i % 16]
        assert torch.equal(out[i], v.repeat_interleave(4, 0)) and torch.isfinite(lse[i]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads", [2, 8])
def test_tree_attention_first_key_nan(ops, heads, dtype):  # noqa: F811
    """A chain of 700 nodes, cut into parts, whose first key is NaN in one head: every row of that head sees it, the
    first row sees nothing else."""
    import torch
    c = _tree_case([0], [700], heads, 2, 64, 16, dtype, seed=5)
    c["kc"][int(c["table"][0, 0]), 0, 1, 9] = float("nan")
    out, lse = _run_tree(ops, c, mask=False)
    assert torch.isnan(out[:, heads // 2:]).all() and torch.isnan(lse[:, heads // 2:]).all()
    assert torch.isfinite(out[:, :heads // 2]).all() and torch.isfinite(lse[:, :heads // 2]).all()


# ---- kernels that start early -----------------------------------------------------------------------
@pytest.mark.parametrize("adapters", ["none", "few", "all"])
def test_adapters_between_calls_with_inputs_ready(ops, adapters):  # noqa: F811
    """base_linear, the adapters' delta on its output with the inputs declared ready, the rotation of the result: each
    may start before the one before it has ended. The same as with a wait in between, whether or not a token of the
    batch has an adapter."""
    import torch
    from rank_adapter_apply_gb300 import binding as B
    from rank_adapter_apply_gb300.slots import LoraSlots
    tokens, d_in, d_out = 64, 4096, 2048
    x, qw, sc, z = _linear_inputs(tokens, d_in, d_out, 64, True, "bf16", seed=41)
    slots = LoraSlots([(d_in, d_out)], 4, 16, tokens)
    try:
        gen = torch.Generator().manual_seed(5)
        for s in range(4):
            slots.load_slot(s, [(torch.randn((16, d_in), generator=gen) / 64).bfloat16().pin_memory()],
                            [(torch.randn((d_out, 16), generator=gen) / 4).bfloat16().pin_memory()], 16, 16.0)
        slots.sync_uploads()
        every = {"none": tokens + 1, "few": 13, "all": 1}[adapters]
        idx = torch.tensor([t % 4 if t % every == every - 1 else -1 for t in range(tokens)], dtype=torch.int32, device="cuda")
        pos, table = torch.arange(tokens, dtype=torch.int32, device="cuda"), ops.rope_table(tokens, 128)
        xs = [x * (1 + i / 8) for i in range(6)]
        ys, turned = [torch.empty((tokens, d_out), dtype=x.dtype, device="cuda") for _ in xs], []
        torch.cuda.synchronize()
        with torch.cuda.stream(slots.compute):
            for wait in (True, False, False):
                B.lora_set_inputs_ready(slots.ctx, not wait)
                for i, xi in enumerate(xs):
                    for step in (lambda: ops.base_linear(xi, qw, sc, z, out=ys[i]), lambda: slots.apply(0, xi, ys[i], idx),
                                 lambda: turned.append(ops.rope(ys[i].view(tokens, 16, 128), pos, table))):
                        step()
                        if wait:
                            torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert slots.stats()["device_wait_timeouts"] == 0
        for i in range(len(xs), len(turned)):
            assert torch.equal(turned[i], turned[i % len(xs)]), i
    finally:
        slots.close()


# ---- verify_drafts: rows that start at different places within 16 bytes -----------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("requests,vocab", [(5, 301), (3, 40001), (400, 1003)])
@pytest.mark.parametrize("at", [(3, 6, 1), (0, 1, 0), (5, 0, 2), (1, 1, 3)])
def test_verify_rows_at_different_offsets(ops, at, requests, vocab, dtype):  # noqa: F811
    """Target, draft and noise inside wider rows of different widths, starting at different elements, with enough
    rejections that both the sums and the final pass read them; NaN lies around them."""
    import torch
    c = _verify_case(requests, 6, 3, vocab, dtype, True, seed=requests + vocab)
    c["u"][::2] = 0.97
    plain = _run_verify(ops, c, 6)
    _check_verify(c, plain, 6)
    assert (plain[1] == 0).any() and (plain[1] > 0).any()

    def inside(t, first, width):
        w = torch.full((t.shape[0], width), float("nan"), dtype=t.dtype, device="cuda")
        w[:, first:first + vocab] = t
        return w[:, first:first + vocab]
    got = ops.verify_drafts(inside(c["target"], at[0], vocab + 11), inside(c["draft"], at[1], vocab + 22), _dev(c["tokens"]),
                            _dev(c["parents"]), _dev(c["starts"]), _dev(c["u"]), inside(_dev(c["noise"]), at[2], vocab + 5), 6)
    _check_verify(c, got, 6)


# ---- tree_attention: as many keys as an int counts ----------------------------------------------------
@pytest.mark.parametrize("heads,dtype", [(8, "bf16"), (64, "bf16"), (8, "f32")])
def test_tree_attention_two_to_the_31_keys(ops, heads, dtype):  # noqa: F811
    """A context of 2^31 - 1 over one large page that fills the page table's row: the keys that an int can count are
    seen, and nothing outside the table is read. Each row of the page counts 32768 times, the last 64 one time less. A
    query of zero weighs all alike and the values are 0 or 1, so the sums of a block's share (2^31 / 304) are exact."""
    import torch
    page, dim = 65536, 8
    gen = torch.Generator(device="cuda").manual_seed(6)
    q = torch.zeros((1, heads, dim), device="cuda", dtype=_dt(dtype))
    kc = torch.randn((1, page, 1, dim), generator=gen, device="cuda").to(_dt(dtype))
    vc = torch.randint(0, 2, (1, page, 1, dim), generator=gen, device="cuda").to(_dt(dtype))
    i32 = dict(dtype=torch.int32, device="cuda")
    out, lse = ops.tree_attention(q, kc, vc, torch.zeros((1, (1 << 31) // page), **i32), torch.tensor([2**31 - 1], **i32),
                                  torch.tensor([0, 1], **i32))
    count = torch.full((page, 1), 32768.0, dtype=torch.float64, device="cuda")
    count[-64:] -= 1
    want = (vc[0, :, 0].double() * count).sum(0) / count.sum()
    tol = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -18
    assert ((out[0].double() - want).abs() <= tol * want).all()
    assert ((lse[0].double() - count.sum().log()).abs() <= 2.0 ** -18).all()


# ---- the count of waits that gave up --------------------------------------------------------------
def test_wait_timeouts_waits_for_every_stream(ops):  # noqa: F811
    """The count is read when the device is idle: work queued on a stream that no other waits for is done by then."""
    import torch
    from rank_adapter_apply_gb300 import binding as B
    side = torch.cuda.Stream()
    B.lora_step_wait_timeouts()
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)
    assert B.lora_step_wait_timeouts() == 0
    assert side.query()


# ---- what autograd has to know ------------------------------------------------------------------------
def _in_place_calls(ops):  # noqa: F811
    """(call, tensors that it writes in place) of each call that takes such tensors."""
    import torch
    x, qw, sc, z = _linear_inputs(3, 128, 20, 32, True, "bf16")
    y = torch.empty((3, 20), dtype=x.dtype, device="cuda")
    q, k, v, pos, kc, vc, slots = _rope_inputs(4, 4, 2, 64, 64, "bf16")
    turned, again, table = torch.empty_like(q), q.clone(), ops.rope_table(500, 64)
    c = _tree_case([5], [3], 4, 2, 64, 16, "bf16")
    out = torch.empty_like(c["q"])
    return [(lambda: ops.base_linear(x, qw, sc, z, out=y), [y]),
            (lambda: ops.rope(q, pos, table, out=turned), [turned]),
            (lambda: ops.rope(again, pos, table, out=again), [again]),
            (lambda: ops.rope_append(q, k, v, pos, table, kc, vc, slots, out=turned), [turned, kc, vc]),
            (lambda: _run_tree(ops, c, out=out), [out])]


def test_tensors_written_in_place_change_version(ops):  # noqa: F811
    """A tensor that a call writes (out, the caches) has a new version, by which autograd finds that a value saved for
    a backward pass is gone; tensors that are only read keep theirs."""
    import torch
    for i, (call, written) in enumerate(_in_place_calls(ops)):
        before = [t._version for t in written]
        call()
        assert all(t._version > b for t, b in zip(written, before)), i
    x, qw, sc, z = _linear_inputs(3, 128, 20, 32, True, "f32")
    y = torch.ones((3, 20), device="cuda", requires_grad=True)
    saved = (y * 2).exp()                        # exp keeps its result for the backward pass
    before = [t._version for t in (x, qw, sc, z)]
    ops.base_linear(x, qw, sc, z, out=saved.detach())
    assert [t._version for t in (x, qw, sc, z)] == before
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        saved.sum().backward()


def test_inference_tensors_are_written_as_before(ops):  # noqa: F811
    """Tensors of the inference mode have no version; they are taken inside the mode and outside."""
    import torch
    with torch.inference_mode():
        x, qw, sc, z = _linear_inputs(3, 128, 20, 32, True, "bf16")
        y = torch.zeros((3, 20), dtype=x.dtype, device="cuda")
        want = ops.base_linear(x, qw, sc, z)
        assert torch.equal(ops.base_linear(x, qw, sc, z, out=y), want)
    y2 = ops.base_linear(x, qw, sc, z, out=y)
    assert torch.equal(y2, want)


def test_forward_mode_tangents_are_refused(ops):  # noqa: F811
    """A dual tensor's tangent would be dropped: refused, like one that requires a gradient, unless forward mode is off."""
    import torch
    import torch.autograd.forward_ad as fwAD
    x, qw, sc, z = _linear_inputs(3, 128, 20, 32, True, "bf16")
    q, _, _, pos, _, _, _ = _rope_inputs(4, 4, 2, 64, 64, "bf16")
    table = ops.rope_table(500, 64)
    want = ops.base_linear(x, qw, sc, z)
    with fwAD.dual_level():
        dual = fwAD.make_dual(x, torch.ones_like(x))
        with pytest.raises(ValueError, match="tangent"):
            ops.base_linear(dual, qw, sc, z)
        with pytest.raises(ValueError, match="tangent"):
            ops.rope(fwAD.make_dual(q.contiguous(), torch.ones_like(q)), pos, table)
        assert torch.equal(ops.base_linear(fwAD.unpack_dual(dual).primal, qw, sc, z), want)


# ---- arguments --------------------------------------------------------------------------------------
def test_rope_table_zero_is_not_a_default(ops):  # noqa: F811
    """A frequency bound, or an original length, of zero is refused by the library, not replaced."""
    from rank_adapter_apply_gb300 import binding as B
    for scaling in ("pieces", "yarn"):
        for kw in (dict(low_freq=0), dict(low_freq=0.0, high_freq=4.0), dict(high_freq=0), dict(original=0)):
            with pytest.raises(B.LoraError):
                ops.rope_table(10, 64, scaling=scaling, factor=2.0, **{"original": 4096, **kw})


def test_flags_without_a_truth_value(ops):  # noqa: F811
    """A flag whose truth raises: that error, and nothing is queued."""
    import torch
    q, k, v, pos, kc, vc, slots = _rope_inputs(4, 4, 2, 64, 64, "bf16")
    table, two = ops.rope_table(500, 64), torch.tensor([0, 1])
    out = torch.full_like(q, 3.0)
    for call in (lambda: ops.rope(q, pos, table, interleaved=two, out=out), lambda: ops.rope(q, pos, table, inverse=two, out=out),
                 lambda: ops.rope_append(q, k, v, pos, table, kc, vc, slots, interleaved=two, out=out)):
        with pytest.raises(RuntimeError, match="ambiguous"):
            call()
    assert (out == 3.0).all() and (kc == 7.0).all()


# ---- base_linear: prompts -----------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,d_in,d_out,group,zeros", [(257, 640, 200, 128, True), (1000, 96, 130, 32, False),
                                                            (4096, 512, 129, 64, True)])
def test_base_linear_prompts(ops, tokens, d_in, d_out, group, zeros, dtype):  # noqa: F811
    """Many tiles of tokens, with rows that TMA takes and with rows at odd elements."""
    import torch
    x, qw, sc, z = _linear_inputs(tokens, d_in, d_out, group, zeros, dtype, seed=tokens)
    _check_linear(ops.base_linear(x, qw, sc, z), x, qw, sc, z, group, dtype)
    wide = torch.full((tokens, d_in + 9), float("nan"), dtype=x.dtype, device=x.device)
    wide[:, 5:5 + d_in] = x
    _check_linear(ops.base_linear(wide[:, 5:5 + d_in], qw, sc, z), x, qw, sc, z, group, dtype)


# ---- rope: the inverse ----------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot,kw", [
    (128, 128, {}), (80, 64, dict(scaling="linear", factor=4.0)), (30, 10, {}),
    (64, 64, dict(scaling="yarn", factor=16.0, original=4096)), (36, 20, dict(scaling="yarn", factor=8.0, original=1024))])
def test_rope_inverse_is_the_gradient(ops, dim, rot, kw, interleaved, dtype):  # noqa: F811
    """The rotation by the negative angle, with the table's magnitude (above 1 with "yarn"): for y = m R x it is m R^T, the
    gradient, and undoes y only where m is 1."""
    r = np.random.default_rng(dim + rot)
    g = _dev(r.standard_normal((50, 3, dim)), _dt(dtype))
    pos = _dev(r.integers(0, 500, 50).astype(np.int32))
    table = ops.rope_table(500, rot, **kw)
    got = _np(ops.rope(g, pos, table, interleaved=interleaved, inverse=True))
    tab, p = _np(table), pos.cpu().numpy()
    want, mass = ref.rope(_np(g), tab[p, :rot // 2], -tab[p, rot // 2:], interleaved)
    m = max(1.0, np.hypot(tab[0, 0], tab[0, rot // 2]))
    _close(got, want, (mass > 0) * (ROUND[dtype] * np.abs(want) + 2.0 ** -22 * mass * m))
    x = r.standard_normal((50, 3, dim))
    turned, _ = ref.rope(x, tab[p, :rot // 2], tab[p, rot // 2:], interleaved)
    both = (turned * _np(g)).sum(), (x * want).sum()                        # <m R x, g> = <x, m R^T g>
    assert abs(both[0] - both[1]) <= 1e-9 * np.abs(turned * _np(g)).sum()
    assert (m > 1.05) == (kw.get("scaling") == "yarn")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens", [1, 20])
@pytest.mark.parametrize("power", [-100, -103, -112, -122])
def test_base_linear_small_activations(ops, power, tokens, dtype):  # noqa: F811
    """Activations near the smallest normal numbers: an fp32 x loses less than 2^-125 of itself where its parts are
    subnormal, a bf16 x nothing; sums of 64ths may lose a few 2^-149 each."""
    x, qw, sc, z = _linear_inputs(tokens, 256, 70, 64, True, dtype, seed=7)
    x = (x.double() * 2.0 ** power).to(x.dtype)
    want, mass = ref.linear(_np(x), qw.cpu().numpy(), _np(sc), z.cpu().numpy(), 64)
    _, weights = ref.linear(np.ones((1, 256)), qw.cpu().numpy(), _np(sc), z.cpu().numpy(), 64)
    lost = 2.0 ** -125 if dtype == "f32" else 2.0 ** -133
    small = 2.0 ** -134 if dtype == "bf16" else 2.0 ** -149               # a result's own rounding below the normal numbers
    _close(_np(ops.base_linear(x, qw, sc, z)), want,
           ROUND[dtype] * np.abs(want) + 2.0 ** -22 * mass + lost * weights + 256 * 64 * 2.0 ** -149 + small)
