"""The drafted-token step's operators on the GPU against plain 64-bit forms.

Tolerances, per element. Rounding the result: at most half a unit in the last
place, 2^-9 |o| in bf16 (2^-8 is allowed) and 2^-24 |o| in fp32 (2^-23). An fp32
sum of n terms with random signs has partial sums of about mass / sqrt(n) (mass =
the sum of the terms' magnitudes), so n roundings of 2^-24 of them that are
independent in sign come to about 2^-24 mass; 2^-22 mass is allowed.
"""
import numpy as np
import pytest

from tests import step_reference as ref

pytestmark = pytest.mark.gpu

ROUND = {"bf16": 2.0 ** -8, "f32": 2.0 ** -23}


@pytest.fixture(scope="module")
def ops():
    from rank_adapter_apply_gb300 import build
    build.build()
    from rank_adapter_apply_gb300 import operators
    return operators


def _dt(name):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _dev(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def _np(t):
    return t.detach().double().cpu().numpy()


def _close(got, want, tol):
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4],
                           np.broadcast_to(tol, got.shape)[bad][:4])


# ---- base_linear ------------------------------------------------------------------------
def _linear_inputs(tokens, d_in, d_out, group, zeros, dtype, seed=0):
    r = np.random.default_rng(seed)
    x = _dev(r.standard_normal((tokens, d_in)), _dt(dtype))
    qw = _dev(r.integers(0, 256, (d_out, d_in // 2), dtype=np.uint8))
    sc = _dev(r.uniform(0.2, 1.5, (d_out, d_in // group)) / np.sqrt(d_in), _dt(dtype))
    z = _dev(r.integers(0, 16, (d_out, d_in // group), dtype=np.uint8)) if zeros else None
    return x, qw, sc, z


def _check_linear(y, x, qw, sc, z, group, dtype):
    want, mass = ref.linear(_np(x), qw.cpu().numpy(), _np(sc), None if z is None else z.cpu().numpy(), group)
    _close(_np(y), want, ROUND[dtype] * np.abs(want) + 2.0 ** -22 * mass)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,d_in,d_out,group,zeros", [
    (1, 32, 1, 32, False), (1, 4096, 520, 128, False), (2, 96, 17, 32, True), (3, 192, 129, 64, True),
    (7, 1152, 250, 128, True), (8, 4160, 64, 32, False), (9, 512, 300, 64, False), (16, 2176, 131, 128, True),
    (17, 14336, 48, 32, True), (31, 640, 257, 128, False), (33, 352, 65, 32, True), (64, 1024, 400, 64, True),
    (65, 256, 33, 128, False), (130, 4224, 40, 64, False), (1, 14336, 33, 32, True), (64, 5120, 1000, 128, False),
    (5, 8192, 1024, 64, True), (24, 4096, 4096, 128, False), (40, 1056, 2000, 32, False),
])
def test_base_linear(ops, tokens, d_in, d_out, group, zeros, dtype):
    x, qw, sc, z = _linear_inputs(tokens, d_in, d_out, group, zeros, dtype)
    _check_linear(ops.base_linear(x, qw, sc, z), x, qw, sc, z, group, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens", [1, 6, 20, 50])
def test_base_linear_strided_rows(ops, tokens, dtype):
    """Rows inside wider ones, starting at an odd element; what lies around them is NaN and stays untouched."""
    import torch
    x, qw, sc, z = _linear_inputs(tokens, 640, 77, 64, True, dtype, seed=3)
    wide = torch.full((tokens, 651), float("nan"), dtype=x.dtype, device=x.device)
    wide[:, 3:643] = x
    out = torch.full((tokens, 90), float("nan"), dtype=x.dtype, device=x.device)
    y = ops.base_linear(wide[:, 3:643], qw, sc, z, out=out[:, 5:82])
    assert y.data_ptr() == out[:, 5:].data_ptr()
    _check_linear(y, x, qw, sc, z, 64, dtype)
    assert torch.isnan(out[:, :5]).all() and torch.isnan(out[:, 82:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("tokens", [4, 9, 16, 17, 32, 33, 64, 65, 200])
def test_base_linear_more_tokens(ops, tokens, group, dtype):
    """Every tile of tokens with each group: rows of W past a tile of 128, columns past a block of 256, rows of x and y
    inside wider ones that keep the 16-byte alignment, zeros over the whole range the call takes."""
    import torch
    for d_in, d_out in ((group, 1), (256 + group, 128), (2560 + group, 300)):
        x, qw, sc, z = _linear_inputs(tokens, d_in, d_out, group, True, dtype, seed=tokens + d_out)
        z = torch.randint(0, 129, z.shape, dtype=torch.uint8, device=z.device) if d_out == 300 else z
        wide = torch.full((tokens, d_in + 24), float("nan"), dtype=x.dtype, device=x.device)
        wide[:, 8:8 + d_in] = x
        out = torch.full((tokens, d_out + 16), float("nan"), dtype=x.dtype, device=x.device)
        y = ops.base_linear(wide[:, 8:8 + d_in], qw, sc, z, out=out[:, 8:8 + d_out])
        _check_linear(y, x, qw, sc, z, group, dtype)
        assert torch.isnan(out[:, :8]).all() and torch.isnan(out[:, 8 + d_out:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens", [3, 19])
def test_base_linear_keeps_tokens_apart(ops, tokens, dtype):
    """An infinity or NaN in one token's row shows in that token's outputs alone."""
    import torch
    x, qw, sc, z = _linear_inputs(tokens, 256, 70, 128, False, dtype, seed=4)
    clean = ops.base_linear(x, qw, sc, z)
    x2 = x.clone()
    x2[1, 200] = float("nan")
    x2[2, 7] = float("inf")
    y = ops.base_linear(x2, qw, sc, z)
    assert torch.isnan(y[1]).all() and not torch.isfinite(y[2]).any()
    keep = [t for t in range(tokens) if t not in (1, 2)]
    assert torch.equal(y[keep], clean[keep])


def test_base_linear_no_tokens(ops):
    x, qw, sc, z = _linear_inputs(1, 64, 5, 32, False, "bf16")
    assert ops.base_linear(x[:0], qw, sc, z).shape == (0, 5)


def test_base_linear_repeats_bit_for_bit(ops):
    import torch
    x, qw, sc, z = _linear_inputs(12, 4096, 512, 128, True, "bf16", seed=8)
    first = ops.base_linear(x, qw, sc, z)
    for _ in range(5):
        assert torch.equal(ops.base_linear(x, qw, sc, z), first)


# ---- rotary positions ---------------------------------------------------------------------
@pytest.mark.parametrize("n,rot,kw", [
    (1, 2, {}), (300, 64, {}), (131, 128, dict(base=500000.0)), (200, 64, dict(scaling="linear", factor=4.0)),
    (200, 64, dict(scaling="base", factor=8.0)), (90, 96, dict(base=1e6)),
    (150, 128, dict(base=500000.0, scaling="pieces", factor=8.0, original=8192, low_freq=1.0, high_freq=4.0)),
    (150, 128, dict(scaling="yarn", factor=16.0, original=4096, low_freq=1.0, high_freq=32.0)),
    (65, 80, dict(scaling="yarn", factor=1.0, original=2048, low_freq=1.0, high_freq=32.0)),
])
def test_rope_table(ops, n, rot, kw):
    """Rounding to fp32 once (2^-24 of the magnitude), and 1e-9 for the angles' roundings in double."""
    got = _np(ops.rope_table(n, rot, **kw))
    args = dict(base=10000.0)
    args.update(kw)
    cos, sin = ref.rope_table(n, rot, **args)
    mag = max(np.abs(cos[0]).max(), 1.0)
    _close(got, np.concatenate([cos, sin], 1), 2.0 ** -24 * mag + 1e-9)


def test_rope_table_far_positions(ops):
    """At positions of a million the angles are still right (a product in fp32 would be 0.06 rad off)."""
    n = 1 << 20
    got = ops.rope_table(n, 16, base=10000.0)[-3:].double().cpu().numpy()
    f = 10000.0 ** (-np.arange(8) / 8.0)
    angle = np.arange(n - 3, n)[:, None] * f
    _close(got, np.concatenate([np.cos(angle), np.sin(angle)], 1), 2.0 ** -24 + 1e-8)


def _rope_inputs(tokens, heads, kv, dim, rot, dtype, n_pos=500, page=16, seed=0):
    import torch
    r = np.random.default_rng(seed)
    qkv = _dev(r.standard_normal((tokens, (heads + 2 * kv) * dim)), _dt(dtype))
    q = qkv[:, :heads * dim].view(tokens, heads, dim)
    k = qkv[:, heads * dim:(heads + kv) * dim].view(tokens, kv, dim)
    v = qkv[:, (heads + kv) * dim:].view(tokens, kv, dim)
    pos = _dev(r.integers(0, n_pos, tokens).astype(np.int32))
    pages = tokens // page + 2
    kc = torch.full((pages, page, kv, dim), 7.0, dtype=_dt(dtype), device="cuda")
    vc = torch.full_like(kc, 9.0)
    slots = _dev(r.permutation(pages * page)[:tokens].astype(np.int64))
    return q, k, v, pos, kc, vc, slots


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,heads,kv,dim,rot,page", [
    (1, 1, 1, 2, 2, 1), (1, 32, 8, 128, 128, 64), (5, 4, 2, 64, 32, 16), (33, 7, 1, 80, 64, 16), (70, 6, 3, 96, 96, 8),
    (9, 5, 5, 50, 22, 3), (200, 28, 4, 128, 64, 32), (3, 2, 1, 36, 20, 16), (1000, 8, 2, 128, 128, 64),
    (17, 3, 3, 72, 8, 16), (12, 1, 1, 7, 6, 4),
])
def test_rope_append(ops, tokens, heads, kv, dim, rot, page, interleaved, dtype):
    q, k, v, pos, kc, vc, slots = _rope_inputs(tokens, heads, kv, dim, rot, dtype, page=page)
    table = ops.rope_table(500, rot)
    want_k, want_v = _np(kc), _np(vc)
    out = ops.rope_append(q, k, v, pos, table, kc, vc, slots, interleaved=interleaved)
    tab, p, s = _np(table), pos.cpu().numpy(), slots.cpu().numpy()
    cos, sin = tab[p, :rot // 2], tab[p, rot // 2:]
    yq, mq = ref.rope(_np(q), cos, sin, interleaved)
    yk, mk = ref.rope(_np(k), cos, sin, interleaved)
    _close(_np(out), yq, (mq > 0) * (ROUND[dtype] * np.abs(yq) + 2.0 ** -22 * mq))
    mass = np.zeros_like(want_k)
    want_k[s // page, s % page], mass[s // page, s % page] = yk, mk
    want_v[s // page, s % page] = _np(v)
    _close(_np(kc), want_k, (mass > 0) * (ROUND[dtype] * np.abs(want_k) + 2.0 ** -22 * mass))
    _close(_np(vc), want_v, 0.0)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(128, 128), (80, 64), (30, 10)])
def test_rope_in_place_and_inverse(ops, dim, rot, interleaved):
    """In place gives the same bits; the inverse undoes it (two fp32 rotations: 2^-21 of the pair)."""
    import torch
    q = _rope_inputs(40, 6, 2, dim, rot, "f32")[0]
    pos = torch.arange(40, dtype=torch.int32, device="cuda") * 11
    table = ops.rope_table(500, rot)
    y = ops.rope(q, pos, table, interleaved=interleaved)
    z = q.clone()
    ops.rope(z, pos, table, interleaved=interleaved, out=z)
    assert torch.equal(y, z)
    back = ops.rope(y, pos, table, interleaved=interleaved, inverse=True)
    _close(_np(back), _np(q), 2.0 ** -21 * 2 * np.abs(_np(q)).max())


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_gradient(ops, interleaved):
    """The inverse rotation of g is the gradient of sum(g * rope(x)): against the formula's in 64 bits, and against
    central differences of the kernel itself (exact for a linear map up to 2^-22 of the sum over a step of 1)."""
    import torch
    r = np.random.default_rng(5)
    x = _dev(r.standard_normal((3, 2, 24)), torch.float32)
    g = _dev(r.standard_normal((3, 2, 24)), torch.float32)
    pos = _dev(np.array([0, 17, 400], np.int32))
    table = ops.rope_table(500, 16)
    grad = _np(ops.rope(g, pos, table, interleaved=interleaved, inverse=True))
    tab, p = _np(table), pos.cpu().numpy()
    want, mass = ref.rope(_np(g), tab[p, :8], -tab[p, 8:], interleaved)
    _close(grad, want, 2.0 ** -22 * mass + 2.0 ** -23 * np.abs(want))
    for at in [(0, 0, 0), (1, 1, 3), (2, 0, 15), (2, 1, 20), (1, 0, 8)]:
        h = torch.zeros_like(x)
        h[at] = 1.0
        up = (ops.rope(x + h, pos, table, interleaved=interleaved).double() * g.double()).sum().item()
        down = (ops.rope(x - h, pos, table, interleaved=interleaved).double() * g.double()).sum().item()
        assert abs((up - down) / 2 - grad[at]) <= 2.0 ** -22 * 16 * np.abs(_np(g)).max() * 3


def test_rope_entries_out_of_range(ops):
    """Positions outside the table write nothing; slots outside the cache write no cache row."""
    import torch
    for dtype, dim in [("bf16", 64), ("f32", 24)]:
        q, k, v, pos, kc, vc, slots = _rope_inputs(8, 2, 1, dim, 8, dtype)
        table = ops.rope_table(500, 8)
        good_k, good_v = kc.clone(), vc.clone()
        good = ops.rope_append(q, k, v, pos, table, good_k, good_v, slots)
        pos2, slots2 = pos.clone(), slots.clone()
        pos2[1], pos2[4] = -1, 500
        slots2[2], slots2[6] = -1, kc.shape[0] * kc.shape[1]
        out = torch.full_like(good, 5.0)
        ops.rope_append(q, k, v, pos2, table, kc, vc, slots2, out=out)
        want = good.clone()
        want[[1, 4]] = 5.0
        assert torch.equal(out, want)
        for lost in (1, 2, 4, 6):
            s = int(slots[lost])
            good_k[s // 16, s % 16], good_v[s // 16, s % 16] = 7.0, 9.0
        assert torch.equal(kc, good_k) and torch.equal(vc, good_v)


def test_rope_offsets_past_32_bits(ops):
    """A cache row more than 2^31 elements from the cache's start."""
    import torch
    page, kv, dim = 64, 8, 128
    pages = (1 << 31) // (page * kv * dim) + 3
    kc = torch.empty((pages, page, kv, dim), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    q, k, v, pos, _, _, _ = _rope_inputs(2, 8, kv, dim, dim, "bf16")
    slots = torch.tensor([pages * page - 1, 5], dtype=torch.int64, device="cuda")
    table = ops.rope_table(500, dim)
    ops.rope_append(q, k, v, pos, table, kc, vc, slots)
    want = ops.rope(k, pos, table)
    assert torch.equal(kc[-1, -1], want[0]) and torch.equal(vc[-1, -1], v[0]) and torch.equal(kc[0, 5], want[1])


# ---- attention of drafted trees -------------------------------------------------------------
def _tree_case(ctx, nodes, heads, kv, dim, page, dtype, words=1, seed=0, spread=1.0, spare_rows=0):
    """Ragged requests with random trees; every cache row that no query sees is NaN."""
    import torch
    r = np.random.default_rng(seed)
    ctx, nodes = list(ctx), list(nodes)
    per = max(1, max(-(-(c + n) // page) for c, n in zip(ctx, nodes)))
    pages = per * len(ctx) + 2
    table = r.permutation(pages)[:per * len(ctx)].reshape(len(ctx), per).astype(np.int32)
    kc = np.full((pages, page, kv, dim), np.nan)
    vc = np.full_like(kc, np.nan)
    starts = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int64)
    total = int(starts[-1]) + spare_rows
    mask = np.zeros((max(total, 1), words * 64), bool)
    for b in range(len(ctx)):
        for p in range(ctx[b] + nodes[b]):
            kc[table[b, p // page], p % page] = r.standard_normal((kv, dim))
            vc[table[b, p // page], p % page] = r.standard_normal((kv, dim))
        for i in range(nodes[b]):
            t = starts[b] + i
            if i > 0:
                mask[t] = mask[starts[b] + r.integers(max(0, i - 4), i)]
            if i < 64 * words:
                mask[t, i] = True
    q = r.standard_normal((total, heads, dim)) * spread
    bits = np.packbits(mask, axis=1, bitorder="little").view(np.int64).reshape(mask.shape[0], words)[:total]
    return dict(q=_dev(q, _dt(dtype)), kc=_dev(kc, _dt(dtype)), vc=_dev(vc, _dt(dtype)), table=table, ctx=ctx,
                starts=starts, mask=mask, bits=_dev(bits), dtype=dtype, torch=torch)


def _run_tree(ops, c, mask=True, out=None, scale=None):
    return ops.tree_attention(c["q"], c["kc"], c["vc"], _dev(c["table"]), _dev(np.array(c["ctx"], np.int32)),
                              _dev(c["starts"].astype(np.int32)), c["bits"] if mask else None, scale=scale, out=out)


def _check_tree(c, out, lse, mask=True, scale=None):
    """On top of the rounding: P in bf16 (2^-9 relative, 2^-8 allowed) for bf16 caches, and scores whose errors
    (2^-22 of the largest score mass, times 4 for the scaling and the exponential) shift every weight."""
    dim = c["q"].shape[2]
    scale = dim ** -0.5 if scale is None else scale
    sees = (lambda t, i, j: j < c["mask"].shape[1] and c["mask"][t, j]) if mask else (lambda t, i, j: j <= i)
    want, want_lse, mass, reach = ref.tree_attention(_np(c["q"]), _np(c["kc"]), _np(c["vc"]), c["table"], c["ctx"],
                                                     c["starts"], sees, scale)
    part = 2.0 ** -8 if c["dtype"] == "bf16" else 2.0 ** -21
    owned = ~np.isnan(want_lse).any(1)
    got, got_lse = _np(out)[owned], _np(lse)[owned]
    tol = ROUND[c["dtype"]] * np.abs(want) + (part + 2.0 ** -20 * (1 + reach[:, :, None])) * mass
    _close(got, want[owned], tol[owned])
    want_lse = want_lse[owned]
    empty = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(got_lse), empty) and (got[empty] == 0).all()
    _close(np.where(empty, 0, got_lse), np.where(empty, 0, want_lse),
           2.0 ** -20 * (1 + reach[owned] + np.abs(np.where(empty, 0, want_lse))))


TREES = [
    ([0], [1], 1, 1, 8, 16), ([1], [1], 4, 2, 64, 1), ([5], [3], 8, 2, 128, 16), ([63, 64, 65], [1, 1, 1], 8, 8, 64, 64),
    ([0, 17, 200], [4, 0, 9], 14, 2, 96, 16), ([130], [16], 32, 8, 128, 64), ([257, 1, 40], [7, 33, 2], 16, 2, 72, 48),
    ([700], [64], 4, 1, 128, 32), ([31, 500, 3, 77, 0], [5, 6, 20, 1, 12], 24, 3, 64, 128), ([1500], [2], 16, 8, 128, 16),
    ([0, 0], [64, 1], 6, 6, 40, 16), ([90] * 20, [3] * 20, 4, 4, 128, 16), ([2100, 33], [17, 40], 8, 1, 128, 64),
    # more than 32 rows a head: whole nodes in a tile (groups of 7, 3 and 48), pages of 8, 24 and 128 places, pages that
    # no box of eight rows fits, many short units, a unit over many blocks
    ([150, 3], [40, 64], 14, 2, 128, 8), ([64, 65, 0, 1], [33, 20, 64, 64], 9, 3, 72, 24), ([500], [3], 48, 1, 96, 128),
    ([77, 200], [30, 21], 8, 2, 64, 12), ([1, 2, 3, 4, 5, 6, 7, 8], [11] * 8, 32, 8, 128, 32), ([6000], [64], 16, 1, 128, 64),
    ([40, 900, 0], [64, 1, 30], 64, 8, 128, 16), ([127, 128, 129], [48, 64, 49], 130, 1, 64, 16),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ctx,nodes,heads,kv,dim,page", TREES)
def test_tree_attention(ops, ctx, nodes, heads, kv, dim, page, dtype):
    c = _tree_case(ctx, nodes, heads, kv, dim, page, dtype, seed=len(ctx) + dim)
    out, lse = _run_tree(ops, c)
    _check_tree(c, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ctx,nodes,heads,kv,dim,page", [TREES[2], TREES[6], TREES[7], ([3, 0], [150, 70], 4, 2, 64, 16)])
def test_tree_attention_chain(ops, ctx, nodes, heads, kv, dim, page, dtype):
    """Without a mask node i sees nodes 0..i, however many there are."""
    c = _tree_case(ctx, nodes, heads, kv, dim, page, dtype, seed=2)
    _check_tree(c, *_run_tree(ops, c, mask=False), mask=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nodes", [[1, 300, 9], [40, 130, 64, 700, 3], [513] * 2])
def test_tree_attention_many_row_tiles(ops, nodes, dtype):
    """Chains of one to dozens of row tiles in one call, over contexts that end anywhere in a tile of keys."""
    c = _tree_case([(137 * i) % 700 for i in range(len(nodes))], nodes, 8, 2, 64, 32, dtype, seed=len(nodes))
    _check_tree(c, *_run_tree(ops, c, mask=False), mask=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("requests", [33, 400])
def test_tree_attention_many_requests(ops, requests, dtype):
    """More requests than a warp or a block has threads, some without nodes, with one to three row tiles."""
    nodes = [(7 * i) % 41 for i in range(requests)]
    c = _tree_case([(11 * i) % 90 for i in range(requests)], nodes, 8, 2, 64, 16, dtype, seed=requests)
    _check_tree(c, *_run_tree(ops, c))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tree_attention_wide_masks(ops, dtype):
    """Two and three mask words; nodes past the words are seen by nobody."""
    c = _tree_case([20, 5], [100, 30], 4, 2, 64, 16, dtype, words=2, seed=3)
    _check_tree(c, *_run_tree(ops, c))
    c = _tree_case([9], [200], 2, 1, 128, 32, dtype, words=3, seed=4)
    _check_tree(c, *_run_tree(ops, c))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tree_attention_rows_without_keys(ops, dtype):
    """No context and an empty mask: zeros and -inf, beside rows that see keys."""
    c = _tree_case([0, 40, 0], [5, 3, 2], 8, 4, 64, 16, dtype, seed=5)
    c["mask"][[1, 3, 8, 9]] = False
    c["mask"][6] = False                 # sees its context alone
    c["bits"] = _dev(np.packbits(c["mask"], axis=1, bitorder="little").view(np.int64).reshape(-1, 1))
    out, lse = _run_tree(ops, c)
    _check_tree(c, out, lse)
    assert np.isneginf(_np(lse)[[1, 3, 8, 9]]).all() and not _np(out)[[1, 3, 8, 9]].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tree_attention_bad_entries(ops, dtype):
    """Page ids out of range and keys past the page table are not seen; a negative context is none; rows of no
    request stay as they were."""
    import torch
    c = _tree_case([50, 70, 20], [4, 3, 6], 4, 2, 64, 16, dtype, seed=6, spare_rows=3)
    c["table"] = c["table"].copy()
    c["table"][0, 1], c["table"][1, 2], c["table"][1, 4] = -1, c["kc"].shape[0], 1 << 30
    c["table"] = c["table"][:, :4]       # request 1: keys 64.. are past its row
    out = torch.full(c["q"].shape, 3.0, dtype=c["q"].dtype, device="cuda")
    out, lse = _run_tree(ops, c, out=out)
    _check_tree(c, out, lse)
    assert (out[-3:] == 3.0).all()
    # request 2's tree lies at keys 20..25 of its pages; with a context of -5 it is read from key 0 on
    c = _tree_case([0, 3], [4, 3], 4, 2, 64, 16, dtype, seed=7)
    want = _run_tree(ops, c)
    c["ctx"][0] = -5
    got = _run_tree(ops, c)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nodes", [[5, 12], [25, 60]])
def test_tree_attention_layouts(ops, nodes, dtype):
    """q inside a fused projection's rows, a cache with heads before places, keys and values interleaved, an output
    with padded heads: the same as from contiguous tensors."""
    import torch
    c = _tree_case([100, 33], nodes, 8, 2, 64, 16, dtype, seed=8)
    want = _run_tree(ops, c)
    _check_tree(c, *want)
    total = sum(nodes)
    q = torch.full((total, 3, 8, 64), float("nan"), dtype=c["q"].dtype, device="cuda")
    q[:, 1] = c["q"]
    both = torch.stack([c["kc"].permute(0, 2, 1, 3), c["vc"].permute(0, 2, 1, 3)], 1).contiguous()
    d = dict(c, q=q[:, 1], kc=both[:, 0].permute(0, 2, 1, 3), vc=both[:, 1].permute(0, 2, 1, 3))
    out = torch.full((total, 8, 80), 4.0, dtype=c["q"].dtype, device="cuda")
    got = _run_tree(ops, d, out=out[:, :, :64])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert (out[:, :, 64:] == 4.0).all()
    # queries with tokens inside heads, and a cache with places outermost
    e = dict(c, q=c["q"].permute(1, 0, 2).contiguous().permute(1, 0, 2),
             kc=c["kc"].permute(1, 0, 2, 3).contiguous().permute(1, 0, 2, 3),
             vc=c["vc"].permute(1, 0, 2, 3).contiguous().permute(1, 0, 2, 3))
    _check_tree(e, *_run_tree(ops, e))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("spread", [40.0, 1e-3])
@pytest.mark.parametrize("nodes", [[6, 3], [60, 33]])
@pytest.mark.parametrize("scale", [0.5, -0.3, 0.0])
def test_tree_attention_score_range(ops, scale, nodes, spread, dtype):
    """Scores of hundreds (one key takes all the weight, and the running maximum moves often) and of nothing; other
    scales, negative and zero."""
    c = _tree_case([300, 64], nodes, 8, 2, 128, 16, dtype, seed=9, spread=spread)
    _check_tree(c, *_run_tree(ops, c, scale=scale), scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,nodes", [(64, 2), (128, 3), (72, 9), (128, 20), (64, 60)])
def test_tree_attention_poison_in_skipped_keys(ops, dim, nodes, dtype):
    """Infinities and NaN in tree keys reach the rows that see those keys and no other row: two forks of the root, a
    poisoned value in one of them, a poisoned key in the other, and both in a node that nobody sees."""
    import torch
    c = _tree_case([70], [nodes + 2], 8, 2, dim, 16, dtype, seed=13)
    n = nodes + 2
    mask = np.zeros((n, 64), bool)
    mask[:, 0] = True
    for i in range(1, n):
        mask[i, i] = True
    mask[n - 1, n - 1] = False
    c["mask"], c["bits"] = mask, _dev(np.packbits(mask, axis=1, bitorder="little").view(np.int64).reshape(n, 1))
    want = _run_tree(ops, c)
    _check_tree(c, *want)

    def at(node):
        return int(c["table"][0, (70 + node) // 16]), (70 + node) % 16
    c["vc"][at(1)[0], at(1)[1], 0, 5] = float("inf")
    c["kc"][at(2)[0], at(2)[1], 1, 3] = float("nan")
    c["kc"][at(n - 1)[0], at(n - 1)[1]] = float("-inf")
    c["vc"][at(n - 1)[0], at(n - 1)[1]] = float("nan")
    out, lse = _run_tree(ops, c)
    assert torch.isinf(out[1, :4, 5]).all() and (out[1, :4, 5] > 0).all()
    assert torch.isnan(lse[2, 4:]).all() and torch.isnan(out[2, 4:]).all()
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[1, :4, 5] = False
    keep[2, 4:] = False
    tol = 2.0 ** -6 if dtype == "bf16" else 2.0 ** -18      # both within their tolerance of the same values
    assert ((out - want[0]).abs()[keep] <= tol * (1 + want[0].abs()[keep])).all()
    assert torch.equal(lse[[0, 1] + list(range(3, n))], want[1][[0, 1] + list(range(3, n))])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nodes", [3, 7, 40])
@pytest.mark.parametrize("at", [10, 66])
def test_tree_attention_poison_in_context(ops, at, nodes, dtype):
    """An infinity in a context key's value reaches every row of its head, and no other head, whether the key lies in a
    tile of context keys alone or beside tree keys."""
    import torch
    c = _tree_case([70], [nodes], 8, 2, 128, 16, dtype, seed=14)
    want = _run_tree(ops, c)
    c["vc"][int(c["table"][0, at // 16]), at % 16, 0, 5] = float("-inf")
    out, lse = _run_tree(ops, c)
    assert torch.isinf(out[:, :4, 5]).all() and (out[:, :4, 5] < 0).all()
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[:, :4, 5] = False
    tol = 2.0 ** -6 if dtype == "bf16" else 2.0 ** -18
    assert ((out - want[0]).abs()[keep] <= tol * (1 + want[0].abs()[keep])).all()
    assert torch.equal(lse, want[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tree_attention_long_context(ops, dtype):
    """A context long enough to be split over many blocks, beside short ones."""
    for nodes in ([3, 5, 2], [20, 33, 14]):
        c = _tree_case([9000, 3, 400], nodes, 4, 1, 64, 64, dtype, seed=10)
        _check_tree(c, *_run_tree(ops, c))


def test_tree_attention_offsets_past_32_bits(ops):
    """Pages more than 2^31 elements into the cache."""
    import torch
    page, kv, dim = 64, 8, 128
    far = (1 << 31) // (page * kv * dim) + 1
    kc = torch.empty((far + 5, page, kv, dim), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    for nodes in (4, 30):
        c = _tree_case([100], [nodes], 16, kv, dim, page, "bf16", seed=11)
        kc[far:far + c["kc"].shape[0]], vc[far:far + c["kc"].shape[0]] = c["kc"], c["vc"]
        want = _run_tree(ops, c)
        d = dict(c, kc=kc, vc=vc, table=c["table"] + far)
        got = _run_tree(ops, d)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_tree_attention_repeats_bit_for_bit(ops):
    import torch
    from rank_adapter_apply_gb300 import binding as B
    for nodes in ([9, 3], [60, 14]):
        c = _tree_case([1000, 77], nodes, 16, 4, 128, 16, "bf16", seed=12)
        first = _run_tree(ops, c)
        for _ in range(4):
            again = _run_tree(ops, c)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    assert B.lora_step_wait_timeouts() == 0


# ---- verification ---------------------------------------------------------------------------
def _verify_case(requests, nodes, children, vocab, dtype, drafts, seed=0, sharp=2.0):
    import torch
    r = np.random.default_rng(seed)
    sizes = [nodes if b == 0 else int(r.integers(0, nodes + 1)) for b in range(requests)]
    starts = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    total = int(starts[-1])
    logits = r.standard_normal((total, vocab)) * sharp
    other = logits + 0.8 * r.standard_normal((total, vocab))

    def soft(z):
        e = np.exp(z - z.max(1, keepdims=True))
        return torch.from_numpy(e / e.sum(1, keepdims=True)).cuda().to(_dt(dtype))
    target, draft = soft(logits), soft(other)
    q = _np(draft)
    parents, tokens = np.full(total, -1, np.int32), np.zeros(total, np.int32)
    for b in range(requests):
        for i in range(1, sizes[b]):
            parents[starts[b] + i] = max(0, i - int(r.integers(1, children + 1)))
            row = q[starts[b] + parents[starts[b] + i]]
            tokens[starts[b] + i] = r.choice(vocab, p=row / row.sum())
    u = r.uniform(size=total).astype(np.float32)
    noise = np.maximum(r.exponential(size=(requests, vocab)), 1e-20).astype(np.float32)
    return dict(target=target, draft=draft if drafts else None, tokens=tokens, parents=parents, starts=starts, u=u,
                noise=noise)


def _run_verify(ops, c, max_path):
    return ops.verify_drafts(c["target"], c["draft"], _dev(c["tokens"]), _dev(c["parents"]), _dev(c["starts"]),
                             _dev(c["u"]), _dev(c["noise"]), max_path)


def _check_verify(c, got, max_path):
    """Equal wherever the 64-bit decisions are not within 2^-16 of their other outcome (sums of a vocabulary in fp32
    and the residual's differences come to a few 2^-20)."""
    path, count, chosen, margin = ref.verify(_np(c["target"]), None if c["draft"] is None else _np(c["draft"]),
                                             c["tokens"], c["parents"], c["starts"], c["u"].astype(np.float64),
                                             c["noise"].astype(np.float64), max_path)
    sure = margin > 2.0 ** -16
    assert sure.mean() > 0.9
    got = [g.cpu().numpy() for g in got]
    assert np.array_equal(got[0][sure], path[sure])
    assert np.array_equal(got[1][sure], count[sure])
    assert np.array_equal(got[2][sure], chosen[sure])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("drafts", [True, False])
@pytest.mark.parametrize("requests,nodes,children,vocab", [
    (1, 1, 1, 1), (1, 5, 1, 2), (3, 4, 1, 7), (40, 6, 1, 1000), (40, 13, 3, 333), (25, 16, 4, 4099), (60, 9, 2, 30),
    (2, 60, 8, 5000), (7, 5, 4, 32001), (150, 7, 3, 64),
])
def test_verify_drafts(ops, requests, nodes, children, vocab, drafts, dtype):
    c = _verify_case(requests, nodes, children, vocab, dtype, drafts, seed=requests + vocab)
    _check_verify(c, _run_verify(ops, c, nodes), nodes)


@pytest.mark.parametrize("drafts", [True, False])
def test_verify_max_path(ops, drafts):
    """The walk stops at max_path nodes and draws the next token from that node's own row."""
    for most in (0, 1, 2):
        c = _verify_case(30, 8, 2, 500, "f32", drafts, seed=20, sharp=6.0)
        _check_verify(c, _run_verify(ops, c, most), most)


def test_verify_strides_and_order(ops):
    """Rows inside wider ones; a tie of the race goes to the lowest index."""
    import torch
    c = _verify_case(12, 6, 2, 301, "f32", True, seed=21)
    want = [g.clone() for g in _run_verify(ops, c, 6)]

    def wide(t):
        w = torch.full((t.shape[0], 320), float("nan"), device="cuda")
        w[:, 3:304] = t
        return w[:, 3:304]
    got = ops.verify_drafts(wide(c["target"]), wide(c["draft"]), _dev(c["tokens"]), _dev(c["parents"]),
                            _dev(c["starts"]), _dev(c["u"]), wide(_dev(c["noise"])), 6)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    flat = torch.full((1, 5000), 1 / 5000, device="cuda")
    ones = torch.ones((1, 5000), device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = ops.verify_drafts(flat, None, zero, zero - 1, torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                            torch.zeros(1, device="cuda"), ones, 3)
    assert got[2].tolist() == [0] and got[0].tolist() == [[-1, -1, -1]]


def test_verify_degenerate_rows(ops):
    """Equal rows leave no residual after a forced rejection: the row itself is drawn from. A row without a positive
    probability gives -1. Tokens and parents out of range are no one's children. Requests without nodes."""
    import torch
    i32 = dict(dtype=torch.int32, device="cuda")
    p = torch.zeros((4, 10), device="cuda")
    p[0, 2], p[0, 5] = 0.5, 0.5
    p[1, 7] = 1.0
    p[2, 3] = 1.0
    u = torch.tensor([0.0, 1.0, 0.0, 0.0], device="cuda")    # 1.0: above U[0, 1), so never accepted
    noise = torch.ones((3, 10), device="cuda")
    noise[0, 2] = 2.0
    got = ops.verify_drafts(p, p.clone(), torch.tensor([0, 2, 0, 0], **i32), torch.tensor([-1, 0, -1, -1], **i32),
                            torch.tensor([0, 2, 2, 4], **i32), u, noise, 2)
    assert got[1].tolist() == [0, 0, 0] and got[2].tolist() == [5, -1, 3]
    zero = torch.zeros((1, 10), device="cuda")
    got = ops.verify_drafts(zero, None, torch.tensor([0], **i32), torch.tensor([-1], **i32),
                            torch.tensor([0, 1], **i32), u[:1], noise[:1], 2)
    assert got[2].tolist() == [-1]
    tokens = torch.tensor([0, -1, 10, 7], **i32)
    parents = torch.tensor([-1, 0, 0, 3], **i32)
    got = ops.verify_drafts(p, None, tokens, parents, torch.tensor([0, 4], **i32), torch.zeros(4, device="cuda"),
                            noise[:1], 3)
    assert got[1].tolist() == [0] and got[2].tolist() == [5]


def test_verify_is_distributed_as_the_target(ops):
    """Over many requests with one pair of rows, the first token out (accepted or drawn) follows the target: each
    share is within five standard deviations of its probability."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(3)
    n, vocab = 20000, 8
    p = torch.softmax(torch.randn(vocab, generator=g, device="cuda"), 0)
    q = torch.softmax(torch.randn(vocab, generator=g, device="cuda"), 0)
    target, draft = p.expand(3 * n, vocab), q.expand(3 * n, vocab)
    drafted = torch.multinomial(q, 3 * n, replacement=True, generator=g).int()
    parents = torch.tensor([-1, 0, 0], dtype=torch.int32, device="cuda").repeat(n)
    starts = torch.arange(n + 1, dtype=torch.int32, device="cuda") * 3
    u = torch.rand(3 * n, generator=g, device="cuda")
    noise = torch.empty((n, vocab), device="cuda").exponential_(generator=g)
    path, count, nxt = ops.verify_drafts(target, draft, drafted, parents, starts, u, noise, 1)
    at = (starts[:-1].long() + path[:, 0].clamp(min=0).long())
    first = torch.where(count > 0, drafted[at], nxt)
    share = torch.bincount(first.long(), minlength=vocab).double() / n
    sd = (p.double() * (1 - p.double()) / n).sqrt()
    assert ((share - p.double()).abs() < 5 * sd).all(), (share, p)
    assert 0.2 < (count > 0).double().mean().item() < 1.0


# ---- streams and graphs -----------------------------------------------------------------------
def test_other_stream_and_graph(ops):
    """The calls follow torch's current stream and may be captured; a replay reads the inputs of its time."""
    import torch
    x, qw, sc, z = _linear_inputs(4, 512, 96, 64, True, "bf16", seed=30)
    c = _tree_case([90, 5], [4, 2], 4, 2, 64, 16, "bf16", seed=31)
    args = (c["kc"], c["vc"], _dev(c["table"]), _dev(np.array(c["ctx"], np.int32)),
            _dev(c["starts"].astype(np.int32)), c["bits"])
    want = (ops.base_linear(x, qw, sc, z), *ops.tree_attention(c["q"], *args))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = (ops.base_linear(x, qw, sc, z), *ops.tree_attention(c["q"], *args))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    q, x2 = torch.zeros_like(c["q"]), torch.zeros_like(x)
    with torch.cuda.graph(graph):
        got = (ops.base_linear(x2, qw, sc, z), *ops.tree_attention(q, *args))
    q.copy_(c["q"])
    x2.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# ---- refusals of the tensor form ------------------------------------------------------------------
def test_tensor_form_refusals(ops):
    import torch
    x, qw, sc, z = _linear_inputs(3, 128, 20, 32, True, "bf16")
    bad = [
        lambda: ops.base_linear(x.float(), qw, sc, z), lambda: ops.base_linear(x, qw[:, :32], sc, z),
        lambda: ops.base_linear(x, qw, sc, z[:, :2]), lambda: ops.base_linear(x.t(), qw, sc, z),
        lambda: ops.base_linear(x, qw, sc.t().contiguous().t(), z), lambda: ops.base_linear(x, qw.to(torch.int8), sc),
        lambda: ops.base_linear(x, qw, sc, out=x), lambda: ops.base_linear(x, qw.cpu(), sc),
        lambda: ops.base_linear(x[0], qw, sc),
    ]
    q, k, v, pos, kc, vc, slots = _rope_inputs(4, 4, 2, 64, 64, "bf16")
    table = ops.rope_table(500, 64)
    app = ops.rope_append
    bad += [
        lambda: ops.rope(q, pos.long(), table), lambda: ops.rope(q, pos[:3], table),
        lambda: ops.rope(q, pos, table.half()), lambda: ops.rope(q[0], pos, table),
        lambda: app(q, k[:3], v, pos, table, kc, vc, slots), lambda: app(q, k, v.float(), pos, table, kc, vc, slots),
        lambda: app(q, k, v, pos, table, kc, vc, slots.int()), lambda: app(q, k, v, pos, table, kc[:, :, :1], vc, slots),
        lambda: app(q, k, v, pos, table, kc, vc.permute(1, 0, 2, 3).contiguous().permute(1, 0, 2, 3), slots),
        lambda: app(q, k, v, pos, table, kc, vc, slots, out=q.float()),
    ]
    c = _tree_case([5], [3], 4, 2, 64, 16, "bf16")
    page, ctx, st = _dev(c["table"]), _dev(np.array([5], np.int32)), _dev(c["starts"].astype(np.int32))
    att = ops.tree_attention
    bad += [
        lambda: att(c["q"], c["kc"], c["vc"], page.long(), ctx, st), lambda: att(c["q"], c["kc"], c["vc"], page, ctx, ctx),
        lambda: att(c["q"], c["kc"], c["vc"], page, ctx, st, c["bits"].int()),
        lambda: att(c["q"], c["kc"], c["vc"], page, ctx, st, c["bits"][:2]),
        lambda: att(c["q"][:, :, :56], c["kc"], c["vc"], page, ctx, st), lambda: att(c["q"], c["kc"].float(), c["vc"], page, ctx, st),
    ]
    w = _verify_case(3, 3, 2, 50, "f32", True)
    args = [w["target"], w["draft"], _dev(w["tokens"]), _dev(w["parents"]), _dev(w["starts"]), _dev(w["u"]), _dev(w["noise"])]

    def changed(i, value):
        a = list(args)
        a[i] = value
        return lambda: ops.verify_drafts(*a, 3)
    bad += [changed(0, args[0].half()), changed(1, args[1][:, :40]), changed(2, args[2].long()), changed(3, args[3][:1]),
            changed(5, args[5].double()), changed(6, args[6][:1])]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    with pytest.raises(Exception) as e:      # the library's own refusal, with its message
        ops.tree_attention(c["q"][:, :3], c["kc"], c["vc"], page, ctx, st)
    assert "n_kv_heads" in str(e.value)
