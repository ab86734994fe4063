"""A decoding step's operators on the GPU against plain 64-bit forms.

Tolerances, per element: as in test_gpu_step.py (rounding at most half a unit in the last place, doubled; fp32 sums
within 2^-22 of the sum of their terms' magnitudes), and for the norm, whose factor is off by the sum's error, a division
and the reciprocal root's two units, 2^-21 of the turned pair's magnitudes.
"""
import numpy as np
import pytest

from tests import decode_reference as ref
from tests.test_gpu_step import ROUND, _close, _dev, _dt, _np, _rope_inputs, ops  # noqa: F401

pytestmark = pytest.mark.gpu


# ---- norms and rotary positions -----------------------------------------------------------
def _weights(kind, heads, kv, dim, dtype, seed=5):
    r = np.random.default_rng(seed)
    if kind == "none":
        return None, None
    q, k = ((heads, dim), (kv, dim)) if kind == "each" else ((dim,), (dim,))
    return _dev(1 + r.standard_normal(q) / 2, _dt(dtype)), _dev(1 + r.standard_normal(k) / 2, _dt(dtype))


def _check_norm(got, x, weight, cos, sin, interleaved, eps, dtype):
    want, mass = ref.norm_rope(_np(x), None if weight is None else _np(weight), cos, sin, interleaved, eps)
    _close(_np(got), want, ROUND[dtype] * np.abs(want) + 2.0 ** -21 * mass)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,heads,kv,dim,rot,page,kind", [
    (1, 1, 1, 2, 2, 1, "one"), (1, 32, 8, 128, 128, 64, "one"), (5, 4, 2, 64, 32, 16, "each"), (33, 7, 1, 80, 64, 16, "none"),
    (70, 6, 3, 96, 96, 8, "each"), (9, 5, 5, 50, 22, 3, "one"), (200, 28, 4, 128, 64, 32, "one"), (3, 2, 1, 36, 20, 16, "each"),
    (1000, 8, 2, 128, 128, 64, "each"), (17, 3, 3, 72, 8, 16, "one"), (12, 1, 1, 7, 6, 4, "one"), (6, 2, 2, 256, 256, 16, "one"),
    (400, 30, 2, 512, 64, 16, "each"), (2, 3, 1, 1024, 512, 16, "one"), (300, 40, 10, 24, 16, 64, "one"),
    (2000, 5, 1, 16, 16, 16, "each"),
])
def test_norm_rope_append(ops, tokens, heads, kv, dim, rot, page, kind, interleaved, dtype):  # noqa: F811
    import torch
    q, k, v, pos, kc, vc, slots = _rope_inputs(tokens, heads, kv, dim, rot, dtype, page=page)
    size = torch.exp(torch.linspace(-3, 3, tokens, device="cuda"))[:, None, None]        # rows of different norms
    q, k = (q * size).to(q.dtype), (k * size).to(k.dtype)
    qw, kw = _weights(kind, heads, kv, dim, dtype)
    table = ops.rope_table(500, rot)
    want_k, want_v = _np(kc), _np(vc)
    out = ops.norm_rope_append(q, k, v, qw, kw, pos, table, kc, vc, slots, eps=1e-5, interleaved=interleaved)
    tab, p, s = _np(table), pos.cpu().numpy(), slots.cpu().numpy()
    cos, sin = tab[p, :rot // 2], tab[p, rot // 2:]
    _check_norm(out, q, qw, cos, sin, interleaved, 1e-5, dtype)
    _check_norm(kc[s // page, s % page], k, kw, cos, sin, interleaved, 1e-5, dtype)
    want_v[s // page, s % page] = _np(v)
    _close(_np(vc), want_v, 0.0)
    rest = np.ones(want_k.shape[:2], bool)
    rest[s // page, s % page] = False
    assert (_np(kc)[rest] == want_k[rest]).all()
    alone = ops.norm_rope(q, qw, pos, table, eps=1e-5, interleaved=interleaved)
    assert torch.equal(alone, out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,rot,tokens", [(128, 128, 9), (80, 64, 700), (30, 10, 9), (128, 64, 3000)])
def test_norm_rope_layouts(ops, dim, rot, tokens, dtype):  # noqa: F811
    """In place; inside wider rows from an odd element; weights from an odd element and in wider rows: the same bits
    where the layout takes the same kernel, else the same values."""
    import torch
    heads = 6
    q, _, _, pos, _, _, _ = _rope_inputs(tokens, heads, 1, dim, rot, dtype, seed=2)
    q = q.contiguous()
    w = _weights("each", heads, 1, dim, dtype)[0]
    table = ops.rope_table(500, rot)
    want = ops.norm_rope(q, w, pos, table)
    same = q.clone()
    assert ops.norm_rope(same, w, pos, table, out=same).data_ptr() == same.data_ptr() and torch.equal(same, want)
    wide = torch.full((tokens, heads, dim + 9), float("nan"), dtype=q.dtype, device="cuda")
    wide[:, :, 1:dim + 1] = q
    wide_w = torch.full((heads, dim + 5), float("nan"), dtype=q.dtype, device="cuda")
    wide_w[:, 3:dim + 3] = w
    out = torch.full_like(wide, 7.0)
    ops.norm_rope(wide[:, :, 1:dim + 1], wide_w[:, 3:dim + 3], pos, table, out=out[:, :, 1:dim + 1])
    cos, sin = _np(table)[pos.cpu().numpy(), :rot // 2], _np(table)[pos.cpu().numpy(), rot // 2:]
    _check_norm(out[:, :, 1:dim + 1], q, w, cos, sin, False, 1e-6, dtype)
    assert (out[:, :, 0] == 7.0).all() and (out[:, :, dim + 1:] == 7.0).all()


@pytest.mark.parametrize("dtype,interleaved,tokens,heads,kv,dim,rot,kind", [
    ("bf16", False, 2500, 32, 8, 128, 128, "one"), ("bf16", True, 2301, 42, 1, 80, 64, "each"),
    ("f32", False, 3000, 28, 4, 80, 32, "one"), ("f32", True, 1100, 64, 16, 64, 64, "none"),
    ("bf16", False, 1200, 64, 8, 256, 128, "each"), ("bf16", True, 9000, 9, 1, 512, 512, "one"),
])
def test_norm_rope_many_rows(ops, dtype, interleaved, tokens, heads, kv, dim, rot, kind):  # noqa: F811
    """Batches whose blocks go over several tokens: rows with and without a vector for every lane, tokens in several
    chunks of rows, positions and slots out of range among the others; in place, and alone as with the append."""
    import torch
    q, k, v, pos, kc, vc, slots = _rope_inputs(tokens, heads, kv, dim, rot, dtype, page=16, seed=7)
    qw, kw = _weights(kind, heads, kv, dim, dtype)
    table = ops.rope_table(500, rot)
    bad = torch.arange(tokens, device="cuda") % 13 == 5
    lost = torch.arange(tokens, device="cuda") % 17 == 3
    pos = torch.where(bad, torch.where(torch.arange(tokens, device="cuda") % 2 == 0, -1, 500).int(), pos)
    slots = torch.where(lost, kc.shape[0] * 16 + slots, slots)
    out = torch.full((tokens, heads, dim), 5.0, dtype=q.dtype, device="cuda")
    ops.norm_rope_append(q, k, v, qw, kw, pos, table, kc, vc, slots, interleaved=interleaved, out=out)
    good, there = (~bad).cpu().numpy(), (~bad & ~lost).cpu().numpy()
    tab, p, s = _np(table), pos.cpu().numpy()[good], slots.cpu().numpy()[there]
    _check_norm(out[~bad], q[~bad], qw, tab[p, :rot // 2], tab[p, rot // 2:], interleaved, 1e-6, dtype)
    assert (out[bad] == 5.0).all()
    p = pos.cpu().numpy()[there]
    _check_norm(kc[s // 16, s % 16], k[~bad & ~lost], kw, tab[p, :rot // 2], tab[p, rot // 2:], interleaved, 1e-6, dtype)
    assert torch.equal(vc[s // 16, s % 16], v[~bad & ~lost])
    rest = np.ones(kc.shape[:2], bool)
    rest[s // 16, s % 16] = False
    assert (kc[_dev(rest)] == 7.0).all() and (vc[_dev(rest)] == 9.0).all()
    same = q.contiguous()
    ops.norm_rope(same, qw, pos, table, interleaved=interleaved, out=same)
    assert torch.equal(same[~bad], out[~bad]) and torch.equal(same[bad], q[bad])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [128, 50])
def test_norm_rope_values(ops, dim, dtype):  # noqa: F811
    """A head of zeros stays zero (with eps), one of tiny values is divided by eps's root, and a NaN or infinity stays in
    its head."""
    import torch
    x = torch.ones((5, 3, dim), dtype=_dt(dtype), device="cuda")
    x[0, 1] = 0.0
    x[1, 2] = 2.0 ** -40
    x[2, 0, 3], x[3, 1, 4] = float("nan"), float("inf")
    pos = torch.zeros(5, dtype=torch.int32, device="cuda")          # position 0: nothing is turned
    table = ops.rope_table(4, dim)
    y = ops.norm_rope(x, None, pos, table, eps=2.0 ** -60)
    assert (y[0, 1] == 0).all() and (y[1, 2].float() - 2.0 ** -40 / (2.0 ** -80 + 2.0 ** -60) ** 0.5).abs().max() < 2.0 ** -19
    pair = [4, 4 + dim // 2]                                        # inf / inf, and its partner by NaN * sin 0
    rest = [i for i in range(dim) if i not in pair]
    assert torch.isnan(y[2, 0]).all() and torch.isnan(y[3, 1, pair]).all() and not y[3, 1, rest].any()
    keep = torch.ones((5, 3), dtype=torch.bool)
    keep[0, 1] = keep[1, 2] = keep[2, 0] = keep[3, 1] = False
    assert (y[keep.cuda()].float() - 1).abs().max() <= 2.0 ** -21


def test_norm_rope_entries_out_of_range(ops):  # noqa: F811
    """Positions outside the table write nothing; slots outside the cache write no cache row."""
    import torch
    for dtype, dim, tokens in [("bf16", 64, 8), ("f32", 22, 8), ("bf16", 128, 3000)]:
        q, k, v, pos, kc, vc, slots = _rope_inputs(tokens, 6, 1, dim, 8, dtype)
        qw, kw = _weights("one", 6, 1, dim, dtype)
        table = ops.rope_table(500, 8)
        good_k, good_v = kc.clone(), vc.clone()
        good = ops.norm_rope_append(q, k, v, qw, kw, pos, table, good_k, good_v, slots)
        pos2, slots2 = pos.clone(), slots.clone()
        pos2[1], pos2[4] = -1, 500
        slots2[2], slots2[6] = -1, kc.shape[0] * kc.shape[1]
        out = torch.full_like(good, 5.0)
        ops.norm_rope_append(q, k, v, qw, kw, pos2, table, kc, vc, slots2, out=out)
        want = good.clone()
        want[[1, 4]] = 5.0
        assert torch.equal(out, want)
        for lost in (1, 2, 4, 6):
            s = int(slots[lost])
            good_k[s // 16, s % 16], good_v[s // 16, s % 16] = 7.0, 9.0
        assert torch.equal(kc, good_k) and torch.equal(vc, good_v)


def test_norm_rope_offsets_past_32_bits(ops):  # noqa: F811
    """A cache row more than 2^31 elements from the cache's start."""
    import torch
    page, kv, dim = 64, 8, 128
    pages = (1 << 31) // (page * kv * dim) + 3
    kc = torch.empty((pages, page, kv, dim), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    q, k, v, pos, _, _, _ = _rope_inputs(2, 8, kv, dim, dim, "bf16")
    slots = torch.tensor([pages * page - 1, 5], dtype=torch.int64, device="cuda")
    table = ops.rope_table(500, dim)
    ops.norm_rope_append(q, k, v, None, None, pos, table, kc, vc, slots)
    want = ops.norm_rope(k, None, pos, table)
    assert torch.equal(kc[-1, -1], want[0]) and torch.equal(vc[-1, -1], v[0]) and torch.equal(kc[0, 5], want[1])


# ---- attention over shared prefixes ----------------------------------------------------------
def _prefix_case(prefix, members, ctx, nodes, heads, kv, dim, page, dtype, seed=0, spread=1.0, first=0, spare_rows=0):
    """Group g has members[g] requests and prefix[g] shared keys; the first `first` requests and those past the last group
    have none. Every cache row that no query sees is NaN."""
    r = np.random.default_rng(seed)
    ctx, nodes, prefix = list(ctx), list(nodes), list(prefix)
    per = max(1, max(-(-(c + n) // page) for c, n in zip(ctx, nodes)))
    shared = max(1, max([-(-p // page) for p in prefix] + [0]))
    pages = per * len(ctx) + shared * len(prefix) + 2
    ids = r.permutation(pages).astype(np.int32)
    table = ids[:per * len(ctx)].reshape(len(ctx), per)
    ptable = ids[per * len(ctx):per * len(ctx) + shared * len(prefix)].reshape(len(prefix), shared)
    kc = np.full((pages, page, kv, dim), np.nan)
    vc = np.full_like(kc, np.nan)
    starts = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int64)
    total = int(starts[-1]) + spare_rows
    mask = np.zeros((max(total, 1), 64), bool)
    for t, n in [(ptable[g], prefix[g]) for g in range(len(prefix))] + [(table[b], ctx[b] + nodes[b]) for b in range(len(ctx))]:
        for p in range(n):
            kc[t[p // page], p % page] = r.standard_normal((kv, dim))
            vc[t[p // page], p % page] = r.standard_normal((kv, dim))
    for b in range(len(ctx)):
        for i in range(nodes[b]):
            if i > 0:
                mask[starts[b] + i] = mask[starts[b] + r.integers(max(0, i - 4), i)]
            mask[starts[b] + i, i] = True
    bits = np.packbits(mask, axis=1, bitorder="little").view(np.int64).reshape(mask.shape[0], 1)[:total]
    q = r.standard_normal((total, heads, dim)) * spread
    return dict(q=_dev(q, _dt(dtype)), kc=_dev(kc, _dt(dtype)), vc=_dev(vc, _dt(dtype)), table=table, ptable=ptable,
                prefix=prefix, groups=np.concatenate([[first], first + np.cumsum(members)]).astype(np.int64), ctx=ctx,
                starts=starts, mask=mask, bits=_dev(bits), dtype=dtype)


def _run_prefix(ops, c, mask=True, out=None, scale=None):  # noqa: F811
    i32 = lambda a: _dev(np.asarray(a, np.int32))  # noqa: E731
    return ops.prefix_attention(c["q"], c["kc"], c["vc"], i32(c["ptable"]), i32(c["prefix"]), i32(c["groups"]),
                                i32(c["table"]), i32(c["ctx"]), i32(c["starts"]), c["bits"] if mask else None, scale=scale,
                                out=out)


def _check_prefix(c, out, lse, mask=True, scale=None):
    """Tolerances as in test_gpu_step.py's _check_tree."""
    dim = c["q"].shape[2]
    scale = dim ** -0.5 if scale is None else scale
    sees = (lambda t, i, j: j < 64 and c["mask"][t, j]) if mask else (lambda t, i, j: j <= i)
    want, want_lse, mass, reach = ref.prefix_attention(_np(c["q"]), _np(c["kc"]), _np(c["vc"]), c["ptable"], c["prefix"],
                                                       c["groups"], c["table"], c["ctx"], c["starts"], sees, scale)
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


PREFIXES = [
    # prefix, members of each group, contexts, nodes, heads, kv heads, head dim, page
    ([1], [1], [0], [1], 1, 1, 8, 16), ([5], [3], [0, 1, 7], [1, 1, 1], 4, 2, 64, 1), ([0], [2], [3, 9], [1, 2], 4, 4, 40, 16),
    ([], [], [5, 70], [1, 3], 8, 2, 64, 16), ([777], [3], [40, 0, 33], [1, 1, 1], 32, 8, 128, 64),
    ([64, 65], [2, 3], [64, 1, 0, 63, 130], [1] * 5, 8, 8, 64, 64), ([100, 0, 300], [4, 1, 5], [17] * 10, [1, 3, 2, 7, 1] * 2, 14, 2, 96, 16),
    # groups on tiles of 128 rows, requests on 16 or 32; whole nodes in a tile (groups of heads of 7 and 3)
    ([500], [40], [20] * 40, [1] * 40, 8, 2, 128, 16), ([130, 257, 1], [20, 15, 30], list(range(65)), [1] * 65, 14, 2, 72, 32),
    ([3000], [9], [200] * 9, [5] * 9, 12, 4, 96, 16), ([90], [300], [3] * 300, [1] * 300, 4, 1, 64, 16),
    # both on 128
    ([300, 40], [2, 2], [100, 0, 65, 7], [40, 64, 17, 33], 8, 2, 128, 16), ([1000], [3], [10, 500, 64], [64, 1, 30], 16, 1, 64, 24),
    # pages that no box of eight rows fits; long prefixes over many blocks; more groups than requests
    ([200], [30], [9] * 30, [2] * 30, 8, 2, 64, 12), ([6000], [2], [30, 3], [1, 2], 16, 1, 128, 64), ([2000], [20], [64] * 20, [3] * 20, 16, 1, 128, 64),
    ([9, 30, 70, 3], [0, 1, 0, 1], [20, 30], [2, 1], 4, 2, 128, 16),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", PREFIXES, ids=lambda c: f"{len(c[2])}of{c[0]}")
def test_prefix_attention(ops, case, dtype):  # noqa: F811
    c = _prefix_case(*case, dtype)
    _check_prefix(c, *_run_prefix(ops, c))


def _widen(c, group_bytes, request_bytes):
    """Tables as wide as contexts of so many bytes, read 16 rows at a time, would need: entries with more than 16 rows then
    go to the tiles of 128 (80 MB)."""
    (tokens, heads, dim), (_, page, kv, _) = c["q"].shape, c["kc"].shape

    def wide(table, n, size):
        each = max(1, -(-tokens * heads // kv // max(n, 1) // 16)) * max(n, 1) * kv * page * dim * 4
        return np.pad(table, ((0, 0), (0, int(size // each))), constant_values=-1)
    return dict(c, ptable=wide(c["ptable"], len(c["prefix"]), group_bytes), table=wide(c["table"], len(c["ctx"]), request_bytes))


@pytest.mark.parametrize("widths", [(2e8, 0), (2e8, 2e8), (0, 2e8), (2e8, 7e8)])
@pytest.mark.parametrize("case", PREFIXES[3:], ids=lambda c: f"{len(c[2])}of{c[0]}")
def test_prefix_attention_wide_tables(ops, case, widths):  # noqa: F811
    c = _widen(_prefix_case(*case, "bf16", seed=9), *widths)
    _check_prefix(c, *_run_prefix(ops, c))


@pytest.mark.parametrize("widths", [(2e8, 0), (2e8, 2e8), (0, 2e8)])
@pytest.mark.parametrize("case", PREFIXES[3:], ids=lambda c: f"{len(c[2])}of{c[0]}")
def test_prefix_attention_wide_tables_fp32(ops, case, widths):  # noqa: F811
    """Above 30 MB entries with more than 16 rows go to tiles of 64, the others to 16 in a launch of their own."""
    c = _widen(_prefix_case(*case, "f32", seed=11), *widths)
    _check_prefix(c, *_run_prefix(ops, c))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nodes,request_bytes", [(1, 0), (5, 2e8)])
def test_prefix_attention_many_entries(ops, nodes, request_bytes, dtype):  # noqa: F811
    """More entries than threads of any block that finds its share among them; some have no rows."""
    import torch
    n = 290
    sizes = [0 if i % 29 == 7 else nodes + i % 2 for i in range(n)]
    c = _widen(_prefix_case([70, 0, 33] * 20, [4, 3, 5] * 20, [(7 * i) % 90 for i in range(n)], sizes, 4, 1, 64, 16, dtype,
                            seed=12, first=20), 2e8, request_bytes)
    out, lse = _run_prefix(ops, c)
    _check_prefix(c, out, lse)
    again, _ = _run_prefix(ops, c)
    assert torch.equal(out, again)


@pytest.mark.parametrize("members", [9, 30])
@pytest.mark.parametrize("nodes", [1, 20])
@pytest.mark.parametrize("widths", [(2e8, 0), (2e8, 2e8), (2e8, 7e8)])
def test_prefix_attention_wide_tables_edges(ops, widths, nodes, members):  # noqa: F811
    """Entries without keys or rows, page ids and lengths out of range, values that are not finite, on the same routes."""
    import torch
    n = members + 7
    c = _widen(_prefix_case([150, 0, 700, 90], [members, 2, 1, 2], [20, 0, 64] * (n // 3) + [1] * (n % 3),
                            [nodes, 1, 0] * (n // 3) + [1] * (n % 3), 8, 1, 64, 16, "bf16", seed=10, first=1, spare_rows=3), *widths)
    c["ptable"][0, 1], c["ptable"][2, 4], c["ptable"][3, 2] = -1, c["kc"].shape[0], 1 << 30
    c["mask"][0] = False
    c["bits"][0] = 0
    want = _run_prefix(ops, c)
    _check_prefix(c, *want)
    c["ctx"][0] = -3
    _check_prefix(c, *_run_prefix(ops, c))
    c["ctx"][0] = 20
    d = dict(c, vc=c["vc"].clone())
    d["vc"][int(c["ptable"][0, 0]), 3, 0, 5] = float("inf")
    out, lse = _run_prefix(ops, d)
    rows = slice(int(c["starts"][1]), int(c["starts"][1 + members]))
    assert (out[rows, :, 5] == float("inf")).all() and torch.equal(lse[:-3], want[1][:-3])
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[rows, :, 5] = False
    keep[-3:] = False
    assert ((out - want[0]).abs()[keep] <= 2.0 ** -6 * (1 + want[0].abs()[keep])).all()     # both near the same values


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", [PREFIXES[6], PREFIXES[8], PREFIXES[11]], ids=lambda c: f"{len(c[2])}of{c[0]}")
def test_prefix_attention_chain(ops, case, dtype):  # noqa: F811
    """Without a mask node i sees the nodes 0..i, and all of the prefix."""
    c = _prefix_case(*case, dtype, seed=1)
    _check_prefix(c, *_run_prefix(ops, c, mask=False), mask=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("members", [[2, 3], [15, 14]])
def test_prefix_attention_requests_of_no_group(ops, members, dtype):  # noqa: F811
    """Requests before the first and past the last group have their own keys alone; rows of no request stay."""
    import torch
    n = sum(members) + 5
    c = _prefix_case([70, 130], members, [33, 0] * (n // 2) + [9] * (n % 2), [1, 2, 3] * (n // 3) + [1] * (n % 3), 8, 2, 64, 16,
                     dtype, seed=2, first=3, spare_rows=4)
    out = torch.full(c["q"].shape, 3.0, dtype=c["q"].dtype, device="cuda")
    out, lse = _run_prefix(ops, c, out=out)
    _check_prefix(c, out, lse)
    assert (out[-4:] == 3.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("members", [3, 40])
def test_prefix_attention_rows_without_keys(ops, members, dtype):  # noqa: F811
    """No prefix, no context and a mask that leaves nothing: 0 and -inf; with a prefix alone, the prefix's result."""
    for prefix in (0, 150):
        c = _prefix_case([prefix], [members], [0] * members, [1] * members, 8, 2, 64, 16, dtype, seed=3)
        c["mask"][1] = c["mask"][members - 1] = False
        c["bits"][1] = c["bits"][members - 1] = 0
        out, lse = _run_prefix(ops, c)
        _check_prefix(c, out, lse)
        assert (lse[1] == float("-inf")).all() == (prefix == 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("members", [3, 40])
def test_prefix_attention_bad_entries(ops, members, dtype):  # noqa: F811
    """Page ids out of range, keys past a prefix table's row and lengths below zero are not seen; group starts outside
    the requests are clamped, and ones that fall lead nowhere."""
    import torch
    c = _prefix_case([150, 90], [members, 2], [20] * (members + 2), [1] * (members + 2), 8, 2, 64, 16, dtype, seed=4)
    c["ptable"] = c["ptable"].copy()
    c["ptable"][0, 1], c["ptable"][0, 4], c["ptable"][1, 2] = -1, c["kc"].shape[0], 1 << 30
    c["ptable"] = c["ptable"][:, :8]      # group 0: keys 128.. are past its row
    _check_prefix(c, *_run_prefix(ops, c))
    c["prefix"][1] = -7
    _check_prefix(c, *_run_prefix(ops, c))
    want = _run_prefix(ops, c)
    c["groups"][2] = 1 << 30
    got = _run_prefix(ops, c)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c["groups"][:] = [4, 1, 3]
    out = torch.full(c["q"].shape, 3.0, dtype=c["q"].dtype, device="cuda")
    assert _run_prefix(ops, c, out=out)[0].shape == c["q"].shape
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("members", [4, 50])
def test_prefix_attention_layouts(ops, members, dtype):  # noqa: F811
    """Heads outside the tokens, places inside the heads, wider rows, tables inside wider ones."""
    import torch
    c = _prefix_case([100, 33], [members, 2], [40] * (members + 2), [2] * (members + 2), 8, 2, 64, 16, dtype, seed=5)
    want = _run_prefix(ops, c)
    n = c["q"].shape[0]
    q = torch.zeros((8, n, 72), dtype=c["q"].dtype, device="cuda")
    q[:, :, :64] = c["q"].transpose(0, 1)
    kc, vc = (t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for t in (c["kc"], c["vc"]))
    out = torch.full((n, 8, 80), 7.0, dtype=q.dtype, device="cuda")
    d = dict(c, q=q[:, :, :64].transpose(0, 1), kc=kc, vc=vc)
    i32 = lambda a: _dev(np.asarray(a, np.int32))  # noqa: E731
    wide = i32(np.pad(c["ptable"], ((0, 0), (2, 3)), constant_values=-1))[:, 2:-3]
    got, lse = ops.prefix_attention(d["q"], kc, vc, wide, i32(c["prefix"]), i32(c["groups"]), i32(c["table"]), i32(c["ctx"]),
                                    i32(c["starts"]), c["bits"], out=out[:, :, :64])
    _check_prefix(c, got, lse)
    assert (out[:, :, 64:] == 7.0).all() and torch.allclose(lse, want[1], rtol=0, atol=2.0 ** -15)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("spread", [40.0, 1e-3])
@pytest.mark.parametrize("members", [3, 40])
@pytest.mark.parametrize("scale", [0.5, -0.3, 0.0])
def test_prefix_attention_score_range(ops, scale, members, spread, dtype):  # noqa: F811
    c = _prefix_case([300], [members], [64, 0] * (members // 2) + [5] * (members % 2), [1] * members, 8, 2, 128, 16, dtype,
                     seed=6, spread=spread)
    _check_prefix(c, *_run_prefix(ops, c, scale=scale), scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("members", [2, 7, 40])
@pytest.mark.parametrize("at", [10, 68])
def test_prefix_attention_values_not_finite(ops, at, members, dtype):  # noqa: F811
    """An infinity in a prefix value reaches every row of its group and head and no other; a NaN in a prefix key makes
    those rows NaN; a query row that is not finite is its own alone."""
    import torch
    c = _prefix_case([70, 70], [members, members], [30] * (2 * members), [1] * (2 * members), 8, 2, 128, 16, dtype, seed=7)
    want = _run_prefix(ops, c)
    _check_prefix(c, *want)
    where = int(c["ptable"][0, at // 16]), at % 16
    tol = 2.0 ** -6 if dtype == "bf16" else 2.0 ** -18      # both within their tolerance of the same values
    d = dict(c, vc=c["vc"].clone())
    d["vc"][where[0], where[1], 0, 5] = float("-inf")
    out, lse = _run_prefix(ops, d)
    assert (out[:members, :4, 5] == float("-inf")).all() and torch.equal(lse, want[1])
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[:members, :4, 5] = False
    assert ((out - want[0]).abs()[keep] <= tol * (1 + want[0].abs()[keep])).all()
    d = dict(c, kc=c["kc"].clone(), q=c["q"].clone())
    d["kc"][where[0], where[1], 1, 9] = float("nan")
    d["q"][2 * members - 1, 1, 5] = float("nan")
    out, lse = _run_prefix(ops, d)
    assert torch.isnan(out[:members, 4:]).all() and torch.isnan(lse[:members, 4:]).all()
    assert torch.isnan(out[-1, 1]).all() and torch.isnan(lse[-1, 1])
    keep = torch.ones_like(lse, dtype=torch.bool)
    keep[:members, 4:] = keep[-1, 1] = False
    assert ((out - want[0]).abs()[keep] <= tol * (1 + want[0].abs()[keep])).all()


def test_prefix_attention_offsets_past_32_bits(ops):  # noqa: F811
    """Pages more than 2^31 elements into the cache."""
    import torch
    page, kv, dim = 64, 8, 128
    far = (1 << 31) // (page * kv * dim) + 1
    kc = torch.empty((far + 50, page, kv, dim), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    for members in (2, 40):
        c = _prefix_case([100], [members], [20] * members, [1] * members, 16, kv, dim, page, "bf16", seed=8)
        kc[far:far + c["kc"].shape[0]], vc[far:far + c["kc"].shape[0]] = c["kc"], c["vc"]
        want = _run_prefix(ops, c)
        got = _run_prefix(ops, dict(c, kc=kc, vc=vc, table=c["table"] + far, ptable=c["ptable"] + far))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefix_attention_as_one_context(ops, dtype):  # noqa: F811
    """What tree_attention gives with the prefix's pages in front of each request's own."""
    import torch
    for members, nodes in ((3, 2), (30, 1), (4, 30)):
        c = _prefix_case([128], [members], [40] * members, [nodes] * members, 8, 2, 64, 16, dtype, seed=9)
        got = _run_prefix(ops, c)
        whole = np.concatenate([np.repeat(c["ptable"], members, 0), c["table"]], 1)
        want = ops.tree_attention(c["q"], c["kc"], c["vc"], _dev(whole), _dev(np.array(c["ctx"], np.int32) + 128),
                                  _dev(c["starts"].astype(np.int32)), c["bits"])
        tol = 2.0 ** -6 if dtype == "bf16" else 2.0 ** -18
        assert ((got[0] - want[0]).abs() <= tol * (1 + want[0].abs())).all()
        assert torch.allclose(got[1], want[1], rtol=0, atol=2.0 ** -15)


def test_prefix_attention_repeats_bit_for_bit(ops):  # noqa: F811
    import torch
    from rank_adapter_apply_gb300 import binding as B
    for members, nodes in ((5, 1), (50, 2), (5, 40)):
        c = _prefix_case([3000], [members], [77] * members, [nodes] * members, 16, 4, 128, 16, "bf16", seed=10)
        first = _run_prefix(ops, c)
        for _ in range(4):
            again = _run_prefix(ops, c)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    assert B.lora_step_wait_timeouts() == 0


# ---- the draw of the next token ----------------------------------------------------------------
def _sample_case(rows, vocab, dtype, kinds, seed=0, sharp=2.0):
    r = np.random.default_rng(seed)
    logits = r.standard_normal((rows, vocab)) * sharp * r.uniform(0.5, 2.0, (rows, 1))
    logits[:, r.integers(0, vocab, 3)] += 6.0
    c = dict(logits=_dev(logits, _dt(dtype)), noise=_dev(np.maximum(r.exponential(size=(rows, vocab)), 1e-30).astype(np.float32)))
    pick = np.array([kinds[i % len(kinds)] for i in range(rows)])
    on = lambda names: np.isin(pick, names)  # noqa: E731
    c["temperature"] = np.where(on(["greedy"]), 0.0, r.uniform(0.5, 1.5, rows)).astype(np.float32)
    c["top_k"] = np.where(on(["k", "all"]), r.choice([1, 2, 7, 40, 1000], rows), 0).astype(np.int32)
    c["top_p"] = np.where(on(["p", "all"]), r.uniform(0.3, 0.99, rows), 1.0).astype(np.float32)
    c["min_p"] = np.where(on(["m", "all"]), r.choice([0.01, 0.2, 1.0], rows), 0.0).astype(np.float32)
    return c


def _run_sample(ops, c):  # noqa: F811
    dev = lambda a: None if a is None else _dev(a)  # noqa: E731
    return ops.sample_tokens(c["logits"], c["noise"], dev(c["temperature"]), dev(c["top_k"]), dev(c["top_p"]), dev(c["min_p"]))


def _check_sample(c, got, most_unsure=0.02):
    tokens, logprobs, tol, margin = ref.sample(_np(c["logits"]), _np(c["noise"]), c["temperature"], c["top_k"], c["top_p"],
                                               c["min_p"])
    sure = margin > 2.0 ** -17             # fp32 sums and exponentials of arguments up to 2^6 stay below this
    assert (~sure).sum() <= 1 + most_unsure * len(sure)
    assert (got[0].cpu().numpy()[sure] == tokens[sure]).all()
    _close(_np(got[1])[sure], logprobs[sure], (2.0 ** -24 * tol)[sure])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kinds", [["none"], ["k"], ["p"], ["m"], ["none", "all", "greedy", "k", "p", "m"]], ids="-".join)
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 2), (9, 7), (5, 63), (40, 1000), (2, 4097), (1, 32000), (7, 32001),
                                        (333, 517), (12, 100003), (4, 131072), (3, 300007)])
def test_sample_tokens(ops, rows, vocab, kinds, dtype):  # noqa: F811
    c = _sample_case(rows, vocab, dtype, kinds)
    _check_sample(c, _run_sample(ops, c))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab,sharp", [(30, 30000, 0.01), (30, 1000, 20.0), (300, 20011, 0.5)])
def test_sample_tokens_flat_and_sharp(ops, rows, vocab, sharp, dtype):  # noqa: F811
    """Nearly equal logits, where a race over all tokens is mostly lost, and ones far apart."""
    c = _sample_case(rows, vocab, dtype, ["k", "p", "all", "none"], seed=1, sharp=sharp)
    _check_sample(c, _run_sample(ops, c))


def test_sample_tokens_without_filters(ops):  # noqa: F811
    """Filters that are not given are those that keep everything; a temperature that is not given is 1."""
    import torch
    c = _sample_case(20, 5000, "f32", ["none"], seed=2)
    c["temperature"][:] = 1.0
    want = _run_sample(ops, c)
    got = ops.sample_tokens(c["logits"], c["noise"])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [1000, 40000, 200000])
def test_sample_tokens_ties_and_unkind_noise(ops, vocab, dtype):  # noqa: F811
    """Equal logits are ordered by index. The noise makes the last token of the order win every race, so that the border is
    found by bisection: the last kept one is drawn."""
    import torch
    rows = 12
    levels = torch.zeros((rows, vocab), device="cuda")
    levels[4:8, ::2] = 1.0                                    # two levels: the order is not the index's
    logits = levels.to(_dt(dtype))
    place = torch.arange(vocab, device="cuda").expand(rows, -1).clone()
    evens = (vocab + 1) // 2
    place[4:8] = torch.where(torch.arange(vocab, device="cuda") % 2 == 0, torch.arange(vocab, device="cuda") // 2,
                             evens + torch.arange(vocab, device="cuda") // 2)
    p = torch.softmax(logits.double(), 1)
    noise = (p * 4.0 ** (-place.double() / vocab)).float()    # p / noise rises along the order
    k = np.array([1, 2, 50, 0, 1, 2, 50, 0, 999, 0, 0, 0], np.int32)
    top_p = np.array([1, 1, 1, 1, 1, 1, 1, 1, 1, 0.25, 0.5, 0.7501], np.float32)
    tokens, _ = ops.sample_tokens(logits, noise, None, _dev(k), _dev(top_p))
    kept = [int(n) if n else vocab for n in k]
    for r in (9, 10, 11):
        kept[r] = int(np.ceil(float(top_p[r]) * vocab))
    for r in range(rows):
        drawn = int(place[r, tokens[r]])
        # of keys 4^(place / vocab) in fp32 many neighbours are equal: the lowest index of them wins
        low = kept[r] - 1 - vocab * 2.0 ** -21 / np.log(4.0) - 1
        assert low <= drawn <= kept[r] - 1 + (1 if r >= 9 else 0), (r, drawn, kept[r])


def test_sample_tokens_values_out_of_the_ordinary(ops):  # noqa: F811
    import torch
    inf, nan = float("inf"), float("nan")
    for vocab in (37, 5000):
        x = torch.zeros((16, vocab), device="cuda")
        x[:, 11] = 3.0
        noise = torch.ones((16, vocab), device="cuda")
        temperature, top_k = torch.ones(16, device="cuda"), torch.zeros(16, dtype=torch.int32, device="cuda")
        top_p, min_p = torch.ones(16, device="cuda"), torch.zeros(16, device="cuda")
        x[0] = -inf                                           # nothing to draw
        x[1] = nan
        x[2, 5] = nan                                         # a NaN is not drawn
        x[3, 7] = inf                                         # takes all
        x[4, 3] = x[4, 20] = inf
        noise[4, 3] = 9.0
        x[5, :30] = -inf
        noise[6] = nan                                        # no noise to go by: the first
        noise[7] = -1.0
        noise[8, 2] = 0.0                                     # at once
        temperature[9], temperature[10], temperature[11] = nan, -1.0, 1e-42
        top_p[12], top_p[13] = nan, 0.0
        min_p[14], min_p[15] = nan, 2.0
        tokens, logprobs = (t.tolist() for t in ops.sample_tokens(x, noise, temperature, top_k, top_p, min_p))
        e = np.exp(-3.0)
        total = 1 + (vocab - 1) * e
        assert tokens[0] == tokens[1] == -1 and logprobs[0] == logprobs[1] == -inf
        assert tokens[2] == 11 and abs(logprobs[2] + np.log(total - e)) < 1e-5
        assert tokens[3] == 7 and logprobs[3] == 0.0
        assert tokens[4] == 20 and abs(logprobs[4] + np.log(2.0)) < 1e-6
        assert tokens[5] == 30 and abs(logprobs[5] + np.log(vocab - 30)) < 1e-5
        assert tokens[6:8] == [11, 11] and tokens[8] == 2 and abs(logprobs[8] + 3 + np.log(total)) < 1e-5
        assert tokens[9:] == [11] * 7
        # the same p summed in other orders (rows start at different places within 16 bytes): their sum, 1 + less than vocab e^-3, is off by at most 2^-24 of itself for each of
        # its at most 32 levels (a thread's tokens, then halves), and the logarithm by as much
        assert max(logprobs[9], logprobs[10], logprobs[6]) - min(logprobs[9], logprobs[10], logprobs[6]) <= 2 * 32 * 2.0 ** -24
        assert logprobs[11] == 0.0


def test_sample_tokens_infinite_temperature_is_flat(ops):  # noqa: F811
    import torch
    x = torch.randn((3, 700), device="cuda")
    x[:, 400:] = float("-inf")
    noise = torch.rand((3, 700), device="cuda") + 0.1
    noise[:, 650] = 1e-6
    tokens, logprobs = ops.sample_tokens(x, noise, torch.full((3,), float("inf"), device="cuda"))
    assert torch.equal(tokens.long(), noise[:, :400].argmin(1)) and (logprobs + np.log(400.0)).abs().max() < 1e-5


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab", [(5, 301), (3, 40001), (400, 1003)])
@pytest.mark.parametrize("at", [(3, 1), (0, 1), (5, 2), (1, 3), (7, 0)])
def test_sample_tokens_rows_at_different_offsets(ops, at, rows, vocab, dtype):  # noqa: F811
    """Logits and noise inside wider rows of different widths, starting at different elements; NaN lies around them."""
    import torch
    c = _sample_case(rows, vocab, dtype, ["none", "all", "p", "k"], seed=3)
    want = _run_sample(ops, c)
    for i, name in enumerate(("logits", "noise")):
        wide = torch.full((rows, vocab + 11 + i), float("nan"), dtype=c[name].dtype, device="cuda")
        wide[:, at[i]:at[i] + vocab] = c[name]
        c[name] = wide[:, at[i]:at[i] + vocab]
    got = _run_sample(ops, c)
    _check_sample(c, got)
    assert (got[1] - want[1]).abs().max() < 2.0 ** -18 or not torch.equal(got[0], want[0])


@pytest.mark.parametrize("filters", [dict(), dict(top_k=3), dict(top_p=0.6), dict(min_p=0.3), dict(top_k=5, top_p=0.8)])
def test_sample_tokens_is_distributed_as_the_kept(ops, filters):  # noqa: F811
    """Frequencies of 200000 draws of one row against the kept tokens' probabilities: within five standard deviations."""
    import torch
    n, vocab = 200000, 24
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((1, vocab), generator=gen, device="cuda") * 1.5
    noise = torch.empty((n, vocab), device="cuda").exponential_(generator=gen)
    each = {k: torch.full((n,), v, dtype=torch.int32 if k == "top_k" else torch.float32, device="cuda") for k, v in filters.items()}
    tokens, _ = ops.sample_tokens(x.expand(n, -1), noise, torch.full((n,), 0.8, device="cuda"), **each)
    p = torch.softmax(x[0].double() / 0.8, 0)
    order = p.argsort(descending=True)
    kept = torch.ones(vocab, dtype=torch.bool, device="cuda")
    if "top_k" in filters:
        kept[order[filters["top_k"]:]] = False
    if "top_p" in filters:
        kept[order[(p[order].cumsum(0) - p[order]) >= filters["top_p"]]] = False
    if "min_p" in filters:
        kept &= p >= filters["min_p"] * p.max()
    q = torch.where(kept, p, 0.0)
    q = q / q.sum()
    freq = torch.bincount(tokens.long(), minlength=vocab).double() / n
    assert ((freq - q).abs() <= 5 * (q * (1 - q) / n).sqrt()).all()


def test_sample_tokens_offsets_past_32_bits(ops):  # noqa: F811
    """Rows more than 2^31 elements into the logits and the noise."""
    import torch
    vocab, stride = 1000, (1 << 31) + 8
    for dtype in (torch.bfloat16, torch.float32):
        flat = torch.empty(stride + vocab, dtype=dtype, device="cuda")
        logits = torch.as_strided(flat, (2, vocab), (stride, 1))
        logits.copy_(torch.randn((2, vocab), device="cuda"))
        noise = torch.empty((2, vocab), device="cuda").exponential_()
        got = ops.sample_tokens(logits, noise)
        want = ops.sample_tokens(logits.contiguous(), noise)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        del flat, logits


# ---- all of them: a decoding step, streams, graphs, refusals ---------------------------------------
def _calls(ops, s):  # noqa: F811
    q = ops.norm_rope_append(s["q"], s["k"], s["v"], s["qw"], s["kw"], s["pos"], s["table"], s["kc"], s["vc"], s["slots"])
    out, lse = ops.prefix_attention(q, s["kc"], s["vc"], *s["prefix"])
    return (q, out, lse, *ops.sample_tokens(s["logits"], s["noise"], s["t"], s["top_k"], s["top_p"], s["min_p"]))


def _step_inputs():
    import torch
    q, k, v, pos, _, _, _ = _rope_inputs(6, 8, 2, 64, 64, "bf16", seed=11)
    c = _prefix_case([70], [6], [20] * 6, [1] * 6, 8, 2, 64, 16, "bf16", seed=11)
    slots = torch.tensor([int(c["table"][b, 20 // 16]) * 16 + 20 % 16 for b in range(6)], dtype=torch.int64, device="cuda")
    i32 = lambda a: _dev(np.asarray(a, np.int32))  # noqa: E731
    w = _sample_case(6, 3001, "bf16", ["all", "p", "k", "none", "greedy"], seed=12)
    qw, kw = _weights("one", 8, 2, 64, "bf16")
    return dict(q=q.contiguous(), k=k, v=v, pos=pos, qw=qw, kw=kw, kc=c["kc"], vc=c["vc"], slots=slots,
                prefix=[i32(c[n]) for n in ("ptable", "prefix", "groups", "table", "ctx", "starts")],
                logits=w["logits"], noise=w["noise"], t=_dev(w["temperature"]), top_k=_dev(w["top_k"]),
                top_p=_dev(w["top_p"]), min_p=_dev(w["min_p"]))


def test_other_stream_and_graph(ops):  # noqa: F811
    """The calls follow torch's current stream and may be captured; a replay reads the inputs of its time. Two graphs that
    share the memory of their workspaces, one replayed after the other, give what the calls give."""
    import torch
    s = _step_inputs()
    s["table"] = ops.rope_table(500, 64)
    want = _calls(ops, s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _calls(ops, s)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    d = dict(s, q=torch.zeros_like(s["q"]), logits=torch.zeros_like(s["logits"]))
    pool, graphs = torch.cuda.graph_pool_handle(), []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=pool):
            got = _calls(ops, d)
        graphs.append((graph, got))
    d["q"].copy_(s["q"])
    d["logits"].copy_(s["logits"])
    for graph, got in graphs + graphs[:1]:
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_streams_at_once(ops):  # noqa: F811
    """Calls on two streams at the same time, each with its own workspace and outputs."""
    import torch
    s = _step_inputs()
    s["table"] = ops.rope_table(500, 64)
    d = {**s, "q": s["q"] * 2, "kc": s["kc"].clone(), "vc": s["vc"].clone(), "logits": s["logits"] * 0.5}
    want = [[t.clone() for t in _calls(ops, x)] for x in (s, d)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i, x in enumerate((s, d)):
            with torch.cuda.stream(streams[i]):
                got[i].append(_calls(ops, x))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


def test_versions(ops):  # noqa: F811
    """What a call writes in place has a new version."""
    import torch
    s = _step_inputs()
    s["table"] = ops.rope_table(500, 64)
    before = s["kc"]._version, s["vc"]._version, s["q"]._version
    ops.norm_rope_append(s["q"], s["k"], s["v"], None, None, s["pos"], s["table"], s["kc"], s["vc"], s["slots"], out=s["q"])
    assert (s["kc"]._version, s["vc"]._version, s["q"]._version) == tuple(v + 1 for v in before)
    out = torch.empty_like(s["q"])
    v = out._version
    ops.prefix_attention(s["q"], s["kc"], s["vc"], *s["prefix"], out=out)
    assert out._version == v + 1
    ops.norm_rope(s["q"], None, s["pos"], s["table"], out=out)
    assert out._version == v + 2


def test_tensor_form_refusals(ops):  # noqa: F811
    import torch
    s = _step_inputs()
    table = ops.rope_table(500, 64)
    q, k, v, pos, qw, kc, vc, slots = (s[n] for n in ("q", "k", "v", "pos", "qw", "kc", "vc", "slots"))
    app, att, draw = ops.norm_rope_append, ops.prefix_attention, ops.sample_tokens
    bad = [
        lambda: ops.norm_rope(q, qw.float(), pos, table), lambda: ops.norm_rope(q, qw[:32], pos, table),
        lambda: ops.norm_rope(q, qw.expand(7, -1), pos, table), lambda: ops.norm_rope(q, qw.view(1, 1, 64), pos, table),
        lambda: ops.norm_rope(q, qw, pos.long(), table), lambda: ops.norm_rope(q, qw, pos[:3], table),
        lambda: ops.norm_rope(q[0], qw, pos, table), lambda: ops.norm_rope(q, qw.cpu(), pos, table),
        lambda: ops.norm_rope(q, torch.stack([qw, qw], 1)[:, 0], pos, table),
        lambda: ops.norm_rope(q, qw.clone().requires_grad_(), pos, table), lambda: ops.norm_rope(q, qw, pos, table, out=q.float()),
        lambda: app(q, k[:3], v, qw, qw, pos, table, kc, vc, slots), lambda: app(q, k, v, qw, qw.float(), pos, table, kc, vc, slots),
        lambda: app(q, k, v, qw, qw.expand(8, -1), pos, table, kc, vc, slots),
        lambda: app(q, k, v, qw, qw, pos, table, kc, vc, slots.int()), lambda: app(q, k, v, qw, qw, pos, table, kc[:, :, :1], vc, slots),
    ]
    for i, change in [(0, lambda t: t.long()), (0, lambda t: t[0]), (1, lambda t: t.float()), (1, lambda t: t[:0]),
                      (2, lambda t: t[:1]), (2, lambda t: t.cpu()), (3, lambda t: t[:2]), (4, lambda t: t.long()),
                      (5, lambda t: t[:3])]:
        args = list(s["prefix"])
        args[i] = change(args[i])
        bad.append(lambda args=args: att(q, kc, vc, *args))
    bad += [
        lambda: att(q, kc, vc.float(), *s["prefix"]), lambda: att(q.clone().requires_grad_(), kc, vc, *s["prefix"]),
        lambda: draw(s["logits"], s["noise"].bfloat16()), lambda: draw(s["logits"], s["noise"][:, :50]),
        lambda: draw(s["logits"].half(), s["noise"]), lambda: draw(s["logits"][0], s["noise"][0]),
        lambda: draw(s["logits"].t(), s["noise"].t()), lambda: draw(s["logits"], s["noise"], s["t"].double()),
        lambda: draw(s["logits"], s["noise"], s["t"][:2]), lambda: draw(s["logits"], s["noise"], None, s["top_k"].long()),
        lambda: draw(s["logits"], s["noise"], None, None, s["top_p"][:, None]), lambda: draw(s["logits"], s["noise"], 1.0),
        lambda: draw(s["logits"].clone().requires_grad_(), s["noise"]),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    from rank_adapter_apply_gb300.binding import LoraError
    with pytest.raises(LoraError, match="eps"):      # the library's own refusal, with its message
        ops.norm_rope(q, qw, pos, table, eps=-1.0)
    with pytest.raises(LoraError, match="n_kv_heads"):
        att(q[:, :3], kc, vc, *s["prefix"])
    with pytest.raises(LoraError, match="vocab"):
        draw(s["logits"][:, :0], s["noise"][:, :0])


def test_wide_prefixes_on_two_streams_and_replayed(ops):  # noqa: F811
    """Calls that fill the SMs' tensor memory, eager on two streams at once beside a graph of others: all as alone."""
    import torch
    cases = [_widen(_prefix_case([500, 90], [20, 9], [40, 0, 7] * 10, [nodes] * 30, 8, 1, 64, 16, "bf16", seed=20 + nodes),
                    2e8, size) for nodes, size in ((1, 0), (3, 2e8), (5, 0))]
    i32 = lambda a: _dev(np.asarray(a, np.int32))  # noqa: E731
    args = [(c["q"], c["kc"], c["vc"], i32(c["ptable"]), i32(c["prefix"]), i32(c["groups"]), i32(c["table"]), i32(c["ctx"]),
             i32(c["starts"]), c["bits"]) for c in cases]
    want = [ops.prefix_attention(*a) for a in args]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed = [ops.prefix_attention(*a) for a in args * 4]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    graph.replay()
    eager = []
    for turn in range(6):
        for s, first in zip(streams, (0, 1)):
            with torch.cuda.stream(s):
                eager.append((first, ops.prefix_attention(*args[first])))
    torch.cuda.synchronize()
    for i, (out, lse) in enumerate(replayed):
        assert torch.equal(out, want[i % 3][0]) and torch.equal(lse, want[i % 3][1])
    for i, (out, lse) in eager:
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])
