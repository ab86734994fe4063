"""prefix_attention of requests with more than 64 query rows: chunks of prompts behind a prefix, without a mask and with
masks of several words. Tolerances as in test_gpu_decode_step.py's _check_prefix."""
import numpy as np
import pytest

from tests import decode_reference as ref
from tests.test_gpu_decode_step import _run_prefix, _widen
from tests.test_gpu_step import ROUND, _close, _dev, _dt, _np, ops  # noqa: F401

pytestmark = pytest.mark.gpu


def _chunks(prefix, members, ctx, nodes, heads, kv, dim, page, dtype, words, seed=0, first=0):
    """As _prefix_case, with masks of `words` words: node i sees itself, about half of the nodes before it, one row nothing
    of its tree. Cache rows that no query sees are NaN."""
    r = np.random.default_rng(seed)
    per = max(-(-(c + n) // page) for c, n in zip(ctx, nodes))
    shared = max(1, max(-(-p // page) for p in prefix))
    pages = per * len(ctx) + shared * len(prefix) + 1
    ids = r.permutation(pages).astype(np.int32)
    table = ids[:per * len(ctx)].reshape(len(ctx), per)
    ptable = ids[per * len(ctx):per * len(ctx) + shared * len(prefix)].reshape(len(prefix), shared)
    kc = np.full((pages, page, kv, dim), np.nan)
    vc = np.full_like(kc, np.nan)
    for t, n in [(ptable[g], prefix[g]) for g in range(len(prefix))] + [(table[b], ctx[b] + nodes[b]) for b in range(len(ctx))]:
        for p in range(n):
            kc[t[p // page], p % page] = r.standard_normal((kv, dim))
            vc[t[p // page], p % page] = r.standard_normal((kv, dim))
    starts = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int64)
    total = int(starts[-1])
    mask = np.zeros((total, 64 * words), bool)
    for b, n in enumerate(nodes):
        own = np.tril(r.random((n, n)) < 0.5) | np.eye(n, dtype=bool)
        mask[starts[b]:starts[b + 1], :n] = own[:, :64 * words]
    mask[total - 1] = False
    bits = np.packbits(mask, axis=1, bitorder="little").view(np.int64).reshape(total, words)
    return dict(q=_dev(r.standard_normal((total, heads, dim)), _dt(dtype)), kc=_dev(kc, _dt(dtype)), vc=_dev(vc, _dt(dtype)),
                table=table, ptable=ptable, prefix=list(prefix),
                groups=np.concatenate([[first], first + np.cumsum(members)]).astype(np.int64), ctx=list(ctx), starts=starts,
                mask=mask, bits=_dev(bits), dtype=dtype)


def _check(c, out, lse, masked):
    sees = (lambda t, i, j: j < c["mask"].shape[1] and c["mask"][t, j]) if masked else (lambda t, i, j: j <= i)
    want, want_lse, mass, reach = ref.prefix_attention(_np(c["q"]), _np(c["kc"]), _np(c["vc"]), c["ptable"], c["prefix"],
                                                       c["groups"], c["table"], c["ctx"], c["starts"], sees,
                                                       c["q"].shape[2] ** -0.5)
    part = 2.0 ** -8 if c["dtype"] == "bf16" else 2.0 ** -21
    _close(_np(out), want, ROUND[c["dtype"]] * np.abs(want) + (part + 2.0 ** -20 * (1 + reach[:, :, None])) * mass)
    empty = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(_np(lse)), empty) and not _np(out)[empty].any()
    _close(np.where(empty, 0, _np(lse)), np.where(empty, 0, want_lse),
           2.0 ** -20 * (1 + reach + np.abs(np.where(empty, 0, want_lse))))


CASES = [
    # prefix, members, contexts, nodes, heads, kv heads, head dim, page, words, first request with a group
    ([300], [1], [0], [200], 4, 1, 64, 16, 4, 0),                  # a prompt behind a prefix
    ([130], [3], [0, 70, 5], [129, 1, 65], 4, 2, 72, 16, 3, 0),    # beside a single token
    ([64, 0], [1, 1], [33, 0, 64, 9], [97, 190, 64, 100], 3, 1, 128, 32, 2, 1),   # past the mask's words; no group, no prefix
    ([40], [2], [17, 0], [150, 80], 10, 1, 32, 12, 3, 0),          # pages that take no box of eight rows
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("widths", [(0, 0), (2e8, 0), (0, 2e8), (2e8, 2e8)])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[3])}of{c[0]}")
def test_prefix_attention_chunks(ops, case, widths, masked, dtype):  # noqa: F811
    c = _widen(_chunks(*case[:8], dtype, case[8], first=case[9]), *widths)
    _check(c, *_run_prefix(ops, c, mask=masked), masked)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefix_attention_chunk_after_chunk(ops, dtype):  # noqa: F811
    """A prompt's rows in two calls, the second with the first's keys as its context, are those of one call."""
    c = _chunks([90], [1], [0], [210], 4, 1, 64, 16, dtype, 4, seed=1)
    whole = _run_prefix(ops, c, mask=False)
    _check(c, *whole, False)
    tol = 2.0 ** -6 if dtype == "bf16" else 2.0 ** -18
    for lo, hi in ((0, 130), (130, 210)):
        part = dict(c, q=c["q"][lo:hi], ctx=[lo], starts=np.array([0, hi - lo]))
        out, lse = _run_prefix(ops, part, mask=False)
        assert ((out - whole[0][lo:hi]).abs() <= tol * (1 + whole[0][lo:hi].abs())).all()
        assert (lse - whole[1][lo:hi]).abs().max() < 2.0 ** -15
