"""Attention over many keys: a row whose maximum stands does not change when the maxima of other rows move."""
import numpy as np
import pytest

from tests.test_gpu_step import _close, _dev, _dt, _np, ops  # noqa: F401

pytestmark = pytest.mark.gpu


def _inputs(dtype, requests=64, kv=16, heads=64, keys=8000, page=64, dim=8):
    """Keys (1, a, 0 ..) whose a rises by one every 64 of them. Query heads (s, 0, ..) score s at every key, (0, 1, 0 ..) more
    and more; both lie in each tile of rows. All requests read the same pages."""
    pages = -(-keys // page)
    k = np.zeros((pages, page, kv, dim))
    at = np.arange(keys)
    k[at // page, at % page, :, 0] = 1.0
    k[at // page, at % page, :, 1] = (at // 64)[:, None]
    v = np.ones_like(k)
    v[:, :, :, 0] = (np.arange(pages * page).reshape(pages, page) < keys // 2)[:, :, None]
    q = np.zeros((requests, heads, dim))
    q[:, 0::2, 0] = 64.0 + 0.5 * np.arange(heads // 2)          # bf16 has them all
    q[:, 1::2, 1] = 1.0
    table = np.broadcast_to(np.arange(pages, dtype=np.int32), (requests, pages))
    i32 = lambda a: _dev(np.array(a, np.int32))  # noqa: E731
    return dict(q=_dev(q, _dt(dtype)), k=_dev(k, _dt(dtype)), v=_dev(v, _dt(dtype)), table=i32(table),
                ctx=i32(np.full(requests, keys - 1)), starts=i32(np.arange(requests + 1)), keys=keys)


def _check(c, out, lse):
    """Scores and values are exact. In units of 2^-24: an lse is its score times two rounded factors, rounded twice, 4 s; each
    weight's argument is off by less than a rounding of the score in powers of two, 1.5 s; the sum has at most 8000 / 16 + 16
    roundings of a thread and its joins' and 4 units of each of 32 exponentials that join parts. Of a weight's rounding to
    bf16 the mean of v keeps 2^-8."""
    heads, keys = c["q"].shape[1], c["keys"]
    s = _np(c["q"])[0, :, 0]
    steps = np.arange(keys) // 64
    z = np.where(np.arange(heads)[:, None] % 2 == 0, s[:, None], steps[None, :].astype(float))
    top = z.max(1)
    w = np.exp(z - top[:, None])
    want = top + np.log(w.sum(1))
    tol = 2.0 ** -24 * (5.5 * top + keys / 16 + 16 + 128)
    _close(_np(lse), np.broadcast_to(want, lse.shape), np.broadcast_to(tol, lse.shape))
    share = (w[:, :keys // 2].sum(1) / w.sum(1))[None, :]
    _close(_np(out)[:, :, 0], np.broadcast_to(share, lse.shape), 2.0 ** -8 if c["q"].element_size() == 2 else tol)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefix_attention_maximum_of_other_rows(ops, dtype):  # noqa: F811
    import torch
    c = _inputs(dtype)
    none = torch.zeros((0, 1), dtype=torch.int32, device="cuda")
    _check(c, *ops.prefix_attention(c["q"], c["k"], c["v"], none, none[:, 0], torch.zeros(1, dtype=torch.int32, device="cuda"),
                                    c["table"], c["ctx"], c["starts"], scale=1.0))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tree_attention_maximum_of_other_rows(ops, dtype):  # noqa: F811
    c = _inputs(dtype)
    _check(c, *ops.tree_attention(c["q"], c["k"], c["v"], c["table"], c["ctx"], c["starts"], scale=1.0))
