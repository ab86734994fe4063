"""The limits that the header sets to a decoding step's operators, at the places of a row and on the routes where a kernel
could keep them differently."""
import numpy as np
import pytest

from tests.test_gpu_step import _dev, _dt, ops  # noqa: F401

pytestmark = pytest.mark.gpu

FAR = float(np.log(2.0 ** -126))                  # tokens further than this below the maximum are not drawn


def _at_every_offset(x, noise, dtype):
    """Row x and its noise in rows that start at every place within 16 bytes, logits and noise at different ones."""
    import torch
    rows, vocab = 8, len(x)
    out = []
    for a, extra, kind in ((x, 9, _dt(dtype)), (noise, 11, torch.float32)):
        wide = torch.full((rows, (vocab + 15) // 8 * 8 + extra), float("nan"), dtype=kind, device="cuda")
        wide[:, 1:vocab + 1] = _dev(np.asarray(a, np.float32)).to(kind)
        out.append(wide[:, 1:vocab + 1])
    return out


def _drawn(ops, x, noise, dtype, temperature=None, top_k=None, top_p=None):  # noqa: F811
    """The token that all rows of _at_every_offset draw."""
    import torch
    logits, wide_noise = _at_every_offset(x, noise, dtype)
    each = lambda v, kind: None if v is None else torch.full((8,), v, dtype=kind, device="cuda")  # noqa: E731
    tokens, _ = ops.sample_tokens(logits, wide_noise, each(temperature, torch.float32), each(top_k, torch.int32),
                                  each(top_p, torch.float32))
    first, = set(tokens.tolist())
    return first


def _far_row(vocab, at, z, likely=3):
    """Row and noise: a few tokens at 0, one at z at once, all others out of reach."""
    x, noise = np.full(vocab, -400.0), np.ones(vocab)
    tops = [i for i in np.linspace(0, vocab - 1, likely + 2).astype(int)[1:-1] if i != at]
    x[tops] = 0.0
    noise[tops] = 1.0 + np.arange(len(tops))[::-1]
    x[at], noise[at] = z, 0.0
    return x, noise, tops[-1]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [23, 5001, 40003, 300007])
@pytest.mark.parametrize("z", [-90.0, -87.0, -100.0, -110.0])
def test_sample_tokens_far_tokens(ops, z, vocab, dtype):  # noqa: F811
    """A token of p < 2^-126 is not drawn even with noise 0, one above it is, whether it is the row's first or last
    element or inside a vector, and whether all tokens are in the race or few."""
    for at in (0, 1, vocab // 2 + 1, vocab - 2, vocab - 1):
        x, noise, top = _far_row(vocab, at, z)
        for top_k in (None, 4 if vocab > 4 else None, vocab - 1):
            assert _drawn(ops, x, noise, dtype, top_k=top_k) == (at if z > FAR else top), (at, top_k)


@pytest.mark.parametrize("temperature", [None, 0.75, 3.1])
def test_sample_tokens_next_to_the_limit(ops, temperature):  # noqa: F811
    """Logits on both sides of the limit: wherever the token lies, the draw is the same. p is off by 2^-24 of |z| for each of
    three roundings and by two units of exp, less than 2^-15 of it."""
    t = 1.0 if temperature is None else temperature
    border = np.float32(FAR * t)
    for n in list(range(-12, 13)) + [-500, 500]:
        z = float(border + n * np.spacing(border))
        drawn = set()
        for vocab in (23, 9001):
            for at in (0, vocab // 2 + 1, vocab - 1):
                x, noise, top = _far_row(vocab, at, z)
                drawn |= {_drawn(ops, x, noise, "f32", temperature, top_k) == at for top_k in (None, 4)}
        assert len(drawn) == 1, (n, z)
        if abs(n) == 500:                         # spacing() of a negative number is negative
            assert drawn == {bool(z > border)}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("best", [1.0, float("nan")])
def test_sample_tokens_far_token_before_a_likelier_one(ops, best, dtype):  # noqa: F811
    """A token below the limit that would win among its neighbours does not hide one above it; only the row's maximum,
    which lies elsewhere, tells them apart."""
    vocab = 40003
    for near, far in ((30001, 30002), (30002, 30001), (vocab - 2, vocab - 1), (1, 0)):
        x, noise = np.full(vocab, -400.0), np.ones(vocab)
        x[17000], noise[17000] = 0.0, best
        x[near], noise[near] = -87.0, 1e-40
        x[far], noise[far] = -90.0, 0.0
        assert _drawn(ops, x, noise, dtype) == near
        assert _drawn(ops, x, noise, dtype, top_k=3) == near
        assert _drawn(ops, x, noise, dtype, top_p=0.5) == 17000
