"""The limits that the header sets to a decoding step's operators, at the places of a row and on the routes where a kernel
could keep them differently."""
import numpy as np
import pytest

from tests.test_gpu_decode_step import _run_sample, _sample_case
from tests.test_gpu_step import _close, _dev, _dt, _np, ops  # noqa: F401

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
@pytest.mark.parametrize("vocab", [40003, 300007])
def test_sample_tokens_far_token_before_a_likelier_one(ops, vocab, best, dtype):  # noqa: F811
    """A token below the limit that would win among its neighbours does not hide one above it; only the row's maximum,
    which lies elsewhere, tells them apart."""
    most = vocab // 4 * 3
    for near, far in ((most, most + 1), (most + 1, most), (vocab - 2, vocab - 1), (1, 0)):
        x, noise = np.full(vocab, -400.0), np.ones(vocab)
        x[17000], noise[17000] = 0.0, best
        x[near], noise[near] = -87.0, 1e-40
        x[far], noise[far] = -90.0, 0.0
        assert _drawn(ops, x, noise, dtype) == near
        assert _drawn(ops, x, noise, dtype, top_k=3) == near
        assert _drawn(ops, x, noise, dtype, top_p=0.5) == 17000


def _settled(c):
    """(tokens, settled, logprobs, tol) of a case: the 64-bit draw of every row, and whether fp32 has to find the same.

    In units of 2^-24, with z = ln p + a row's constant <= 0. A key p / noise: a rounding of z for the difference, for 1 / t
    and for the product, a unit (2) of exp and the division's 1: 3 |z| + 3, 4 allowed. A mass of some p: of each 5 |z| + 4
    (difference, 1 / t, the factor to powers of two, its constant, the product; exponential), weighted 5 E|z| + 4 of the
    total, and an addition for each of a thread's at most vocab / 256 + 1 tokens and 20 levels above them; the mass in front
    and the total are both off by that, and their border's product by 1. ln p: 3 |z| + 2 for z, the total's error, the logarithms'
    units."""
    x, noise = _np(c["logits"]), _np(c["noise"])
    rows, vocab = x.shape
    tokens, settled, logprobs, tol = np.zeros(rows, int), np.zeros(rows, bool), np.zeros(rows), np.zeros(rows)
    for r in range(rows):
        t, k, top_p, min_p = (float(c[n][r]) for n in ("temperature", "top_k", "top_p", "min_p"))
        z = (x[r] - x[r].max()) / (t if t > 0 else 1.0)
        p = np.exp(z)
        total, reach = p.sum(), (p * np.abs(z)).sum() / p.sum()
        of_key = 2.0 ** -24 * (3 * np.abs(z) + 4)
        of_mass = 2.0 ** -24 * (2 * (5 * reach + 4 + vocab / 256 + 21) + 1)
        order = np.argsort(-x[r], kind="stable")
        front = np.empty(vocab)
        front[order] = np.cumsum(p[order]) - p[order]
        rank = np.empty(vocab, int)
        rank[order] = np.arange(vocab)
        kept, near = np.ones(vocab, bool), np.zeros(vocab, bool)
        if k > 0:
            kept &= rank < k
        if top_p < 1:
            kept &= front < top_p * total
            near |= np.abs(front / total - top_p) < of_mass
        if min_p > 0:
            kept &= p >= min_p
            near |= np.abs(p / min_p - 1) < of_key
        kept[order[0]], near[order[0]] = True, False
        if t <= 0:
            kept, near = rank == 0, np.zeros(vocab, bool)
        key = np.where(kept, p / noise[r], -1.0)
        tokens[r] = best = int(key.argmax())
        rivals = kept & (key > key[best] * (1 - of_key - of_key[best]))
        rivals[best] = False
        unsure = near & (p / noise[r] > key[best] * (1 - of_key - of_key[best]))
        settled[r] = not rivals.any() and not unsure.any() and not near[best]
        logprobs[r] = z[best] - np.log(total)
        tol[r] = 2.0 ** -24 * (3 * abs(z[best]) + 2 + 5 * reach + 4 + vocab / 256 + 21 + 4 * (1 + np.log(total)))
    return tokens, settled, logprobs, tol


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab", [(5, 301), (3, 40001), (400, 1003), (64, 20011)])
@pytest.mark.parametrize("at", [(0, 0), (3, 1), (0, 1), (5, 2), (1, 3), (7, 0)])
def test_sample_tokens_row_by_row_at_different_offsets(ops, at, rows, vocab, dtype):  # noqa: F811
    """Wherever rows start, each settled one gives its token, and every row whose tokens are alike nearly the same ln p."""
    import torch
    c = _sample_case(rows, vocab, dtype, ["none", "all", "p", "k", "m"], seed=4)
    tokens, settled, logprobs, tol = _settled(c)
    assert (~settled).sum() <= 1 + rows // 20
    want = _run_sample(ops, c)
    for i, name in enumerate(("logits", "noise")):
        wide = torch.full((rows, vocab + 11 + i), float("nan"), dtype=c[name].dtype, device="cuda")
        wide[:, at[i]:at[i] + vocab] = c[name]
        c[name] = wide[:, at[i]:at[i] + vocab]
    got = _run_sample(ops, c)
    for drawn, ln_p in (want, got):
        assert (drawn.cpu().numpy()[settled] == tokens[settled]).all()
        _close(_np(ln_p)[settled], logprobs[settled], tol[settled])
    alike = (want[0] == got[0]).cpu().numpy()
    _close(_np(got[1])[alike], _np(want[1])[alike], 2 * tol[alike])


@pytest.mark.parametrize("sharp", [1.0, 30.0])
def test_sample_tokens_arguments_up_to_the_limit(ops, sharp):  # noqa: F811
    """Low temperatures, where ln p of the tokens that decide goes up to 87: the border of what fp32 tells apart goes with it."""
    c = _sample_case(200, 2003, "f32", ["none", "p", "m", "k"], seed=6, sharp=sharp)
    c["temperature"][:] = np.geomspace(0.05, 1.0, 200)
    r = np.random.default_rng(6)
    far = r.integers(0, 2003, 200)
    noise = c["noise"].cpu().numpy()
    noise[np.arange(200), far] = 1e-36                # tokens far down that may win
    c["noise"] = _dev(noise)
    z = (_np(c["logits"]) - _np(c["logits"]).max(1, keepdims=True)) / c["temperature"][:, None]
    keep = (np.abs(z[np.arange(200), far] + 87.3) > 0.1)  # not next to the limit of 2^-126
    tokens, settled, logprobs, tol = _settled(c)
    got, ln_p = _run_sample(ops, c)
    below = z[np.arange(200), tokens] < -87.3         # the definition in 64 bits has no such limit
    settled &= keep & ~below
    assert settled.sum() > 100
    assert (got.cpu().numpy()[settled] == tokens[settled]).all()
    _close(_np(ln_p)[settled], logprobs[settled], tol[settled])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens", [5, 3000])
def test_norm_rope_weights_of_no_heads(ops, tokens, dtype):  # noqa: F811
    """A weight whose rows do not exist is not looked at: the same bits as without it, wherever it points."""
    import ctypes

    import torch
    from rank_adapter_apply_gb300 import binding as B
    heads, dim = 32, 128
    gen = torch.Generator(device="cuda").manual_seed(8)
    x = torch.randn((tokens, heads, dim), generator=gen, device="cuda").to(_dt(dtype))
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda") % 500
    table, spare = ops.rope_table(500, dim), torch.zeros(2 * dim, dtype=x.dtype, device="cuda")
    out = []
    for weight in (None, spare.data_ptr() + spare.element_size()):
        y = torch.empty_like(x)
        rope = B.LoraRopeDesc(q=x.data_ptr(), q_token=heads * dim, q_head=dim, q_out=y.data_ptr(), q_out_token=heads * dim,
                              q_out_head=dim, positions=pos.data_ptr(), table=table.data_ptr(), n_positions=500, page_size=1,
                              n_tokens=tokens, n_heads=heads, head_dim=dim, rot_dim=dim,
                              dtype=B.LORA_DTYPE_BF16 if dtype == "bf16" else B.LORA_DTYPE_F32)
        d = B.LoraNormRopeDesc(rope=rope, k_weight=weight, eps=1e-6)
        B.lora_norm_rope(ctypes.byref(d), torch.cuda.current_stream().cuda_stream)
        out.append(y)
    assert torch.equal(out[0], out[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens", [3, 3000])
@pytest.mark.parametrize("dim", [50, 128])
def test_norm_rope_squares_out_of_range(ops, dim, tokens, dtype):  # noqa: F811
    """A head whose squares pass fp32's range is 0, and no other head is touched; one just below it is normed."""
    import torch
    x = torch.ones((tokens, 8, dim), dtype=_dt(dtype), device="cuda")
    x[1, 3], x[1, 4], x[2, 0, 1] = 2.0 ** 66, 2.0 ** 59, 2.0 ** 65
    pos, table = torch.zeros(tokens, dtype=torch.int32, device="cuda"), ops.rope_table(4, dim // 4 * 2)
    y = ops.norm_rope(x, None, pos, table).float()
    assert not y[1, 3].any() and not y[2, 0].any()
    y[1, 3] = y[2, 0] = 1.0
    assert (y - 1).abs().max() <= 2.0 ** -8      # 1 / sqrt(1 + 1e-6), rounded
