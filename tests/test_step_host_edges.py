"""CPU tests of refusals of the drafted-token step's calls that go by several arguments together."""
import ctypes

import numpy as np
import pytest

from rank_adapter_apply_gb300 import binding as B
from tests.test_step_host import _linear, _rope, _tree, lib  # noqa: F401

OVERLAPS = [
    ("lora_tree_attention", _tree, [
        dict(out_token=0), dict(out_head=0), dict(out_token=0, out_head=0), dict(out_head=8), dict(out_token=16),
        dict(out_token=32), dict(out_token=16, out_head=24), dict(out_token=24, out_head=16, n_heads=8)]),
    ("lora_rope", _rope, [
        dict(q_out_token=0), dict(q_out_head=0), dict(q_out_head=15), dict(q_out_token=16), dict(q_out_token=-32),
        dict(q_out_token=48, q_out_head=32), dict(cache_page=0), dict(cache_slot=0), dict(cache_slot=8),
        dict(cache_head=0, n_kv_heads=2), dict(cache_page=128), dict(cache_head=16, cache_slot=16, n_kv_heads=2)]),
    ("lora_base_linear", _linear, [dict(y_stride=0), dict(y_stride=7), dict(y_stride=-8)]),
]


@pytest.mark.parametrize("name,make,change", [(n, m, c) for n, m, cs in OVERLAPS for c in cs])
def test_overlapping_rows_of_outputs_are_refused(lib, name, make, change):  # noqa: F811
    d = make(**change)
    assert getattr(lib, name)(ctypes.byref(d), None) == B.LORA_ERR_ARG
    assert name[5:] in B.last_error()


def _apart(n0, s0, n1, s1, length):
    """Whether the rows share no element, by listing them."""
    first = (np.arange(n0)[:, None] * s0 + np.arange(n1)[None, :] * s1).reshape(-1)
    at = (first[:, None] + np.arange(length)).reshape(-1)
    return len(np.unique(at)) == len(at)


def test_rows_are_refused_only_where_they_overlap(lib):  # noqa: F811
    """Random strides, nested, interleaved and overlapping: refused exactly where two rows share an element. What is not
    refused goes on to a check that comes later, of a NULL workspace, so that nothing is queued anywhere."""
    r = np.random.default_rng(3)
    seen = {True: 0, False: 0}
    for _ in range(4000):
        n0, n1, length = int(r.integers(1, 6)), int(r.integers(1, 6)), 8
        s0, s1 = (int(s) * 8 for s in r.integers(0, 12, 2))
        d = _tree(n_tokens=n0, n_heads=n1, n_kv_heads=1, head_dim=length, out_token=s0, out_head=s1, workspace=None)
        assert lib.lora_tree_attention(ctypes.byref(d), None) == B.LORA_ERR_ARG
        apart = _apart(n0, s0, n1, s1, length)
        assert ("overlap" in B.last_error()) == (not apart), (n0, s0, n1, s1)
        assert apart == ("workspace" in B.last_error())
        seen[apart] += 1
    assert min(seen.values()) > 500
