"""Rules of the decoding step's kernels that no run can show without a fault, read from their sources."""
import re

import pytest

from tests.test_step_source_rules import _code


@pytest.mark.parametrize("name", ["norm_rope.cu", "rope_common.cuh", "prefix_attention.cu", "prefix_rows.cu", "prefix_rows.cuh",
                                  "sample_tokens.cu", "tree_common.cuh"])
def test_inputs_are_read_by_ordinary_loads(name):
    """The kernel before may still write them when these kernels start: nothing goes through the read-only path."""
    code = _code(name)
    for what in ("load8_bf16", "__restrict__", "__ldg", "ld.global.nc"):
        assert what not in code, what


@pytest.mark.parametrize("name", ["norm_rope.cu", "prefix_attention.cu", "prefix_rows.cu", "sample_tokens.cu", "tree_attention_tc.cu"])
def test_every_kernel_waits_for_the_one_before(name):
    """Also where it has nothing to do: a kernel that ended earlier would let the one after it start too early."""
    code = _code(name)
    kernels = len(re.findall(r"__global__", code))
    waits = len(re.findall(r"\bgrid_dependency_wait\s*\(\)", code))
    assert waits == (1 if name == "tree_attention_tc.cu" else kernels)      # there in what both kernels call first
    if name == "tree_attention_tc.cu":
        for body in re.findall(r"__global__.*?\n}\n", code, flags=re.S):
            assert re.search(r"smem\[\];(?:\s*static_assert[^;]*;)?\s*tc_work<", body)


def test_tensor_memory_is_allocated_before_the_next_kernel_may_start():
    """A later kernel that had allocated what a CTA of this one still wants would wait for it, and it for the later one."""
    code = _code("tree_attention_tc.cu")
    at = [code.index(w) for w in ("grid_dependency_wait()", "tmem_alloc(", "tmem_relinquish()", "grid_launch_dependents()",
                                  "find_share<")]
    assert at == sorted(at)
    assert len(re.findall(r"grid_launch_dependents\(\)", code)) == 1
    # by the warp that allocates, and freed on both ways out
    assert re.search(r"if \(warp == 5\) \{\s*tc::tmem_alloc[^}]*grid_launch_dependents\(\);\s*\}", code)
    assert len(re.findall(r"free_tmem\(\);", code)) == 2
