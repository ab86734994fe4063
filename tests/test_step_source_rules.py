"""Rules of the step's kernels that no run can show without a fault, read from their sources."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rank_adapter_apply_gb300", "csrc")


def _code(name):
    """The source without comments and the text of its asm statements kept."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


@pytest.mark.parametrize("name", ["tree_attention_tc.cu", "base_linear_tc.cu"])
def test_a_wait_that_gives_up_leaves_nobody_waiting(name):
    """A warp whose bounded wait gave up leaves its role for the block's last barrier. So no role may wait at a barrier
    of some of the warps that has no bound, and a wait's outcome is the warp's, never a lane's own."""
    code = _code(name)
    assert not re.search(r"\bnamed_bar\s*\(|\bbar\.sync\b|\bbarrier\.sync\b", code)
    assert not re.search(r"__all_sync\([^;]*\bok\s*\)\s*\)\s*(break|return)", code)
    assert not re.search(r"__all_sync\([^;]*\bwait\s*\(", code)


def test_activations_are_read_by_ordinary_loads():
    """The step's kernels start while the kernel before them still writes: what it writes may not be read through the
    read-only path, which is for memory that nobody writes while the kernel runs. The words, scales and zeros of
    base_linear are such memory."""
    for name in ("base_linear.cu", "base_linear_tc.cu", "rope.cu", "tree_attention.cu", "tree_attention_tc.cu",
                 "tree_attention_f32.cu", "tree_common.cuh", "verify_drafts.cu", "step_util.cuh"):
        code = _code(name)
        assert "load8_bf16" not in code and "__restrict__" not in code, name
        for what in re.findall(r"__ldg\(\s*([^;]*)", code):
            assert name == "base_linear.cu" and re.match(r"[sz]src\[h\]", what), (name, what)
        for what in re.findall(r"ld\.global\.nc", code):
            assert name == "base_linear.cu" and re.search(r"uint4 load_w\(const uint8_t \*p\)", code)
    assert re.findall(r"\bload_w\(\s*(\w+)", _code("base_linear.cu")) == ["const", "wsrc"]
