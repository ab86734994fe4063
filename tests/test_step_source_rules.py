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
