"""The drafted tokens' attention and tensor memory, read off the source: every access
lies in its stream's area, and what one warpgroup reads of the other's is ordered behind it."""
import os
import re

import pytest

from paged_kv_cache_188_gb300 import build as B

SOURCE = "pa_tree_attn.cu"


def text():
    return open(os.path.join(B.CSRC, SOURCE)).read()


def test_handover_of_the_other_streams_results():
    """Where a piece's end reads the other stream's O, the barrier in front of it has the fences of tensor memory on both
    sides: one in front of the arrival, one behind it."""
    src = text()
    read = src.index("C::ColO + D + ch * 32")
    barrier = src.rindex("named_bar_sync(1, 256)", 0, read)
    lines = [x.strip() for x in src[:read].splitlines()]
    at = max(i for i, x in enumerate(lines) if "named_bar_sync(1, 256)" in x)
    assert lines[at - 1] == "tc_fence_before();" and lines[at + 1] == "tc_fence_after();"
    assert src.count("named_bar_sync(1, 256)") == 1 and barrier < read
