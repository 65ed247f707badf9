"""The drafted tokens' attention and tensor memory, read off the source: every access
lies in its stream's area, and what one warpgroup reads of the other's is ordered behind it."""
import os
import re

import pytest

from paged_kv_cache_188_gb300 import build as B
from test_tensor_memory_ranges import accesses, last_column

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


def constant(name):
    return int(re.search(rf"constexpr (?:static )?uint32_t {name} = (\d+);", text())[1])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("X", [0, 1])
def test_loads_and_stores(D, X):
    """S (P over it) of stream X is columns 128 X .. 128 X + 127, O is D columns from ColO + D X on."""
    col_o = constant("ColO")
    assert "const uint32_t s_addr = tmem + lane_base + X * 128;" in text()
    seen = list(accesses(SOURCE))
    assert len(seen) == len(re.findall(r"tmem_(?:ld|st)\d+\(", text())) == 6
    for line, width, base, offset, loops in seen:
        where = f"{SOURCE}:{line}"
        if base == "s_addr":
            assert last_column(width, offset, loops, {}) <= 128, where
            continue
        assert base == "tmem" and offset.startswith("lane_base + C::ColO"), where
        rest = offset.replace("lane_base + C::ColO", "0")
        names = {"D": D, "X": X}
        other = rest.startswith("0 + D +")                 # stream B's columns, read by stream A at a joint piece's end
        lo = D * (1 if other else X)
        first = eval(re.sub(r"\bch\b", "0", rest), {}, names)
        assert first == lo and last_column(width, rest, loops, names) <= lo + D, where
    assert 2 * 128 <= col_o and col_o + 2 * D <= constant("kTrTmemCols")


@pytest.mark.parametrize("D", [64, 128])
def test_products(D):
    """The products' results and P lie in the same areas: S 128 columns wide, O D, P 64 words of S."""
    src = text()
    assert src.count("tmem + X * 128, smem_desc_sw128(q") == 2                       # S of both caches' products
    assert "tmem + C::ColO + X * D, tmem + X * 128 + kk * 8," in src                # O, and P in steps of 8 words
    assert "for (int kk = 0; kk < kTrTile / 16; ++kk)" in src and "kTrTile = 128" in src
    assert "idesc_bf16_f32(128, D, 0, 1)" in src and src.count("_f32(128, 128, 0, 0)") == 2
    assert (128 // 16) * 8 <= 128
