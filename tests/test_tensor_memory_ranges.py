"""Every access of the tcgen05 kernels to tensor memory, read off the source: its
columns, at the last turn of the loops around it, lie in what the CTA allocated
and in the area (S or O of a tile) that the address names."""
import os
import re

import pytest

from paged_kv_cache_188_gb300 import build as B

CALL = re.compile(r"tmem_(?:ld|st)(16|32)\((\w+)((?: \+ [^,]+)?),")
LOOP = re.compile(r"for \(int (\w+) = (\d+); \1 < ([^;]+); (?:\+\+\1|\1 \+= (\d+))\)")


def accesses(name):
    """(line, width, base, offset expression, {loop variable: (bound, step)}) of each call."""
    lines = open(os.path.join(B.CSRC, name)).read().splitlines()
    for i, text in enumerate(lines):
        for m in CALL.finditer(text):
            loops, indent = {}, len(text) - len(text.lstrip())
            for j in [i] + list(range(i - 1, -1, -1)):
                lead = len(lines[j]) - len(lines[j].lstrip())
                if j != i and (not lines[j].strip() or lines[j].startswith("#") or lead >= indent):
                    continue
                for loop in LOOP.finditer(lines[j]):
                    loops.setdefault(loop[1], (loop[3], int(loop[4] or 1)))
                indent = min(indent, lead)
                if lead == 0:
                    break
            yield i + 1, int(m[1]), m[2], m[3].lstrip(" +"), loops


def last_column(width, offset, loops, names):
    """Columns behind the base that the access reaches: the largest offset plus its width."""
    expr = offset or "0"
    for var in sorted(set(re.findall(r"\b[A-Za-z_]\w*\b", expr)) - set(names)):
        assert var in loops, f"{var} is no variable of a loop around the access"
        bound, step = loops[var]
        bound = eval(bound.replace("/", "//").replace("C::", ""), {}, dict(names))
        names = dict(names, **{var: (bound - 1) // step * step})
    return eval(expr, {}, dict(names)) + width


@pytest.mark.parametrize("D", [64, 128])
def test_prefill(D):
    area = {"s_addr": 128, "o_addr": D}          # columns of S or P, and of O, of one tile
    seen = list(accesses("pa_prefill.cu"))
    assert len(seen) >= 5
    for line, width, base, offset, loops in seen:
        assert last_column(width, offset, loops, {"D": D}) <= area[base], f"pa_prefill.cu:{line}"


@pytest.mark.parametrize("GP", [4, 8, 16])
@pytest.mark.parametrize("e4m3", [True, False])
def test_block_decode(GP, e4m3):
    up = lambda x: (x + 15) // 16 * 16  # noqa: E731
    names = {"NQ": up((2 if e4m3 else 1) * GP), "NP": up((3 if e4m3 else 2) * GP), "lane_base": 0}
    seen = list(accesses("pa_decode_block.cuh"))
    assert len(seen) == 2
    for line, width, base, offset, loops in seen:
        assert last_column(width, offset, loops, names) <= {"s_col": 64, "o_col": 64}[base], f"pa_decode_block.cuh:{line}"
