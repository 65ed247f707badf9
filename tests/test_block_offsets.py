"""The exponents' offset of a layer, at the sizes the entry points let through.
The function is evaluated by the compiler, where a signed overflow is an error."""
import os
import shutil
import subprocess

import pytest

from paged_kv_cache_188_gb300 import build as B

CUDA = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")


@pytest.mark.parametrize("layer,size,hkv,block", [
    (0, 2 ** 31 - 18, 1, 128),          # the largest layer: size + block - 1 passes 2^31
    (0, 2 ** 31 - 18, 8, 1),
    (1, 2 ** 30 - 9, 8, 1),             # offsets past 2^32
    (3, 2 ** 29 - 5, 16, 128),
    (2, 65, 3, 16),                     # a last block that is short
    (1, 64, 2, 64),
])
def test_layer_offset(layer, size, hkv, block):
    cxx = shutil.which("g++")
    if not cxx or not os.path.exists(os.path.join(CUDA, "cuda.h")):
        pytest.skip("no host compiler or CUDA headers")
    want = layer * -(-size // block) * hkv
    src = f'#include "pa_internal.h"\nstatic_assert(pa::block_layer_offset({layer}, {size}, {hkv}, {block}) == {want}LL, "offset");\n'
    r = subprocess.run([cxx, "-std=c++17", "-fsyntax-only", "-x", "c++", "-I" + B.CSRC, "-I" + B.INCLUDE, "-I" + CUDA, "-"],
                       input=src, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
