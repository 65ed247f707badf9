"""Decode and prefill over the block-scaled cache at the ends of its range: the
smallest scales and empty blocks."""
import math

import numpy as np
import pytest
import torch

import _block_ref as R
from paged_kv_cache_188_gb300 import api
from test_gpu_fp8_block import Cache, decode
from test_gpu_weights_evict import i32, weights_call

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.lib()


def prefill(c, q, qo, scale):
    k, v, table, rws, ke, ve = c.dev
    out = torch.full_like(q, math.nan)
    ws = api.alloc_workspace(api.pa_prefill_workspace_bytes())
    kv = i32(np.cumsum([0] + c.lens).tolist())
    api.pa_paged_prefill_attn_fp8_block(q, k, v, c.layer, i32(qo), kv, table, rws, scale, ke, ve, c.block, ws, out)
    assert api.pa_get_error(ws) == 0
    return out


def check_small(got, r, p_bits, v_step, what):
    """As _block_ref.check_out, for results near the smallest bf16 numbers: instead of its floor of 1e-37, one step of
    the subnormal bf16 numbers (2^-133: half of it for the result's rounding, the rest for fp32's subnormals in the
    partial sums, 2^-149 each) and `v_step`, the step in which V itself is held."""
    rel = 2.0 ** -p_bits + 2 * r["ds"][..., None] + 2.0 ** -18
    tol = 2.0 ** -8 * r["out"].abs() + rel * r["mean"] * 1.01 + r["n"] * 2.0 ** -26 * (r["pmax"] * r["vmax"])[..., None] \
        + 2.0 ** -133 + v_step
    bad = (got.double() - r["out"]).abs() - tol
    assert float(bad.max()) <= 0, f"{what}: off by {float(bad.max()):.3e} more than {float(tol.flatten()[bad.argmax()]):.3e}"


# ------------------------------------------------------- the smallest scales

@pytest.mark.parametrize("ve", [1, 2, 4, 8, 9, 10, 40, (0, 1), (0, 3), (1, 12), (0, 120)])
@pytest.mark.parametrize("D,block", [(128, 16), (64, 1)])
def test_decode_values_of_the_smallest_scales(ve, D, block):
    """V exponents from 0 (an empty block: zeros) and 1 (2^-126) on, one for all or two in turn, in requests of one
    warpgroup and of many."""
    c = Cache([9000, 700, 130, 3, 1], 2, D, 16, block, 81, exp_lo=112, exp_hi=118)
    pick = torch.tensor(ve if isinstance(ve, tuple) else (ve,), dtype=torch.uint8)
    c.ve[...] = pick[torch.randint(0, len(pick), c.ve.shape, generator=c.g)]
    c.cuda()
    q = torch.randn((len(c.lens), 8, D), generator=c.g).to(torch.bfloat16)
    out, ws = decode(c, q.cuda(), 0.05)
    assert api.pa_get_error(ws) == 0
    for b in range(len(c.lens)):
        k, v = c.values(b)
        r = R.attention(q[b][None].double(), k, v, 0.05)
        check_small(out[b][None].cpu(), r, 12, 0.0, f"V exponents {ve}, request {b}")


@pytest.mark.parametrize("ve", [1, 2, 4, 8, 9, (0, 3), (1, 12)])
def test_prefill_values_of_the_smallest_scales(ve):
    """The same in prefill, which holds V in bf16: below 2^-126 in steps of 2^-133."""
    c = Cache([300, 90], 2, 128, 16, 16, 82, exp_lo=112, exp_hi=118)
    pick = torch.tensor(ve if isinstance(ve, tuple) else (ve,), dtype=torch.uint8)
    c.ve[...] = pick[torch.randint(0, len(pick), c.ve.shape, generator=c.g)]
    c.cuda()
    q = torch.randn((130, 8, 128), generator=c.g).to(torch.bfloat16)
    out = prefill(c, q.cuda(), [0, 100, 130], 0.05)
    for b, (lo, hi) in enumerate(((0, 100), (100, 130))):
        k, v = c.values(b)
        r = R.attention(q[lo:hi].double(), k, v, 0.05, first=c.lens[b] - (hi - lo), terms=2.0 ** -19)
        check_small(out[lo:hi].cpu(), r, 8, 2.0 ** -134, f"V exponents {ve}, request {b}")


def test_decode_over_empty_blocks_gives_zeros():
    """Every block empty: whatever its bytes are (numbers), the output is 0 and every token weighs the same."""
    c = Cache([500, 20], 2, 128, 16, 16, 83)
    c.ke.zero_()
    c.ve.zero_()
    c.cuda()
    q = torch.randn((2, 8, 128), generator=c.g).to(torch.bfloat16).cuda()
    out, _ = decode(c, q, 0.05)
    assert torch.count_nonzero(out) == 0
    w = torch.zeros(c.table.shape, device="cuda")
    out, _ = weights_call(c, q, 0.05, w)
    assert torch.count_nonzero(out) == 0
    for b, n in enumerate(c.lens):
        assert float((w[int(c.rows[b]), :n] * n - 8).abs().max()) < 1e-4
