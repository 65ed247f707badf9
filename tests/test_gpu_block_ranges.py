"""Decode and prefill over the block-scaled cache at the ends of its range: the
smallest scales, empty blocks, contexts past 64K tokens, and the tables that an
eviction leaves, single slots of blocks larger than one."""
import math

import numpy as np
import pytest
import torch

import _block_ref as R
from paged_kv_cache_188_gb300 import api
from test_gpu_fp8_block import Cache, check_decode, decode
from test_gpu_weights_evict import Bf16Cache, check_weights, i32, weights_call

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


@pytest.mark.parametrize("block", [16, 1])
def test_prefill_nan_key_is_seen_from_its_token_on(block):
    """A NaN among a later token's keys reaches the queries that see it and no other."""
    c = Cache([300], 2, 128, 16, block, 89)
    c.k[1, c.slots[0][150], 1, 7] = 127
    c.cuda()
    q = torch.randn((300, 8, 128), generator=c.g).to(torch.bfloat16)
    out = prefill(c, q.cuda(), [0, 300], 0.05)
    assert torch.isnan(out[150:, 4:].float()).all()
    k, v = c.values(0)
    r = R.attention(q[:, :4].double(), k[:, :1], v[:, :1], 0.05, first=0, terms=2.0 ** -19)
    R.check_out(out[:, :4].cpu(), r, 8, "the other kv head")
    r = R.attention(q[:150, 4:].double(), k[:150, 1:], v[:150, 1:], 0.05, first=0, terms=2.0 ** -19)
    R.check_out(out[:150, 4:].cpu(), r, 8, "queries before the NaN")


# ------------------------------------------------------------- long contexts

@pytest.mark.parametrize("block", [0, 16])
def test_weights_past_64k_tokens(block):
    """One request of 70001 tokens beside a short one, the second of two layers."""
    lens = [70001, 300]
    c = (Cache(lens, 1, 64, 16, block, 84) if block else Bf16Cache(lens, 1, 64, 16, 84)).cuda()
    q = torch.randn((2, 4, 64), generator=c.g).to(torch.bfloat16)
    w = torch.rand(c.table.shape, generator=c.g)
    dw = w.cuda()
    out, ws = weights_call(c, q.cuda(), 0.1, dw)
    assert api.pa_get_error(ws) == 0
    check_weights(c, q, out, w, dw, 0.1, f"70001 tokens, block {block}")
    if block:
        again, _ = decode(c, q.cuda(), 0.1)
        assert torch.equal(again.view(torch.int16), out.view(torch.int16))


# ------------------------------------------------- tables that eviction left

def evicted(c, budget, recent, seed):
    """pa_kv_evict by random weights on the cache's table: c's slots, lengths and device table as it leaves them."""
    g = torch.Generator().manual_seed(seed)
    w = torch.rand(c.table.shape, generator=g)
    new, freed = i32([-1] * len(c.lens)), torch.zeros((len(c.lens), c.table.shape[1]), dtype=torch.int32, device="cuda")
    dw = w.cuda()
    api.pa_kv_evict(c.dev[2], c.dev[3], c.dlens, dw, budget, recent, new, freed)
    for b, n in enumerate(c.lens):
        row = int(c.rows[b])
        kept, _, _ = R.evict(c.slots[b].tolist(), w[row, :n].tolist(), budget, recent)
        assert c.dev[2][row, :len(kept)].tolist() == kept and int(new[b]) == len(kept)
        c.slots[b], c.lens[b] = torch.tensor(kept), len(kept)
    c.dlens = new
    return dw


EVICT = [(128, 16, 16), (128, 32, 32), (64, 16, 4), (64, 128, 128)]


@pytest.mark.parametrize("D,page,block", EVICT)
def test_decode_of_an_evicted_table(D, page, block):
    c = Cache([2000, 900, 401, 400, 7], 2, D, page, block, 85).cuda()
    evicted(c, 400, 33, 1)
    assert int((c.slots[0][1:] - c.slots[0][:-1] != 1).sum()) > 200      # single slots, not runs
    q = torch.randn((5, 8, D), generator=c.g).to(torch.bfloat16)
    out, ws = decode(c, q.cuda(), 0.05)
    assert api.pa_get_error(ws) == 0
    check_decode(c, q, out, 0.05, f"after eviction, page {page} block {block}")


@pytest.mark.parametrize("D,page,block", EVICT + [(128, 16, 0), (64, 16, 0)])
def test_weights_of_an_evicted_table(D, page, block):
    c = (Cache([2000, 900, 401, 400, 7], 2, D, page, block, 86) if block else Bf16Cache([2000, 900, 401, 400, 7], 2, D, page, 86)).cuda()
    dw = evicted(c, 400, 33, 2)
    w = dw.cpu()
    q = torch.randn((5, 8, D), generator=c.g).to(torch.bfloat16)
    out, ws = weights_call(c, q.cuda(), 0.05, dw)
    assert api.pa_get_error(ws) == 0
    check_weights(c, q, out, w, dw, 0.05, f"after eviction, page {page} block {block}")


@pytest.mark.parametrize("D,page,block", EVICT)
def test_prefill_behind_an_evicted_prefix(D, page, block):
    """New tokens behind what an eviction kept: scattered slots, then whole pages."""
    c = Cache([1200, 500, 90], 2, D, page, block, 87).cuda()
    evicted(c, 230, 200, 3)                                # the last 200 stay: 130 of them new tokens below
    new = [130, 1, 60]
    q = torch.randn((sum(new), 8, D), generator=c.g).to(torch.bfloat16)
    qo = np.cumsum([0] + new).tolist()
    out = prefill(c, q.cuda(), qo, 0.05)
    for b, n in enumerate(new):
        k, v = c.values(b)
        r = R.attention(q[qo[b]:qo[b] + n].double(), k, v, 0.05, first=c.lens[b] - n, terms=2.0 ** -19)
        R.check_out(out[qo[b]:qo[b] + n].cpu(), r, 8, f"behind an evicted prefix, request {b}")


@pytest.mark.parametrize("D,page,block", [(128, 16, 16), (64, 32, 8)])
def test_captured_eviction_then_decode(D, page, block):
    """Decode with weights, eviction, and decode over the table that it left, captured together; the decode behind the
    eviction with overlap off or safe, as the table is its index input."""
    c = Cache([1000, 350, 60], 2, D, page, block, 88).cuda()
    table0, lens0 = c.dev[2].clone(), c.dlens.clone()
    q = torch.randn((3, 8, D), generator=c.g).to(torch.bfloat16).cuda()
    w, newl = torch.zeros(c.table.shape, device="cuda"), torch.zeros_like(c.dlens)
    freed = torch.zeros((3, c.table.shape[1]), dtype=torch.int32, device="cuda")
    ws = api.alloc_workspace(api.pa_decode_weights_workspace_bytes(3, sum(c.lens), 8, 2, D))
    out1, out2 = torch.empty_like(q), torch.empty_like(q)

    def chain():
        c.dev[2].copy_(table0)
        c.dlens.copy_(lens0)
        w.zero_()
        weights_call(c, q, 0.05, w, ws=ws, out=out1)
        api.pa_kv_evict(c.dev[2], c.dev[3], c.dlens, w, 128, 16, c.dlens, freed)
        weights_call(c, q, 0.05, w, ws=ws, out=out2)

    chain()
    torch.cuda.synchronize()
    want = [x.clone() for x in (out1, out2, w, c.dev[2], c.dlens, freed)]
    assert c.dlens.tolist() == [128, 128, 60]
    # the second output is that of the kept slots
    keep = Cache([1000, 350, 60], 2, D, page, block, 88)
    keep.lens = c.dlens.tolist()
    keep.slots = [c.dev[2][int(c.rows[b]), :n].cpu().long() for b, n in enumerate(keep.lens)]
    assert all(set(keep.slots[b].tolist()) <= set(c.slots[b].tolist()) for b in range(3))
    check_decode(keep, q.cpu(), out2, 0.05, "behind the eviction")
    try:
        for mode in (api.OVERLAP_OFF, api.OVERLAP_SAFE):
            api.pa_set_launch_overlap(mode)
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr):
                chain()
            for _ in range(3):
                for x in (out1, out2, w, freed):
                    x.zero_()
                gr.replay()
                torch.cuda.synchronize()
                for x, y in zip((out1, out2, w, c.dev[2], c.dlens, freed), want):
                    assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), mode
    finally:
        api.pa_set_launch_overlap(api.OVERLAP_OFF)
    assert api.pa_get_error(ws) == 0
