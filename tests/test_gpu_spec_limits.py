"""Drafted tokens' calls at their limits: waits that run out midway, two calls at
the same time, offsets past 32 bits, the kernels' variants by size."""
import math

import numpy as np
import pytest
import torch

import _block_ref as R
import _spec_ref as S
from paged_kv_cache_188_gb300 import api
from test_gpu_abort_midway import _drive
from test_gpu_tree import P_BITS, check, make, queries, tree, trees
from test_gpu_verify_accept import Drafts, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.lib()
    yield
    api.pa_set_wait_timeout_ns(api.WAIT_TIMEOUT_DEFAULT_NS)


@pytest.mark.parametrize("block", [0, 16])
@pytest.mark.parametrize("D,page", [(128, 16), (64, 16), (128, 1)])
@pytest.mark.parametrize("chain", [False, True])
def test_calls_that_give_up_midway(D, page, block, chain):
    """Both kinds of pieces (one tile of rows, two), several to a CTA."""
    g = torch.Generator().manual_seed(D + page)
    context = torch.randint(0, 900, (40,), generator=g).tolist()
    nodes = [1 + 11 * (i % 7) for i in range(40)]
    c = make(context, nodes, 4, D, max(page, block), block, 31, layers=1, layer=0)
    _, mask = trees(c, chain)
    q = queries(c, 4, D).cuda()
    want, ws = tree(c, q, 0.05, mask)
    assert api.pa_get_error(ws) == 0
    _drive(lambda w, out: tree(c, q, 0.05, mask, ws=w, out=out), want, lambda: api.alloc_workspace(ws.numel()))


def test_two_calls_at_once():
    """Calls on two streams, each with its own workspace, whose CTAs share the GPU."""
    g = torch.Generator().manual_seed(3)
    cases = []
    for seed, block in ((41, 0), (42, 16)):
        context = torch.randint(100, 2000, (20,), generator=g).tolist()
        c = make(context, [9] * 20, 4, 128, 16, block, seed, layers=1, layer=0)
        _, mask = trees(c)
        q = queries(c, 4, 128).cuda()
        want, ws = tree(c, q, 0.05, mask)
        cases.append((c, q, mask, want, ws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [[torch.full_like(x[3], math.nan) for _ in range(6)] for x in cases]
    torch.cuda.synchronize()
    for i in range(6):
        for (c, q, mask, _, ws, st), out in zip(cases, outs):
            with torch.cuda.stream(st):
                tree(c, q, 0.05, mask, ws=ws, out=out[i])
    torch.cuda.synchronize()
    for (_, _, _, want, ws, _), out in zip(cases, outs):
        assert api.pa_get_error(ws) == 0
        for o in out:
            assert torch.equal(o.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("block", [0, 32])
def test_caches_past_32_bit_offsets(block):
    """A layer of more than 2^32 bytes: rows at both ends of the last layer."""
    Hkv, D, layers = 8, 128, 2
    size = (1 << 21) + 4096 if not block else (1 << 22) + 4096
    g = torch.Generator(device="cuda").manual_seed(5)
    n, m = 700, 6
    slots = torch.cat([torch.arange(300, device="cuda"), size - 1 - torch.arange(n - 300, device="cuda")]).int()
    shape = (layers, size, Hkv, D)
    if block:
        k, v = (torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2))
        ke, ve = (torch.full((layers, -(-size // block), Hkv), 120, dtype=torch.uint8, device="cuda") for _ in range(2))
        for buf in (k, v):
            x = (torch.randn((n, Hkv, D), generator=g, device="cuda") * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
            buf[1, slots.long()] = x.view(torch.uint8)
        val = [buf[1, slots.long()].view(torch.float8_e4m3fn).double().cpu() / 128 for buf in (k, v)]
        more = dict(k_exp=ke, v_exp=ve, block=block)
    else:
        k, v = (torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        for buf in (k, v):
            buf[1, slots.long()] = torch.randn((n, Hkv, D), generator=g, device="cuda").to(torch.bfloat16)
        val = [buf[1, slots.long()].double().cpu() for buf in (k, v)]
        more = {}
    assert layers * size * Hkv * D * (1 if block else 2) > 1 << 33
    q = torch.randn((m, 32, D), generator=g, device="cuda").to(torch.bfloat16)
    table = slots[None].contiguous()
    ws = api.alloc_workspace(api.pa_tree_workspace_bytes(32, Hkv, D))
    out = torch.full_like(q, math.nan)
    api.pa_paged_tree_attn(q, k, v, 1, i32([0, m]), table, i32([0]), i32([n]), 0.05, ws, out, **more)
    assert api.pa_get_error(ws) == 0
    ref = S.attention(q.double().cpu(), *val, 0.05, S.chain_seen(m), terms=2.0 ** -17 if block else 0.0)
    R.check_out(out.cpu(), ref, P_BITS, "past 32 bits")
    if block:
        return
    # the accepted nodes' rows move between the ends of both layers
    table[0, n - m:] = torch.tensor([5, size - 3, 7, size - 9, 11, size - 13], dtype=torch.int32)
    k[:, table[0, n - m:].long()] = torch.arange(m, device="cuda", dtype=torch.bfloat16)[None, :, None, None] + 1
    v[:, table[0, n - m:].long()] = -1 - torch.arange(m, device="cuda", dtype=torch.bfloat16)[None, :, None, None]
    new, freed, err = i32([0]), i32([-1] * m), i32([0])
    api.pa_kv_accept(table, i32([0]), i32([n]), i32([0, m]), i32([[0, 2, 3, 5]]), i32([4]), new, freed, k_buf=k, v_buf=v,
                     error_word=err)
    assert api.pa_get_error_word(err) == 0 and new.item() == n - 2
    assert k[:, table[0, n - m:n - 2].long(), 0, 0].tolist() == [[1, 3, 4, 6]] * 2
    assert v[:, table[0, n - m:n - 2].long(), 7, 127].tolist() == [[-1, -3, -4, -6]] * 2


def test_verify_rows_past_32_bit_offsets():
    V, T = 131072, 17000
    p = torch.zeros((T, V), device="cuda")                    # 2.2e9 numbers
    qo = i32([0, 2, T - 3, T])                                # (the second request has too many nodes)
    p[0, 5], p[1, 6] = 1.0, 1.0
    p[T - 3, V - 1], p[T - 2, V - 2], p[T - 1, 3] = 1.0, 1.0, 1.0
    tokens = torch.zeros(T, dtype=torch.int32, device="cuda")
    tokens[1], tokens[T - 2], tokens[T - 1] = 5, V - 1, V - 2
    parents = torch.zeros(T, dtype=torch.int32, device="cuda")
    parents[T - 1] = 1
    u, us = torch.full((T,), 0.5, device="cuda"), torch.full((3,), 0.5, device="cuda")
    acc, n, nxt, err = torch.empty((3, 4), dtype=torch.int32, device="cuda"), i32([9] * 3), i32([9] * 3), i32([0])
    api.pa_tree_verify(p, tokens, parents, qo, u, us, acc, n, nxt, error_word=err)
    assert api.pa_get_error_word(err) == api.DEVERR_LEN
    assert acc.tolist() == [[0, 1, -1, -1], [-1] * 4, [0, 1, 2, -1]]
    assert n.tolist() == [2, 0, 3] and nxt.tolist() == [6, -1, 3]


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("R,V", [(3, 70001), (90, 5000), (20, 9001), (1, 65536), (2, 65537), (170, 4096)])
def test_verify_by_size(R, V, drawn):
    """Every variant: rows kept in registers or read again, CTAs of 256 and 512 threads, clusters of one to eight."""
    d = Drafts([5] * R, V, R + V, False, drawn, sharp=0.5)
    d.u.mul_(0.2).add_(0.8)                                    # many refusals
    err = i32([0])
    out = d.call(err=err)
    assert api.pa_get_error_word(err) == 0
    d.check(out, f"{R} requests of {V}")


def test_verify_answers_do_not_depend_on_the_batch():
    """One request alone, among others and in a batch of another variant: the same token."""
    V = 30011
    d = Drafts([7], V, 77, False, True, sharp=0.5)
    one = [x.cpu() for x in d.call()]
    for R in (2, 40, 300):
        many = Drafts([7] * R, V, 77, False, True, sharp=0.5)
        many.p, many.f = d.p.repeat(R, 1), d.f.repeat(R, 1)
        many.tokens, many.parents = d.tokens * R, d.parents * R
        many.u, many.ul = d.u.repeat(R), d.ul.repeat(R)
        out = [x.cpu() for x in many.call()]
        for x, y in zip(out, one):
            assert (x == y[0]).all()


def test_tree_results_do_not_depend_on_other_requests_values():
    """The split changes with the batch; within one batch other requests' data change nothing."""
    c = make([700, 90, 300], [12, 5, 40], 2, 64, 16, 0, 17, layers=1, layer=0)
    _, mask = trees(c)
    q = queries(c, 4, 64)
    a, _ = tree(c, q.cuda(), 0.05, mask)
    q[:12] = 7.0
    b, _ = tree(c, q.cuda(), 0.05, mask)
    assert torch.equal(a[12:].view(torch.int16), b[12:].view(torch.int16))
    assert not torch.equal(a[:12].view(torch.int16), b[:12].view(torch.int16))


def test_masks_wider_than_the_nodes_need():
    c = make([200], [10], 1, 64, 16, 0, 18)
    seen, mask = trees(c)
    q = queries(c, 4, 64).cuda()
    a, _ = tree(c, q, 0.05, mask)
    wide = torch.cat([mask, torch.full((10, 9), -1, dtype=torch.int32, device="cuda")], 1).contiguous()
    b, ws = tree(c, q, 0.05, wide)
    assert api.pa_get_error(ws) == 0 and torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert np.isfinite(a.float().cpu().numpy()).all()


@pytest.mark.parametrize("D,block", [(128, 16), (64, 16), (128, 0), (64, 0)])
@pytest.mark.parametrize("order", [0, 1, 2])
def test_short_and_long_requests_in_turn(D, block, order):
    """Several requests to a CTA: of one tile of cached tokens (one stream has nothing to do), of many, of more rows than
    a stream has, behind one another in every order."""
    kinds = [(40, 3), (400, 9), (90, 5), (300, 40), (20, 1), (60, 2), (700, 33), (100, 6), (1000, 4), (5, 40)]
    g = torch.Generator().manual_seed(order)
    picks = [kinds[int(i)] for i in torch.randint(0, len(kinds), (70,), generator=g)]
    c = make([x[0] for x in picks], [x[1] for x in picks], 8, D, 16, block, 50 + order, layers=1, layer=0)
    seen, mask = trees(c)
    q = queries(c, 4, D)
    out, ws = tree(c, q.cuda(), 0.05, mask)
    assert api.pa_get_error(ws) == 0
    check(c, q, out, 0.05, seen, f"D={D} block={block} order {order}")
