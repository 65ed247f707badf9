"""Drafted tokens' calls where a batch holds requests that cannot be read, or rows whose
query is no number: the others are answered as they are in a batch without them."""
import math

import pytest
import torch

import _spec_ref as S
from paged_kv_cache_188_gb300 import api
from test_gpu_tree import check, make, pack, queries, tree
from test_gpu_verify_accept import Batch, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.lib()


def batch(qo, T, valid, context, Hkv, D, block, seed):
    """Requests with the starts `qo`, of which those of `valid` can be read, over contexts that several CTAs share."""
    nodes = [qo[r + 1] - qo[r] if r in valid else 1 for r in range(len(qo) - 1)]
    c = make([context if r in valid else 10 for r in range(len(nodes))], nodes, Hkv, D, 16, block, seed, layers=1, layer=0)
    c.qo = qo
    seen = [S.tree_seen(S.random_parents(n, c.g)) for n in nodes]
    q = torch.randn((T, 4 * Hkv, D), generator=c.g).to(torch.bfloat16)
    mask = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    for r in valid:
        mask[qo[r]:qo[r + 1]] = pack([seen[r]])
    return c, q, seen, mask


def others(out, qo, valid):
    """Rows of no request that is read."""
    mine = [t for r in valid for t in range(qo[r], qo[r + 1])]
    return out[[t for t in range(out.shape[0]) if t not in mine]]


BAD_STARTS = [([0, 9, 5, 8], 8, [2]),
              ([0, 4, 1000, 12, 16], 16, [0, 3]),
              ([0, 4, -7, -7, 4, 9], 9, [0, 4]),
              ([0, 4, 1000, 1000, 12, 12, 16], 16, [0, 5]),
              ([7, 7, 0, 6], 6, [2]),
              ([-4, 4, 8, 12, 16], 16, [1, 2, 3]),
              ([0, 4, 8, 12, 20], 16, [0, 1, 2])]


@pytest.mark.parametrize("qo,T,valid", BAD_STARTS)
@pytest.mark.parametrize("context", [100, 9000])
@pytest.mark.parametrize("block", [0, 16])
def test_starts_out_of_range(qo, T, valid, context, block):
    """A start that is out of range leaves out the requests that it bounds, and no other."""
    c, q, seen, mask = batch(qo, T, valid, context, 2, 64, block, 60 + T)
    out, ws = tree(c, q.cuda(), 0.05, mask)
    assert api.pa_get_error(ws) == api.DEVERR_LEN
    check(c, q, out, 0.05, seen, f"starts {qo}", reqs=valid)
    assert torch.isnan(others(out, qo, valid).float()).all()


def test_a_start_out_of_range_among_many():
    """One bad start in the middle of a batch: the two requests around it are left out."""
    g = torch.Generator().manual_seed(5)
    counts = torch.randint(0, 7, (90,), generator=g).tolist()
    qo = [0]
    for n in counts:
        qo.append(qo[-1] + n)
    T, at = qo[-1], 41
    for bad in (-1, T + 1, 2 ** 31 - 1, -2 ** 31):
        starts = qo[:at] + [bad] + qo[at + 1:]
        valid = [r for r in range(90) if r not in (at - 1, at) and counts[r]]
        c, q, seen, mask = batch(starts, T, valid, 700, 8, 128, 0, 61)
        out, ws = tree(c, q.cuda(), 0.05, mask)
        assert api.pa_get_error(ws) == api.DEVERR_LEN
        check(c, q, out, 0.05, seen, f"start {bad}", reqs=valid)
        assert torch.isnan(others(out, starts, valid).float()).all()


OVERLAPS = [([0, 5, 3, 8], 8, [0]),
            ([0, 8, 2, 6, 8], 8, [0]),
            ([0, 4, 2, 8, 12], 12, [0, 3]),
            ([0, 3, 1, 6, 4, 8, 9], 9, [0, 5]),
            ([5, 12, 0, 12, 12, 16], 16, [0, 4])]


@pytest.mark.parametrize("qo,T,valid", OVERLAPS)
@pytest.mark.parametrize("context", [100, 9000])
@pytest.mark.parametrize("block", [0, 16])
def test_ranges_that_begin_before_an_earlier_end(qo, T, valid, context, block):
    """Of two requests that would have the same rows the first has them."""
    c, q, seen, mask = batch(qo, T, valid, context, 2, 64, block, 70 + T)
    out, ws = tree(c, q.cuda(), 0.05, mask)
    assert api.pa_get_error(ws) == api.DEVERR_LEN
    check(c, q, out, 0.05, seen, f"starts {qo}", reqs=valid)
    assert torch.isnan(others(out, qo, valid).float()).all()


def test_the_same_range_many_times():
    """Starts that go back again and again: the first request has the rows, whatever the number of the others."""
    c, q, seen, mask = batch([0, 4], 4, [0], 5000, 2, 64, 0, 80)
    want, _ = tree(c, q.cuda(), 0.05, mask)
    k, v, table, rws, _, _ = c.dev
    R = 4095
    qo = torch.tensor([0, 4], dtype=torch.int32, device="cuda").repeat((R + 1) // 2)
    ws = api.alloc_workspace(api.pa_tree_workspace_bytes(8, 2, 64))
    out = torch.zeros_like(want)
    api.pa_paged_tree_attn(q.cuda(), k, v, 0, qo, table, rws.repeat(R), c.dlens.repeat(R), 0.05, ws, out, tree_mask=mask)
    assert api.pa_get_error(ws) == api.DEVERR_LEN
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("block", [0, 16])
def test_rows_that_see_nothing_whatever_their_query(what, D, block):
    """A row that sees nothing is zeros, its query a NaN or not; one that sees something is NaN then, and the other
    rows are what they are."""
    c = make([0, 0, 300], [4, 140, 5], 2, D, 16, block, 62)
    seen = [torch.eye(4, dtype=torch.bool), S.chain_seen(140), S.chain_seen(5)]
    seen[0][1] = False                         # blind rows: 1, and 4 + 130 in the second tile of its piece
    seen[1][130] = False
    mask = pack(seen)
    q = queries(c, 4, D)
    rows = [1, 4 + 130, 2, 4 + 7, 4 + 140 + 3]
    q[rows, :, 3] = what
    out, ws = tree(c, q.cuda(), 0.05, mask)
    assert api.pa_get_error(ws) == 0
    out = out.cpu()
    assert torch.count_nonzero(out[rows[:2]]) == 0
    if block or math.isnan(what):
        assert torch.isnan(out[rows[2:]].float()).all()
    good, clean = [t for t in range(c.qo[-1]) if t not in rows], q.clone()
    clean[rows] = 1.0
    base, _ = tree(c, clean.cuda(), 0.05, mask)
    assert torch.equal(out[good].view(torch.int16), base.cpu()[good].view(torch.int16))
    check(c, clean, base, 0.05, seen, f"D={D} block={block}")


@pytest.mark.parametrize("move", [False, True])
@pytest.mark.parametrize("length", [-5, 10 ** 6, 0, 7])
def test_accept_requests_without_nodes(move, length):
    """A request without nodes pads a batch whatever its length and row, as in the attention."""
    b = Batch([30, 0, 9], [20, 0, 4], 63)
    b.lens[1] = length
    b.rows[1] = 77
    kv = {}
    if move:
        k = torch.zeros((1, b.size, 1, 64), dtype=torch.bfloat16, device="cuda")
        kv = dict(k=k, v=k.clone())
    err = i32([0])
    table, lens, freed = b.call(err=err, **kv)
    assert api.pa_get_error_word(err) == 0
    b.rows[1] = b.rows[0]                      # (nobody's)
    b.lens[1] = max(0, min(length, b.table.shape[1]))
    t, l, f, _ = b.want(move=move, skip={1})
    assert torch.equal(table, t) and lens == l and freed == f


@pytest.mark.parametrize("move", [False, True])
def test_accept_ranges_that_begin_before_an_earlier_end(move):
    """Two requests with the same entries of the list of free slots: the first has them, the other one is left as it is."""
    b = Batch([30, 5, 9, 12], [6, 1, 7, 3], 64)
    b.qo = [0, 6, 2, 9, 12]
    k = torch.randn((2, b.size, 2, 64), generator=b.g).to(torch.bfloat16)
    kv = dict(k=k.cuda(), v=k.flip(0).contiguous().cuda()) if move else {}
    err = i32([0])
    table, lens, freed = b.call(err=err, **kv)
    # (request 1, from 6 to 2, has a path of one node, which is longer than its range)
    assert api.pa_get_error_word(err) == api.DEVERR_LEN | api.DEVERR_TREE
    t, l, f, moves = b.want(move=move, skip={1, 2})
    assert torch.equal(table, t) and lens == l and freed == f
    if move:
        now = k.clone()
        for src, dst in moves:
            now[:, dst] = k[:, src]
        assert torch.equal(kv["k"].cpu(), now) and torch.equal(kv["v"].cpu(), now.flip(0))


def test_more_kv_heads_than_sms_set_no_error():
    """One range per kv head, several heads to a CTA, no merge: the error word stays 0, every row of every head is written."""
    c = make([300, 0, 40], [5, 1, 140], 200, 64, 16, 0, 65, layers=1, layer=0)
    seen = [S.chain_seen(n) for n in c.nodes]
    q = queries(c, 1, 64)
    out, ws = tree(c, q.cuda(), 0.1, None)
    assert api.pa_get_error(ws) == 0
    check(c, q, out, 0.1, seen, "200 kv heads")
