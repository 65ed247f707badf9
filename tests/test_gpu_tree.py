"""Attention of drafted tokens on the GPU against a plain 64-bit reference."""
import math

import numpy as np
import pytest
import torch

import _block_ref as R
import _spec_ref as S
from paged_kv_cache_188_gb300 import api
from test_gpu_fp8_block import Cache
from test_gpu_weights_evict import Bf16Cache

pytestmark = pytest.mark.gpu
P_BITS = 8      # the weights enter the second product in bf16: off by at most 2^-8, relative
# over an e4m3 cache q, scaled so that its row's largest element lies in (224, 448], is a sum of two e4m3 terms.  A bf16
# number y of exponent e has 8 significant bits, the first term leaves a multiple of 2^(e - 7) of at most 2^(e - 4), which
# the second holds where e >= -2; below, its steps of 2^-9 leave at most 2^-10 out: 2^-10 / 224 < 2^-17 of the largest
TERMS = 2.0 ** -17


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.lib()


def make(context, nodes, Hkv, D, page, block, seed, **kw):
    lens = [a + b for a, b in zip(context, nodes)]
    c = Cache(lens, Hkv, D, page, block, seed, **kw) if block else Bf16Cache(lens, Hkv, D, page, seed, **kw)
    c.nodes = list(nodes)
    c.qo = [0]
    for n in nodes:
        c.qo.append(c.qo[-1] + n)
    return c.cuda()


def trees(c, chain=False):
    """(seen matrices, mask on the GPU or None)."""
    if chain:
        return [S.chain_seen(n) for n in c.nodes], None
    seen = [S.tree_seen(S.random_parents(n, c.g)) for n in c.nodes]
    return seen, pack(seen)


def pack(seen):
    words = max(1, -(-max(len(s) for s in seen) // 32))
    return torch.cat([S.mask_words(s, words) for s in seen]).cuda()


def queries(c, G, D):
    return torch.randn((c.qo[-1], G * c.k.shape[2], D), generator=c.g).to(torch.bfloat16)


def tree(c, q, scale, mask, ws=None, out=None, **kw):
    k, v, table, rws, ke, ve = c.dev
    if ws is None:
        ws = api.alloc_workspace(api.pa_tree_workspace_bytes(q.shape[1], k.shape[2], q.shape[2]))
    out = torch.full_like(q, math.nan) if out is None else out
    qo = torch.tensor(c.qo, dtype=torch.int32, device="cuda")
    more = dict(k_exp=ke, v_exp=ve, block=c.block) if c.block else {}
    api.pa_paged_tree_attn(q, k, v, c.layer, qo, table, rws, c.dlens, scale, ws, out, tree_mask=mask, **more, **kw)
    return out, ws


def check(c, q, out, scale, seen, what, reqs=None):
    for r in (range(len(c.nodes)) if reqs is None else reqs):
        lo, hi = c.qo[r], c.qo[r + 1]
        if lo == hi:
            continue
        k, v = c.values(r)
        ref = S.attention(q[lo:hi].double(), k, v, scale, seen[r], terms=TERMS if c.block else 0.0)
        R.check_out(out[lo:hi].cpu(), ref, P_BITS, f"{what}, request {r}: {hi - lo} of {len(k)}")


CONTEXT = [1, 120, 128, 250, 0, 1000, 0, 300, 127]
NODES = [1, 8, 3, 33, 5, 16, 0, 64, 2]


@pytest.mark.parametrize("G,Hkv", [(4, 2), (1, 3), (8, 1), (16, 1), (3, 2), (7, 1)])
@pytest.mark.parametrize("D,page", [(128, 16), (64, 16), (128, 1), (64, 1)])
@pytest.mark.parametrize("chain", [False, True])
def test_bf16(G, Hkv, D, page, chain):
    c = make(CONTEXT, NODES, Hkv, D, page, 0, G + 10 * D + page)
    seen, mask = trees(c, chain)
    q = queries(c, G, D)
    out, ws = tree(c, q.cuda(), 0.1, mask)
    assert api.pa_get_error(ws) == 0
    check(c, q, out, 0.1, seen, f"bf16 G={G} D={D} page={page}")


@pytest.mark.parametrize("G,Hkv", [(4, 2), (1, 3), (8, 1), (16, 1), (5, 2)])
@pytest.mark.parametrize("D,page,block", [(128, 16, 16), (64, 1, 1), (128, 32, 8), (64, 128, 128), (128, 1, 1)])
def test_fp8_block(G, Hkv, D, page, block):
    c = make(CONTEXT, NODES, Hkv, D, page, block, G + D + page)
    seen, mask = trees(c)
    q = queries(c, G, D)
    out, ws = tree(c, q.cuda(), 0.05, mask)
    assert api.pa_get_error(ws) == 0
    check(c, q, out, 0.05, seen, f"e4m3 G={G} D={D} page={page} block={block}")


@pytest.mark.parametrize("n", [1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 300])
@pytest.mark.parametrize("block", [0, 16])
def test_nodes_around_tile_edges(n, block):
    """Trees of n nodes behind contexts that put them around the edges of a tile of 128 tokens."""
    context = [0, 1, 127, 128 - min(n, 128), 129, 255]
    c = make(context, [n] * 6, 1, 64, 16, block, n)
    seen, mask = trees(c)
    q = queries(c, 4, 64)
    out, ws = tree(c, q.cuda(), 0.1 if not block else 0.02, mask)
    assert api.pa_get_error(ws) == 0
    check(c, q, out, 0.1 if not block else 0.02, seen, f"{n} nodes")


@pytest.mark.parametrize("block", [0, 16])
def test_long_contexts_over_many_ctas(block):
    c = make([20000, 3, 5000], [40, 7, 64], 2, 128, 16, block, 3, layers=1, layer=0)
    seen, mask = trees(c)
    q = queries(c, 4, 128)
    out, ws = tree(c, q.cuda(), 0.05, mask)
    assert api.pa_get_error(ws) == 0
    check(c, q, out, 0.05, seen, "long")
    again, _ = tree(c, q.cuda(), 0.05, mask)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))      # run to run


def test_many_requests_and_heads():
    """More requests and kv heads than SMs share evenly."""
    g = torch.Generator().manual_seed(9)
    context = torch.randint(0, 400, (170,), generator=g).tolist()
    nodes = torch.randint(0, 6, (170,), generator=g).tolist()
    for Hkv, G in ((1, 8), (7, 2), (40, 1)):
        c = make(context, nodes, Hkv, 64, 16, 0, Hkv, layers=1, layer=0)
        seen, mask = trees(c)
        q = queries(c, G, 64)
        out, ws = tree(c, q.cuda(), 0.1, mask)
        assert api.pa_get_error(ws) == 0
        check(c, q, out, 0.1, seen, f"Hkv={Hkv}", reqs=range(0, 170, 7))


def test_more_kv_heads_than_sms():
    c = make([300, 40], [5, 2], 200, 64, 16, 0, 4, layers=1, layer=0)
    seen, mask = trees(c)
    q = queries(c, 1, 64)
    out, _ = tree(c, q.cuda(), 0.1, mask)
    check(c, q, out, 0.1, seen, "200 kv heads")


@pytest.mark.parametrize("block", [0, 16])
def test_rows_that_see_nothing_and_partial_masks(block):
    """Masks without a node's own bit; without a context a row that sees nothing is zeros.  Bits past the nodes are
    not looked at."""
    c = make([0, 100, 0], [4, 40, 130], 2, 128, 16, block, 8)
    seen = [torch.zeros((4, 4), dtype=torch.bool), torch.zeros((40, 40), dtype=torch.bool), S.chain_seen(130)]
    seen[0][1, 3] = True                       # a node may see a later one
    seen[1][5, 39] = True
    seen[2][128] = False
    mask = pack(seen)
    mask[0:4, 0] |= ~0xF                       # bits 4 .. 31 of requests of 4 nodes
    mask[0:4, 1:] = -1
    q = queries(c, 4, 128)
    out, ws = tree(c, q.cuda(), 0.05, mask)
    assert api.pa_get_error(ws) == 0
    check(c, q, out, 0.05, seen, "partial masks")
    assert torch.count_nonzero(out[0]) == 0 and torch.count_nonzero(out[2:4]) == 0 and torch.count_nonzero(out[44 + 128]) == 0
    k, v = c.values(0)
    assert torch.equal(out[1, 0].cpu(), v[3, 0].to(torch.bfloat16))        # one row seen: that row


@pytest.mark.parametrize("block", [0, 16])
@pytest.mark.parametrize("what", ["nan", "inf"])
@pytest.mark.parametrize("operand", ["k", "v"])
def test_hidden_rows_may_hold_anything(block, what, operand):
    """NaN and infinities in a node's K or V reach the nodes that see it, and no other."""
    if block and what == "inf":
        pytest.skip("an e4m3 cache holds no infinity")
    c = make([100, 0, 128], [20, 20, 140], 2, 64, 16, block, 11)
    seen, mask = trees(c)
    bad = [7, 3, 131]
    for r, b in enumerate(bad):
        s = c.slots[r][c.lens[r] - c.nodes[r] + b]
        buf = getattr(c, operand)
        if block:
            buf[c.layer, s, 0, 5] = 127
        else:
            buf[c.layer, s, 0, 5] = math.nan if what == "nan" else math.inf
    c.cuda()
    q = queries(c, 4, 64)
    out, _ = tree(c, q.cuda(), 0.05, mask)
    out = out.cpu()
    for r, b in enumerate(bad):
        lo = c.qo[r]
        k, v = c.values(r)
        blind = [i for i in range(c.nodes[r]) if not seen[r][i, b]]
        ref = S.attention(q[lo:c.qo[r + 1]].double(), k.nan_to_num(1.0, 1.0), v.nan_to_num(1.0, 1.0), 0.05, seen[r],
                          terms=TERMS if block else 0.0)
        part = {x: (y[blind] if torch.is_tensor(y) and y.dim() > 1 else y) for x, y in ref.items()}
        R.check_out(out[lo:c.qo[r + 1]][blind], part, P_BITS, f"{what} in {operand}")
        for i in range(c.nodes[r]):
            if not seen[r][i, b]:
                continue
            first, other = out[lo + i, :4].double(), out[lo + i, 4:].double()
            assert torch.isfinite(other).all()                              # the other kv head
            if operand == "v":
                bad_col = first[:, 5]
                assert not torch.isfinite(bad_col).any()
                assert torch.isfinite(torch.cat([first[:, :5], first[:, 6:]], 1)).all()
            elif what == "nan":
                assert torch.isnan(first).all()


def test_scores_of_minus_infinity_and_large_scores():
    c = make([200, 10], [6, 3], 1, 64, 16, 0, 12)
    for r in range(2):
        c.k[c.layer, c.slots[r], 0] *= 40                                  # scores of hundreds
    c.cuda()
    seen, mask = trees(c)
    q = queries(c, 8, 64)
    out, _ = tree(c, q.cuda(), 1.0, mask)
    check(c, q, out, 1.0, seen, "large scores")
    for r in range(2):
        c.k[c.layer, c.slots[r], 0] = 0
        c.k[c.layer, c.slots[r], 0, 0] = -math.inf
    c.cuda()
    q[..., 0] = 1.0
    out, _ = tree(c, q.cuda(), 1.0, mask)
    assert torch.count_nonzero(out) == 0


@pytest.mark.parametrize("scale", [0.0, -0.1])
def test_scale_of_zero_and_below(scale):
    c = make([300, 10], [6, 3], 2, 128, 16, 0, 13)
    seen, mask = trees(c)
    q = queries(c, 4, 128)
    out, _ = tree(c, q.cuda(), scale, mask)
    check(c, q, out, scale, seen, f"scale {scale}")


@pytest.mark.parametrize("block", [0, 16])
def test_bad_requests_and_slots(block):
    """What is out of range is flagged and masked, the other requests are right, rows behind the last request stay."""
    c = make([100, 100, 100, 100], [4, 4, 4, 4], 2, 64, 16, block, 14)
    seen, mask = trees(c)
    q = torch.cat([queries(c, 4, 64), torch.zeros((3, 8, 64)).to(torch.bfloat16)])
    mask = torch.cat([mask, mask[:3]])
    base, _ = tree(c, q.cuda(), 0.05, mask)
    assert torch.isnan(base[16:].float()).all()                            # rows of no request
    c.dev[3][1] = 1000                                                     # a row of the table that is not there
    out, ws = tree(c, q.cuda(), 0.05, mask)
    assert api.pa_get_error(ws) == api.DEVERR_ROW and torch.count_nonzero(out[4:8]) == 0
    assert torch.equal(out[:4].view(torch.int16), base[:4].view(torch.int16))
    c.dev[3][1] = int(c.rows[1])
    for bad in (-1, 3, 10 ** 6):                                           # fewer tokens than nodes, more than the table
        c.dlens[1] = bad
        out, ws = tree(c, q.cuda(), 0.05, mask)
        assert api.pa_get_error(ws) == api.DEVERR_LEN and torch.count_nonzero(out[4:8]) == 0
        assert torch.equal(out[8:16].view(torch.int16), base[8:16].view(torch.int16))
    c.dlens[1] = 104
    for bad in (-1, c.size, 2 ** 31 - 1):
        for at in (50, 102):                                               # in the context, a node
            table = c.dev[2].clone()
            row = int(c.rows[1])
            was = int(table[row, at])
            c.dev[2][row, at] = bad
            out, ws = tree(c, q.cuda(), 0.05, mask)
            c.dev[2][row, at] = was
            assert api.pa_get_error(ws) == api.DEVERR_SLOT
            k, v = c.values(1)
            keep = [j for j in range(104) if j != at]
            s2 = seen[1].clone()
            for i in range(4):
                vis = torch.cat([torch.ones(100, dtype=torch.bool), s2[i]])
                vis[at] = False
                j = vis.nonzero()[:, 0]
                ref = S.attention(q[4 + i:5 + i].double(), k[j], v[j], 0.05, torch.ones((1, 1), dtype=torch.bool),
                                  terms=TERMS if block else 0.0)
                R.check_out(out[4 + i:5 + i].cpu(), ref, P_BITS, f"slot {bad} at {at}")
            assert len(keep) == 103
    qo = c.qo
    for bad in ([0, 4, 3, 12, 16], [0, 4, 8, 12, 20], [-4, 4, 8, 12, 16]):
        c.qo = bad
        _, ws = tree(c, q.cuda(), 0.05, mask)
        assert api.pa_get_error(ws) & api.DEVERR_LEN
    c.qo = qo


def test_more_nodes_than_the_mask_has_bits():
    c = make([10, 10], [40, 4], 1, 64, 16, 0, 15)
    seen, mask = trees(c)
    q = queries(c, 4, 64)
    out, ws = tree(c, q.cuda(), 0.1, mask[:, :1].contiguous())
    assert api.pa_get_error(ws) == api.DEVERR_LEN and torch.count_nonzero(out[:40]) == 0
    check(c, q, out, 0.1, seen, "the other request", reqs=[1])


def test_empty_calls_and_padded_batches():
    c = make([10], [4], 1, 64, 16, 0, 16)
    _, mask = trees(c)
    q = queries(c, 4, 64)
    out, ws = tree(c, q.cuda(), 0.1, mask)
    # a batch padded with requests without nodes, whose rows are nothing
    k, v, table, rws, _, _ = c.dev
    qo = torch.tensor([0, 4, 4, 4], dtype=torch.int32, device="cuda")
    rows = torch.cat([rws, torch.tensor([-1, 77], dtype=torch.int32, device="cuda")])
    lens = torch.tensor([14, 0, -5], dtype=torch.int32, device="cuda")
    got = torch.full_like(out, math.nan)
    api.pa_paged_tree_attn(q.cuda(), k, v, c.layer, qo, table, rows, lens, 0.1, ws, got, tree_mask=mask)
    assert api.pa_get_error(ws) == 0 and torch.equal(out.view(torch.int16), got.view(torch.int16))
    api.pa_paged_tree_attn(q[:0].cuda(), k, v, c.layer, qo[:1], table, rows[:0], lens[:0], 0.1, ws, got[:0])


@pytest.mark.parametrize("block", [0, 16])
def test_graphs_streams_and_overlap(block):
    """Captured and replayed in every overlap mode with the lengths and masks of each replay, on a stream of its own;
    two graphs share a workspace."""
    c = make([700, 90], [12, 5], 2, 64, 16, block, 17, layers=1, layer=0)
    seen, mask = trees(c)
    q = queries(c, 4, 64)
    want, ws = tree(c, q.cuda(), 0.05, mask)
    check(c, q, want, 0.05, seen, "first")
    dq, out = q.cuda(), torch.empty_like(want)
    k, v, table, rws, ke, ve = c.dev
    qo = torch.tensor(c.qo, dtype=torch.int32, device="cuda")
    more = dict(k_exp=ke, v_exp=ve, block=c.block) if block else {}
    call = lambda: api.pa_paged_tree_attn(dq, k, v, 0, qo, table, rws, c.dlens, 0.05, ws, out, tree_mask=mask, **more)  # noqa: E731
    try:
        graphs = []
        for mode in (api.OVERLAP_OFF, api.OVERLAP_SAFE, api.OVERLAP_EARLY_METADATA, api.OVERLAP_EARLY_KV):
            api.pa_set_launch_overlap(mode)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                call()
                call()
            graphs.append(g)
        for g in graphs + graphs:
            out.fill_(math.nan)
            g.replay()
            assert torch.equal(out.view(torch.int16), want.view(torch.int16))
        short = [60, 20]
        c.dlens.copy_(torch.tensor(short, dtype=torch.int32))
        for g in graphs:
            g.replay()
        for r in range(2):
            c.slots[r] = c.slots[r][:short[r]]
        check(c, q, out, 0.05, seen, "other lengths")
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        other = torch.full_like(out, math.nan)
        api.pa_paged_tree_attn(dq, k, v, 0, qo, table, rws, c.dlens, 0.05, ws, other, tree_mask=mask, stream=st, **more)
        st.synchronize()
        assert torch.equal(out.view(torch.int16), other.view(torch.int16))
    finally:
        api.pa_set_launch_overlap(api.OVERLAP_OFF)


def test_a_chain_is_what_prefill_computes():
    """No mask: the causal prefill's results, within both calls' roundings of the weights and of the result."""
    c = make([500, 33], [9, 4], 2, 128, 16, 0, 18)
    q = queries(c, 4, 128).cuda()
    out, _ = tree(c, q, 0.08, None)
    k, v, table, rws, _, _ = c.dev
    ws = api.alloc_workspace(api.pa_prefill_workspace_bytes())
    qo = torch.tensor(c.qo, dtype=torch.int32, device="cuda")
    kv = torch.tensor([0, 509, 546], dtype=torch.int32, device="cuda")
    pre = torch.empty_like(out)
    api.pa_paged_prefill_attn(q, k, v, c.layer, qo, kv, table, rws, 0.08, ws, pre)
    for r in range(2):
        kk, vv = c.values(r)
        ref = S.attention(q[c.qo[r]:c.qo[r + 1]].double().cpu(), kk, vv, 0.08, S.chain_seen(c.nodes[r]))
        gap = (out - pre)[c.qo[r]:c.qo[r + 1]].double().cpu().abs()
        assert (gap <= 2 * (2.0 ** -8 * ref["out"].abs() + 1.05 * 2.0 ** -8 * ref["mean"]) + 1e-6).all()


def test_refusals_of_the_wrapper():
    c = make([10], [4], 1, 64, 16, 0, 19)
    _, mask = trees(c)
    q = queries(c, 4, 64).cuda()
    k, v, table, rws, _, _ = c.dev
    qo = torch.tensor(c.qo, dtype=torch.int32, device="cuda")
    ws = api.alloc_workspace(api.pa_tree_workspace_bytes(4, 1, 64))
    good = dict(q=q, k_buf=k, v_buf=v, layer_id=0, qo_indptr=qo, req_to_token=table, req_pool_indices=rws, seq_lens=c.dlens,
                scale=0.1, workspace=ws, out=torch.empty_like(q), tree_mask=mask)
    for bad, err in ((dict(q=q.float()), TypeError), (dict(tree_mask=mask[:2]), ValueError), (dict(qo_indptr=qo[:1]), ValueError),
                     (dict(out=q[:2]), ValueError), (dict(tree_mask=mask.long()), TypeError), (dict(q=q.cpu()), TypeError),
                     (dict(seq_lens=c.dlens.repeat(2)), ValueError), (dict(workspace=ws[:128]), api.PaError),
                     (dict(layer_id=9), api.PaError), (dict(q=q.transpose(0, 1)), ValueError)):
        with pytest.raises(err):
            api.pa_paged_tree_attn(**dict(good, **bad))
    assert np.isfinite(api.pa_get_error(ws))
