"""Speculative steps whose calls overlap on the stream: each reads what the one before wrote."""
import pytest
import torch

from paged_kv_cache_188_gb300 import api
from test_gpu_verify_accept import Batch, Drafts, i32
from test_gpu_verify_accept import test_speculative_steps as _steps

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.lib()
    yield
    api.pa_set_launch_overlap(api.OVERLAP_OFF)


@pytest.mark.parametrize("mode", [api.OVERLAP_SAFE, api.OVERLAP_EARLY_METADATA, api.OVERLAP_EARLY_KV])
@pytest.mark.parametrize("block,move", [(0, False), (0, True), (16, False)])
@pytest.mark.parametrize("graph", [False, True])
def test_steps_in_every_mode(mode, block, move, graph):
    api.pa_set_launch_overlap(mode)
    _steps(block, move, graph)


@pytest.mark.parametrize("move", [False, True])
def test_acceptance_behind_verification_and_itself(move):
    """Verification and acceptance in one graph, replayed with other random numbers: the path and its length are
    this replay's; then the lengths in place, one acceptance behind the other."""
    api.pa_set_launch_overlap(api.OVERLAP_SAFE)
    nodes, context, V = [9, 16, 5, 0, 12], [70, 200, 15, 30, 0], 501
    d, b = Drafts(nodes, V, 91), Batch(context, nodes, 92)
    args = [d.p.cuda(), i32(d.tokens), i32(d.parents), i32(d.qo), d.u.cuda(), d.ul.cuda()]
    R, f = len(nodes), d.f.cuda()
    acc, n, nxt = torch.full((R, 16), -7, dtype=torch.int32, device="cuda"), i32([0] * R), i32([0] * R)
    table, lens, rows, qo = b.table.cuda(), i32(b.lens), b.rows.cuda(), i32(b.qo)
    new, freed, err = i32([0] * R), torch.full((b.qo[-1],), -7, dtype=torch.int32, device="cuda"), i32([0])
    k = torch.randn((2, b.size, 2, 64), generator=b.g).to(torch.bfloat16)
    dk, dv = k.cuda(), k.flip(0).contiguous().cuda()
    kv = dict(k_buf=dk, v_buf=dv) if move else {}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.pa_tree_verify(*args, acc, n, nxt, draft_probs=f, error_word=err)
        api.pa_kv_accept(table, rows, lens, qo, acc, n, new, freed, error_word=err, **kv)
    g = torch.Generator().manual_seed(93)
    for _ in range(4):
        d.u, d.ul = torch.rand(d.u.shape, generator=g), torch.rand(d.ul.shape, generator=g)
        args[4].copy_(d.u)
        args[5].copy_(d.ul)
        table.copy_(b.table)
        dk.copy_(k)
        dv.copy_(k.flip(0))
        freed.fill_(-7)
        graph.replay()
        assert api.pa_get_error_word(err) == 0
        d.check((acc, n, nxt), "replay")
        b.paths = [p[:m] for p, m in zip(acc.tolist(), n.tolist())]
        t, l, fr, moves = b.want(move=move)
        assert torch.equal(table.cpu(), t) and new.tolist() == l and freed.tolist() == fr
        if move:
            now = k.clone()
            for src, dst in moves:
                now[:, dst] = k[:, src]
            assert torch.equal(dk.cpu(), now) and torch.equal(dv.cpu(), now.flip(0))
    if move:
        return
    # twice in a row on the lengths themselves: the second keeps the roots of what the first left
    table.copy_(b.table)
    paths = [list(range(m)) for m in nodes]                    # everything, then one node each
    count, one = i32(nodes), i32([min(m, 1) for m in nodes])
    acc.copy_(i32([p + [-1] * (16 - len(p)) for p in paths]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.pa_kv_accept(table, rows, lens, qo, acc, count, lens, freed, error_word=err)
        api.pa_kv_accept(table, rows, lens, qo, acc, one, lens, freed, error_word=err)
    graph.replay()
    assert api.pa_get_error_word(err) == 0 and torch.equal(table.cpu(), b.table)
    assert lens.tolist() == [c + min(m, 1) for c, m in zip(context, nodes)]
