"""Verification of drafted tokens and acceptance of their path on the GPU against
plain references, equal in every number; then speculative steps end to end."""
import math

import numpy as np
import pytest
import torch

import _spec_ref as S
from paged_kv_cache_188_gb300 import api
from test_gpu_tree import check, make, pack, queries, tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.lib()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def gen(seed):
    return torch.Generator().manual_seed(seed)


class Drafts:
    """Probabilities, tokens (drawn from the draft's, so that many are kept) and random numbers of a batch."""

    def __init__(self, nodes, V, seed, chain=False, drawn=True, sharp=2.0):
        g = gen(seed)
        self.nodes, T = nodes, sum(nodes)
        self.qo = [0]
        for n in nodes:
            self.qo.append(self.qo[-1] + n)
        logits = sharp * torch.randn((T, V), generator=g, dtype=torch.float64)
        self.p = torch.softmax(logits, -1).float()
        f = torch.softmax(logits + 0.7 * torch.randn((T, V), generator=g, dtype=torch.float64), -1).float()
        self.parents = [a for n in nodes for a in S.random_parents(n, g, chain)]
        at = []
        for r, n in enumerate(nodes):
            at += [self.qo[r] + max(a, 0) for a in self.parents[self.qo[r]:self.qo[r + 1]]]
        self.tokens = torch.multinomial(f[at], 1, generator=g)[:, 0].tolist() if T else []
        self.f = f if drawn else None
        self.u, self.ul = torch.rand(T, generator=g), torch.rand(len(nodes), generator=g)

    def call(self, max_path=None, err=None, **kw):
        R = len(self.nodes)
        max_path = max(self.nodes + [1]) if max_path is None else max_path
        out = (torch.full((R, max_path), -7, dtype=torch.int32, device="cuda"), i32([-7] * R), i32([-7] * R))
        api.pa_tree_verify(self.p.cuda(), i32(self.tokens), i32(self.parents), i32(self.qo), self.u.cuda(), self.ul.cuda(),
                           *out, draft_probs=None if self.f is None else self.f.cuda(), error_word=err, **kw)
        return out

    def check(self, out, what):
        accepted, count, after = (x.cpu().tolist() for x in out)
        p, f = self.p.numpy(), None if self.f is None else self.f.numpy()
        kept = 0
        for r, n in enumerate(self.nodes):
            lo, hi = self.qo[r], self.qo[r + 1]
            if n == 0:
                assert count[r] == 0 and after[r] == -1 and set(accepted[r]) == {-1}
                continue
            path, v = S.verify(p[lo:hi], None if f is None else f[lo:hi], self.tokens[lo:hi], self.parents[lo:hi],
                               self.u[lo:hi].numpy(), self.ul[r].numpy(), len(accepted[r]))
            assert count[r] == len(path) and accepted[r] == path + [-1] * (len(accepted[r]) - len(path)), f"{what}, {r}"
            assert after[r] == v, f"{what}, request {r}: token {after[r]}, not {v}"
            kept += len(path) - 1
        return kept


@pytest.mark.parametrize("V", [1, 2, 3, 5, 31, 128, 1000, 4096, 4097, 20011, 50001])
@pytest.mark.parametrize("drawn,chain", [(True, True), (True, False), (False, True), (False, False)])
def test_verify(V, drawn, chain):
    d = Drafts([6, 1, 2, 0, 9, 17], V, V + 2 * drawn + chain, chain, drawn)
    err = i32([0])
    out = d.call(err=err)
    assert api.pa_get_error_word(err) == 0
    d.check(out, f"V={V}")


def test_verify_keeps_and_refuses():
    """The inputs reach what they are meant to: nodes kept and refused, siblings behind a refusal kept."""
    kept = total = second = 0
    for seed in range(12):
        for drawn in (True, False):
            d = Drafts([12] * 8, 40, seed, False, drawn, sharp=1.0)
            out = d.call()
            kept += d.check(out, f"seed {seed}")
            total += 8 * 11
            for r, path in enumerate(out[0].cpu().tolist()):
                for a, b in zip(path, path[1:]):
                    second += b > 0 and b != min(i for i in range(12) if d.parents[12 * r + i] == a and i > 0)
    assert 0.05 * total < kept < 0.95 * total and second > 10


def test_verify_max_path():
    d = Drafts([8] * 6, 300, 5, True, True)
    d.u.zero_()                                        # everything that can be is kept
    for m in (1, 2, 5, 8, 20):
        d.check(d.call(max_path=m), f"max_path {m}")


def test_verify_many_nodes_and_requests():
    d = Drafts([1024, 1000, 33], 64, 6, False, True, sharp=0.3)
    d.check(d.call(), "1024 nodes")
    d = Drafts([2] * 700, 257, 7, True, True)
    d.check(d.call(), "700 requests")
    star = Drafts([200], 500, 8, False, True, sharp=0.1)
    star.parents = [-1] + [0] * 199                    # 199 siblings, most of them refused
    star.u.fill_(0.999)
    star.check(star.call(), "siblings")
    star.f = None
    star.check(star.call(), "chosen siblings")


def test_verify_edges():
    """u = 0, u next to 1, zero and one-hot rows, the draft equal to the target, equal siblings."""
    V = 37
    top = float(np.nextafter(np.float32(1), np.float32(0)))
    for u in (0.0, 0.5, top):
        for drawn in (True, False):
            d = Drafts([5, 5, 5, 5, 5], V, 9, False, drawn)
            d.u.fill_(u)
            d.ul.fill_(u)
            d.p[5:10] = 0                              # no mass
            d.p[10:15] = torch.eye(V)[:5]              # one-hot
            d.tokens[15:20] = [3, 3, 3, 3, 3]          # equal siblings
            d.parents[15:20] = [-1, 0, 0, 0, 0]
            if drawn:
                d.f[20:25] = d.p[20:25]                # draft and target alike
                d.f[0:5] = 0
            d.check(d.call(), f"u {u}")
            assert int(d.call()[2][1]) == -1
    d = Drafts([4], V, 10, True, True)
    d.p[0] = 0.25
    d.f[0] = 1.0                                       # nothing of the target is left behind a refusal: its row is drawn from
    d.u.fill_(0.99)
    out = d.call()
    d.check(out, "nothing left")
    assert out[1].item() == 1 and out[2].item() >= 0


def test_verify_rows_that_are_not_probabilities():
    """NaN and negative entries count as 0; every second entry."""
    V = 1003
    d = Drafts([5, 5], V, 11, False, True)
    d.p[:, ::2] = math.nan
    d.f[:, 1::4] = -1.0
    d.p[3] = -0.5
    d.check(d.call(), "NaN")
    d.f = None
    d.check(d.call(), "NaN, chosen")
    d.p.fill_(math.nan)
    assert d.call()[2].tolist() == [-1, -1]


def test_verify_u_finer_than_24_bits():
    V = 20000
    d = Drafts([1] * 6, V, 12)
    d.ul = torch.tensor([2.0 ** -40, 2.0 ** -33 * 3, 1e-7, 2.0 ** -24, 0.1, 1 / 3])
    d.check(d.call(), "fine u")


def test_verify_bad_inputs():
    d = Drafts([4, 4, 4], 50, 13, True, True)
    d.u.zero_()
    ref = [x.clone() for x in d.call()]
    for field, at, bad in (("tokens", 5, 50), ("tokens", 5, -1), ("parents", 6, 2), ("parents", 6, -1), ("parents", 6, 9),
                           ("tokens", 7, 2 ** 31 - 1)):
        was = getattr(d, field)[at]
        getattr(d, field)[at] = bad
        err = i32([0])
        out = d.call(err=err)
        assert api.pa_get_error_word(err) == api.DEVERR_TREE, (field, bad)
        for x, y in zip(out, ref):
            assert torch.equal(x[::2], y[::2])         # the other requests
        if field == "tokens" or bad != -1:
            d.parents[at] = d.parents[at] if field == "tokens" else 99
            d.check(out, f"{field} {bad}")
        getattr(d, field)[at] = was
    d.parents[4] = 12345                               # the root's is not looked at
    err = i32([0])
    d.call(err=err)
    assert api.pa_get_error_word(err) == 0
    d.qo = [0, 4, 3, 12]                               # (the third request's nodes are then others, parents and all)
    d.call(err=err)
    assert api.pa_get_error_word(err) & api.DEVERR_LEN
    d.qo = [0, 4, 8, 13]                               # past the last row
    err.zero_()
    out = d.call(err=err)
    assert api.pa_get_error_word(err) == api.DEVERR_LEN and out[1].tolist()[2] == 0 and out[2].tolist()[2] == -1
    long = Drafts([1025, 3], 5, 14)
    err.zero_()
    out = long.call(err=err)
    assert api.pa_get_error_word(err) == api.DEVERR_LEN and out[1].tolist()[0] == 0 and set(out[0][0].tolist()) == {-1}


def test_verify_graph_overlap_and_streams():
    d = Drafts([6, 3, 9], 5000, 15)
    want = d.call()
    d.check(want, "first")
    args = [d.p.cuda(), i32(d.tokens), i32(d.parents), i32(d.qo), d.u.cuda(), d.ul.cuda()]
    f, out = d.f.cuda(), [torch.empty_like(x) for x in want]
    try:
        for mode in (api.OVERLAP_OFF, api.OVERLAP_SAFE, api.OVERLAP_EARLY_METADATA, api.OVERLAP_EARLY_KV):
            api.pa_set_launch_overlap(mode)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                api.pa_tree_verify(*args, *out, draft_probs=f)
                api.pa_tree_verify(*args, *out, draft_probs=f)
            for _ in range(2):
                for x in out:
                    x.fill_(-9)
                g.replay()
                assert all(torch.equal(x, y) for x, y in zip(out, want))
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        for x in out:
            x.fill_(-9)
        st.wait_stream(torch.cuda.current_stream())
        api.pa_tree_verify(*args, *out, draft_probs=f, stream=st)
        st.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want))
    finally:
        api.pa_set_launch_overlap(api.OVERLAP_OFF)


# ------------------------------------------------------------------ accept

class Batch:
    """Page table, lengths and paths of a batch; nodes are the last tokens of each row."""

    def __init__(self, context, nodes, seed, page=16, width=None):
        g = gen(seed)
        self.context, self.nodes = context, nodes
        self.lens = [a + b for a, b in zip(context, nodes)]
        pages = [-(-n // page) for n in self.lens]
        perm = torch.randperm(sum(pages) + 3, generator=g)
        self.size = (sum(pages) + 3) * page
        width = width or max(self.lens) + 4
        R = len(nodes)
        self.rows = torch.randperm(R + 2, generator=g)[:R].int()
        self.table = torch.full((R + 2, width), -5, dtype=torch.int32)
        at = 0
        for r, n in enumerate(self.lens):
            j = torch.arange(n)
            self.table[self.rows[r], :n] = (perm[at + j // page] * page + j % page).int()
            at += pages[r]
        self.paths = []
        for n in nodes:
            keep = (torch.rand(n, generator=g) < 0.4).tolist()
            self.paths.append([i for i in range(n) if keep[i] or i == 0])
        self.qo = [0]
        for n in nodes:
            self.qo.append(self.qo[-1] + n)
        self.g = g

    def call(self, max_path=None, k=None, v=None, err=None, in_place=False, **kw):
        mp = max_path or max([len(p) for p in self.paths] + [1]) + 2
        acc = i32([p + [-1] * (mp - len(p)) for p in self.paths])
        n = i32([len(p) for p in self.paths])
        self.dtable, lens = self.table.cuda(), i32(self.lens)
        new = lens if in_place else torch.full_like(lens, -7)
        freed = torch.full((self.qo[-1],), -7, dtype=torch.int32, device="cuda")
        api.pa_kv_accept(self.dtable, self.rows.cuda(), lens, i32(self.qo), acc, n, new, freed, k_buf=k, v_buf=v,
                         error_word=err, **kw)
        return self.dtable.cpu(), new.tolist(), freed.tolist()

    def want(self, move=False, skip=()):
        table, lens, freed, moves = self.table.clone(), [], [-7] * self.qo[-1], []
        for r, n in enumerate(self.nodes):
            row = table[self.rows[r]].tolist()
            if r in skip:
                lens.append(self.lens[r])
                continue
            if move:
                m, new, gone = S.accept_move(row, self.context[r], n, self.paths[r])
                moves += m
            else:
                row, new, gone = S.accept(row, self.context[r], n, self.paths[r])
                table[self.rows[r]] = torch.tensor(row, dtype=torch.int32)
            lens.append(new)
            freed[self.qo[r]:self.qo[r] + len(gone)] = gone
        return table, lens, freed, moves


CONTEXT = [0, 5, 100, 0, 17, 300, 2, 40]
NODES = [1, 7, 32, 0, 130, 300, 3, 16]


@pytest.mark.parametrize("page", [1, 16])
@pytest.mark.parametrize("in_place", [False, True])
def test_accept_table(page, in_place):
    b = Batch(CONTEXT, NODES, 1 + page, page)
    err = i32([0])
    table, lens, freed = b.call(err=err, in_place=in_place)
    t, l, f, _ = b.want()
    assert api.pa_get_error_word(err) == 0 and torch.equal(table, t) and lens == l and freed == f


@pytest.mark.parametrize("dtype,D,Hkv", [(torch.bfloat16, 128, 8), (torch.bfloat16, 64, 3), (torch.uint8, 64, 1),
                                         (torch.float8_e4m3fn, 128, 40), (torch.bfloat16, 8, 1)])
def test_accept_move(dtype, D, Hkv):
    b = Batch(CONTEXT, NODES, 3)
    raw = torch.randint(0, 256, (3, b.size, Hkv, D * dtype.itemsize), generator=b.g, dtype=torch.uint8)
    k, v = raw.cuda().view(dtype), raw.flip(1).contiguous().cuda().view(dtype)
    want_k, want_v = raw.clone(), raw.flip(1).contiguous()
    err = i32([0])
    table, lens, freed = b.call(k=k, v=v, err=err)
    t, l, f, moves = b.want(move=True)
    assert api.pa_get_error_word(err) == 0 and torch.equal(table, t) and lens == l and freed == f
    for buf in (want_k, want_v):
        old = buf.clone()
        for src, dst in moves:
            buf[:, dst] = old[:, src]
    assert torch.equal(k.view(torch.uint8).cpu(), want_k) and torch.equal(v.view(torch.uint8).cpu(), want_v)


def test_accept_everything_and_nothing():
    for keep in (lambda n: list(range(n)), lambda n: [], lambda n: [n - 1] if n else []):
        b = Batch(CONTEXT, NODES, 4)
        b.paths = [keep(n) for n in NODES]
        table, lens, freed = b.call()
        t, l, f, _ = b.want()
        assert torch.equal(table, t) and lens == l and freed == f


def test_accept_bad_inputs():
    base = Batch(CONTEXT, NODES, 5)
    good = base.call()

    def differs(change, bit, skip, move=False):
        b = Batch(CONTEXT, NODES, 5)
        change(b)
        err = i32([0])
        kv = {}
        if move:
            k = torch.zeros((1, b.size, 1, 64), dtype=torch.bfloat16, device="cuda")
            kv = dict(k=k, v=k.clone())
        table, lens, freed = b.call(err=err, max_path=310, **kv)
        assert api.pa_get_error_word(err) == bit
        for r in range(len(NODES)):
            row = table[b.rows[r].clamp(0, 9)]
            if r in skip:
                assert freed[base.qo[r]:base.qo[r + 1]] == [-7] * NODES[r]
                assert lens[r] == max(0, min(b.lens[r], b.table.shape[1]))
            elif not move and int(b.rows[r]) not in [int(b.rows[x]) for x in skip]:
                assert torch.equal(row, good[0][b.rows[r]]) and lens[r] == good[1][r]

    for move in (False, True):
        differs(lambda b: b.paths[2].__setitem__(1, 0), api.DEVERR_TREE, {2}, move)          # not increasing
        differs(lambda b: b.paths[2].__setitem__(-1, 32), api.DEVERR_TREE, {2}, move)        # no such node
        differs(lambda b: b.paths[2].__setitem__(0, -1), api.DEVERR_TREE, {2}, move)
        differs(lambda b: b.paths[1].extend(range(7, 20)), api.DEVERR_TREE, {1}, move)       # longer than the nodes
        differs(lambda b: b.rows.__setitem__(2, 99), api.DEVERR_ROW, {2}, move)
        differs(lambda b: b.rows.__setitem__(5, int(b.rows[2])), api.DEVERR_ROW, {5}, move)  # a row twice
        differs(lambda b: b.lens.__setitem__(4, 129), api.DEVERR_LEN, {4}, move)             # fewer tokens than nodes
        differs(lambda b: b.lens.__setitem__(4, 10 ** 6), api.DEVERR_LEN, {4}, move)
        differs(lambda b: b.lens.__setitem__(4, -3), api.DEVERR_LEN, {4}, move)
        differs(lambda b: b.rows.__setitem__(3, -1), 0, {3}, move)                           # padding: no nodes, no row


def test_accept_move_bad_slots():
    b = Batch([10, 10], [6, 6], 6)
    b.paths = [[0, 2, 4], [0, 3]]
    raw = torch.randn((2, b.size, 2, 64), generator=b.g).to(torch.bfloat16)
    was = b.table.clone()
    for bad in (-1, b.size, 2 ** 31 - 1):
        b.table = was.clone()
        b.table[b.rows[0], 12] = bad                   # node 2: moved to position 11
        k = raw.cuda()
        v = raw.cuda()
        err = i32([0])
        b.call(k=k, v=v, err=err)
        assert api.pa_get_error_word(err) == api.DEVERR_SLOT
        want = raw.clone()
        want[:, was[b.rows[1], 11]] = raw[:, was[b.rows[1], 13]]
        # node 4 goes to position 12, whose slot is bad as well
        assert torch.equal(k.cpu(), want)


def test_accept_graph_and_overlap():
    b = Batch([30, 9], [20, 4], 7)
    want = b.want()
    try:
        for mode in (api.OVERLAP_OFF, api.OVERLAP_SAFE, api.OVERLAP_EARLY_METADATA):
            api.pa_set_launch_overlap(mode)
            acc = i32([p + [-1] * (20 - len(p)) for p in b.paths])
            n, table, lens, rows, qo = i32([len(p) for p in b.paths]), b.table.cuda(), i32(b.lens), b.rows.cuda(), i32(b.qo)
            new, freed = torch.empty_like(lens), torch.full((24,), -7, dtype=torch.int32, device="cuda")
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                api.pa_kv_accept(table, rows, lens, qo, acc, n, new, freed)
            assert torch.equal(table.cpu(), b.table)
            g.replay()
            assert torch.equal(table.cpu(), want[0]) and new.tolist() == want[1] and freed.tolist() == want[2]
    finally:
        api.pa_set_launch_overlap(api.OVERLAP_OFF)


# -------------------------------------------------------------- end to end

@pytest.mark.parametrize("block,move", [(0, False), (0, True), (16, False)])
@pytest.mark.parametrize("graph", [False, True])
def test_speculative_steps(block, move, graph):
    """Attention of the drafted trees, verification, acceptance, then a decode over what stayed: each step's results are
    those of a plain request that only ever had the kept tokens."""
    context, nodes, Hkv, G, D, V = [70, 200, 15], [9, 16, 5], 2, 4, 64, 501
    c = make(context, nodes, Hkv, D, 16, block, 21, layers=2, layer=1)
    g = c.g
    parents = [S.random_parents(n, g) for n in nodes]
    seen = [S.tree_seen(p) for p in parents]
    q = queries(c, G, D)
    d = Drafts(nodes, V, 22)
    d.parents = [a for p in parents for a in p]
    k, v, table, rws, ke, ve = c.dev
    more = dict(k_exp=ke, v_exp=ve, block=block) if block else {}
    mask, qo, dq, out = pack(seen), i32(c.qo), q.cuda(), torch.full_like(q.cuda(), math.nan)
    ws = api.alloc_workspace(api.pa_tree_workspace_bytes(G * Hkv, Hkv, D))
    args = [d.p.cuda(), i32(d.tokens), i32(d.parents), qo, d.u.cuda(), d.ul.cuda()]
    acc, n, nxt = torch.full((3, 16), -7, dtype=torch.int32, device="cuda"), i32([0] * 3), i32([0] * 3)
    f, new, freed, err = d.f.cuda(), i32([0] * 3), torch.full((30,), -7, dtype=torch.int32, device="cuda"), i32([0])
    # the values the cache holds now, before rows move
    kept_kv = [c.values(r) for r in range(3)]
    kept_kv = [(a.clone(), b.clone()) for a, b in kept_kv]
    slots0 = [table[int(c.rows[r]), :c.lens[r]].clone() for r in range(3)]

    def step():
        api.pa_paged_tree_attn(dq, k, v, 1, qo, table, rws, c.dlens, 0.05, ws, out, tree_mask=mask, **more)
        api.pa_tree_verify(*args, acc, n, nxt, draft_probs=f, error_word=err)
        api.pa_kv_accept(table, rws, c.dlens, qo, acc, n, new, freed, k_buf=k if move else None, v_buf=v if move else None,
                         error_word=err)

    if graph:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step()
        gr.replay()
    else:
        step()
    assert api.pa_get_error(ws) == 0 and api.pa_get_error_word(err) == 0
    check(c, q, out, 0.05, seen, "drafted tokens")
    d.check((acc, n, nxt), "verification")
    # a plain decode over what stayed
    qd = torch.randn((3, G * Hkv, D), generator=g).to(torch.bfloat16)
    od = torch.full_like(qd.cuda(), math.nan)
    lens = new.tolist()
    if block:
        wd = api.alloc_workspace(api.pa_decode_fp8_block_workspace_bytes(G * Hkv, Hkv, D))
        api.pa_paged_decode_attn_fp8_block(qd.cuda(), k, v, 1, table, rws, new, 0.05, ke, ve, block, wd, od)
    else:
        wd = api.alloc_workspace(api.pa_decode_workspace_bytes(3, G * Hkv, Hkv, D, 8))
        api.pa_paged_decode_attn(qd.cuda(), k, v, 1, table, rws, new, 0.05, wd, 8, od)
    assert api.pa_get_error(wd) == 0
    import _block_ref as R
    for r in range(3):
        path = acc[r, :n[r]].tolist()
        at = list(range(context[r])) + [context[r] + e for e in path]
        assert lens[r] == len(at)
        kk, vv = kept_kv[r][0][at], kept_kv[r][1][at]
        ref = S.attention(qd[r][None].double(), kk, vv, 0.05, torch.ones((1, 1), dtype=torch.bool))
        # decode's weights: bf16 (plain) or 12 bits with q within 2^-22 of its largest element
        ref["ds"] = ref["ds"] + 2.0 ** -19
        R.check_out(od[r][None].cpu(), ref, 8, f"decode behind the step, request {r}")
        gone = freed[c.qo[r]:c.qo[r + 1]][:nodes[r] - len(path)].tolist()
        row = table[int(c.rows[r])]
        assert set(gone).isdisjoint(row[:lens[r]].tolist())
        assert sorted(gone + row[:lens[r]].tolist()) == sorted(slots0[r].tolist())
