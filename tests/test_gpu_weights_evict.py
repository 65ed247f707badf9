"""Decode attention with accumulated weights, and eviction by them, on the GPU
against plain 64-bit and plain Python references; then a serving loop of store,
decode with weights and eviction."""
import math

import numpy as np
import pytest
import torch

import _block_ref as R
from paged_kv_cache_188_gb300 import api
from test_gpu_fp8_block import Cache, gen, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.lib()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Bf16Cache(Cache):
    """The page table of a Cache over bf16 rows; unused slots hold NaN."""

    def __init__(self, lens, Hkv, D, page, seed, **kw):
        super().__init__(lens, Hkv, D, page, 1, seed, **kw)
        layers = self.k.shape[0]
        self.block = 0
        self.k = torch.full((layers, self.size, Hkv, D), math.nan, dtype=torch.bfloat16)
        self.v = self.k.clone()
        for s in self.slots:
            self.k[self.layer, s] = rows((len(s), Hkv, D), self.g)
            self.v[self.layer, s] = rows((len(s), Hkv, D), self.g)

    def values(self, b):
        return self.k[self.layer, self.slots[b]].double(), self.v[self.layer, self.slots[b]].double()


def weights_call(c, q, scale, weights, ws=None, out=None):
    k, v, table, rws, ke, ve = c.dev
    if ws is None:
        ws = api.alloc_workspace(api.pa_decode_weights_workspace_bytes(len(c.lens), sum(c.lens), q.shape[1], k.shape[2],
                                                                       q.shape[2]))
    out = torch.full_like(q, math.nan) if out is None else out
    more = dict(k_exp=ke, v_exp=ve, block=c.block) if c.block else {}
    api.pa_paged_decode_attn_weights(q, k, v, c.layer, table, rws, c.dlens, scale, weights, ws, out, **more)
    return out, ws


def check_weights(c, q, out, w0, w1, scale, what):
    """Each row's additions within the scores' error (2 ds, relative, per head) and fp32 sums; other rows and entries
    behind a request's length as they were."""
    want, tol = w0.double().clone(), torch.zeros_like(w0, dtype=torch.float64)
    for b, n in enumerate(c.lens):
        if n == 0:
            assert torch.count_nonzero(out[b]) == 0
            continue
        k, v = c.values(b)
        r = R.attention(q[b][None].double(), k, v, scale)
        R.check_out(out[b][None].cpu(), r, 12, f"{what}, request {b} of {n}")
        row = int(c.rows[b])
        want[row, :n] += r["p"][0].sum(0)
        tol[row, :n] = (r["p"][0] * (2 * r["ds"][0][:, None] + 2.0 ** -18)).sum(0) + 2.0 ** -22 * want[row, :n] + 1e-30
    d = (w1.cpu().double() - want).abs()
    assert (d <= tol).all(), f"{what}: weights off by {float((d - tol).max()):.3e}"


LENS = [1, 127, 128, 129, 0, 300, 1500, 16]


@pytest.mark.parametrize("G,Hkv", [(4, 2), (1, 3), (8, 1), (16, 2), (5, 1)])
@pytest.mark.parametrize("D,page", [(128, 16), (64, 16), (128, 1), (64, 1)])
def test_weights_bf16(G, Hkv, D, page):
    c = Bf16Cache(LENS, Hkv, D, page, G + 10 * D + page).cuda()
    q = torch.randn((len(LENS), G * Hkv, D), generator=c.g).to(torch.bfloat16)
    w = torch.rand(c.table.shape, generator=c.g)
    dw = w.cuda()
    out, ws = weights_call(c, q.cuda(), 0.1, dw)
    assert api.pa_get_error(ws) == 0
    check_weights(c, q, out, w, dw, 0.1, f"bf16 G={G} D={D} page={page}")


@pytest.mark.parametrize("G,Hkv", [(4, 2), (1, 3), (8, 1), (16, 1)])
@pytest.mark.parametrize("D,page,block", [(128, 16, 16), (64, 1, 1), (128, 32, 8), (64, 128, 128)])
def test_weights_fp8_block(G, Hkv, D, page, block):
    c = Cache(LENS, Hkv, D, page, block, G + D + page).cuda()
    q = torch.randn((len(LENS), G * Hkv, D), generator=c.g).to(torch.bfloat16)
    w = torch.rand(c.table.shape, generator=c.g)
    dw = w.cuda()
    out, ws = weights_call(c, q.cuda(), 0.05, dw)
    assert api.pa_get_error(ws) == 0
    check_weights(c, q, out, w, dw, 0.05, f"e4m3 G={G} D={D} page={page} block={block}")


def test_weights_output_is_decode_of_the_same_cache():
    """Keeping weights changes no bit of the output."""
    from test_gpu_fp8_block import decode
    c = Cache([3000, 0, 70], 2, 128, 16, 16, 5).cuda()
    q = torch.randn((3, 8, 128), generator=c.g).to(torch.bfloat16).cuda()
    out, _ = decode(c, q, 0.05)
    got, _ = weights_call(c, q, 0.05, torch.zeros(c.table.shape, device="cuda"))
    assert torch.equal(out.view(torch.int16), got.view(torch.int16))


@pytest.mark.parametrize("bf16", [True, False])
def test_weights_add_up_over_calls_graphs_and_overlap(bf16):
    """Long request over many CTAs; three replays add three times, deterministically, in every overlap mode."""
    lens = [20000, 3]
    c = (Bf16Cache(lens, 2, 128, 16, 6, layers=1, layer=0) if bf16 else Cache(lens, 2, 128, 16, 16, 6, layers=1, layer=0)).cuda()
    q = torch.randn((2, 8, 128), generator=c.g).to(torch.bfloat16)
    w = torch.zeros(c.table.shape, device="cuda")
    out, ws = weights_call(c, q.cuda(), 0.05, w)
    check_weights(c, q, out, torch.zeros(c.table.shape), w, 0.05, f"20000, bf16 {bf16}")
    one = w.clone()
    assert abs(float(one.sum()) - 16.0) < 1e-3               # 8 heads, two requests
    dq, o = q.cuda(), torch.empty_like(out)
    try:
        for mode in (api.OVERLAP_OFF, api.OVERLAP_SAFE, api.OVERLAP_EARLY_METADATA, api.OVERLAP_EARLY_KV):
            api.pa_set_launch_overlap(mode)
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr):
                weights_call(c, dq, 0.05, w, ws=ws, out=o)
                weights_call(c, dq, 0.05, w, ws=ws, out=o)
            w.zero_()
            gr.replay()
            torch.cuda.synchronize()
            assert torch.equal(w, one + one), mode
            assert torch.equal(o.view(torch.int16), out.view(torch.int16)), mode
    finally:
        api.pa_set_launch_overlap(api.OVERLAP_OFF)


def test_weights_refuse_a_shared_row_and_a_small_workspace():
    c = Bf16Cache([200, 300, 50], 1, 64, 16, 7).cuda()
    q = torch.randn((3, 2, 64), generator=c.g).to(torch.bfloat16)
    c.dev[3][2] = c.dev[3][0]                          # request 2 names request 0's row
    w = torch.zeros(c.table.shape, device="cuda")
    out, ws = weights_call(c, q.cuda(), 0.1, w)
    assert api.pa_get_error(ws) == api.DEVERR_ROW
    r0, r1 = int(c.rows[0]), int(c.rows[1])
    for b, row in ((0, r0), (1, r1)):
        k, v = c.values(b)
        r = R.attention(q[b][None].double(), k, v, 0.1)
        assert float((w[row, :c.lens[b]].cpu().double() - r["p"][0].sum(0)).abs().max()) < 1e-5
    k, v = c.values(0)
    R.check_out(out[2][None].cpu(), R.attention(q[2][None].double(), k[:50], v[:50], 0.1), 12, "the later request")
    # a workspace of fewer tokens than the batch has: right outputs, an error, no addition out of place
    c = Bf16Cache([100, 1000], 1, 64, 16, 8).cuda()
    q = torch.randn((2, 2, 64), generator=c.g).to(torch.bfloat16)
    ws = api.alloc_workspace(api.pa_decode_weights_workspace_bytes(2, 128, 2, 1, 64))
    w = torch.zeros(c.table.shape, device="cuda")
    out, _ = weights_call(c, q.cuda(), 0.1, w, ws=ws)
    assert api.pa_get_error(ws) == api.DEVERR_LEN
    for b in range(2):
        k, v = c.values(b)
        r = R.attention(q[b][None].double(), k, v, 0.1)
        R.check_out(out[b][None].cpu(), r, 12, "small workspace")
        n = 100 if b == 0 else 256                     # three tiles' room: the first request's and two of the second's
        assert float((w[int(c.rows[b]), :n].cpu().double() - r["p"][0].sum(0)[:n]).abs().max()) < 1e-5
        assert torch.count_nonzero(w[int(c.rows[b]), n:]) == 0


def test_weights_wait_limit_zero_aborts():
    c = Bf16Cache([3000], 2, 128, 16, 9).cuda()
    q = torch.randn((1, 8, 128), generator=c.g).to(torch.bfloat16).cuda()
    w = torch.zeros(c.table.shape, device="cuda")
    try:
        api.pa_set_wait_timeout_ns(0)
        _, ws = weights_call(c, q, 0.05, w)
        torch.cuda.synchronize()
    finally:
        api.pa_set_wait_timeout_ns(api.WAIT_TIMEOUT_DEFAULT_NS)
    assert api.pa_get_error(ws) & api.DEVERR_TIMEOUT


# ------------------------------------------------------------------ eviction

def evict_case(lens, max_ctx, budget, recent, make, seed, dup=None):
    g = gen(seed)
    B, R_ = len(lens), len(lens) + 2
    table = torch.randint(0, 10 ** 6, (R_, max_ctx), generator=g).int()
    w = make((R_, max_ctx), g).float()
    rws = torch.randperm(R_, generator=g)[:B].int()
    dt, dw, dr = table.cuda(), w.cuda(), rws.cuda()
    new = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    freed = torch.full((B, max_ctx), -9, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.pa_kv_evict(dt, dr, i32(lens), dw, budget, recent, new, freed, err)
    assert api.pa_get_error_word(err) == 0
    for b, n in enumerate(lens):
        row = int(rws[b])
        slots, ws, gone = R.evict(table[row, :n].tolist(), w[row, :n].tolist(), budget, recent)
        m = len(slots)
        assert int(new[b]) == m
        table[row, :m] = torch.tensor(slots, dtype=torch.int32)
        w[row, :n] = torch.tensor(ws + [0.0] * (n - m))
        assert freed[b, :n - m].tolist() == gone and (freed[b, n - m:] == -9).all()
    assert torch.equal(dt.cpu(), table)
    assert torch.equal(dw.cpu().view(torch.int32), w.view(torch.int32))


uniform = lambda shape, g: torch.rand(shape, generator=g)  # noqa: E731
ties = lambda shape, g: torch.randint(0, 3, shape, generator=g).float()  # noqa: E731
zeros = lambda shape, g: torch.zeros(shape)  # noqa: E731


def odd(shape, g):
    """Both zeros, negatives, infinities, subnormals and neighbours in the last place."""
    pool = torch.tensor([0.0, -0.0, -1.0, math.inf, -math.inf, 1e-42, -1e-42, 1.0, 1.0 + 2.0 ** -23, 1.0 - 2.0 ** -24, 3e38])
    return pool[torch.randint(0, len(pool), shape, generator=g)]


@pytest.mark.parametrize("make", [uniform, ties, zeros, odd])
@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (64, 0), (64, 64), (100, 37), (1000, 8)])
def test_evict_small(make, budget, recent):
    evict_case([0, 1, 2, 63, 64, 65, 101, 500, 999, 1000, 1001], 1003, budget, recent, make, budget + recent)


@pytest.mark.parametrize("make", [uniform, ties])
@pytest.mark.parametrize("max_ctx", [4096, 4097, 8192, 16001, 32768, 33000, 100003])
def test_evict_cluster_sizes_and_chunks(make, max_ctx):
    """One CTA to eight per request, one chunk to several; rows that are not 16-byte aligned."""
    evict_case([max_ctx, max_ctx - 1, 4096, 3000], max_ctx, 2500, 300, make, max_ctx)
    evict_case([max_ctx], max_ctx, max_ctx - 1, 17, make, max_ctx + 1)


def test_evict_nan_counts_as_minus_infinity():
    w = torch.tensor([[math.nan, 1.0, -math.inf, 2.0, math.nan, 0.5]], device="cuda")
    t = i32([[10, 11, 12, 13, 14, 15]])
    new, freed = i32([0]), torch.full((1, 6), -1, dtype=torch.int32, device="cuda")
    api.pa_kv_evict(t, i32([0]), i32([6]), w, 4, 0, new, freed)
    assert t[0, :4].tolist() == [10, 11, 13, 15] and freed[0].tolist() == [12, 14, -1, -1, -1, -1]
    assert math.isnan(float(w[0, 0])) and w[0, 1:].tolist() == [1.0, 2.0, 0.5, 0.0, 0.0]


def test_evict_refused_requests_stay_as_they_are():
    t = torch.arange(40, dtype=torch.int32, device="cuda").view(4, 10).contiguous()
    w = torch.rand((4, 10), generator=gen(1)).cuda()
    t0, w0 = t.clone(), w.clone()
    new, freed, err = i32([0] * 5), torch.full((5, 10), -1, dtype=torch.int32, device="cuda"), i32([0])
    api.pa_kv_evict(t, i32([2, 4, 2, 1, 0]), i32([8, 8, 8, 11, -3]), w, 3, 1, new, freed, err)
    assert api.pa_get_error_word(err) == api.DEVERR_ROW | api.DEVERR_LEN
    assert new.tolist() == [3, 8, 8, 10, 0]
    keep = [0, 1, 3]
    assert torch.equal(t[keep], t0[keep]) and torch.equal(w[keep], w0[keep])
    assert (freed[1:] == -1).all() and int((freed[0] >= 0).sum()) == 5


def test_evict_lengths_in_place_and_in_a_graph():
    """new_lens may be seq_lens; a captured call evicts once and then leaves the request alone."""
    g = gen(2)
    t0 = torch.randint(0, 10 ** 6, (3, 5000), generator=g).int()
    w0 = torch.rand((3, 5000), generator=g)
    t, w, lens = t0.cuda(), w0.cuda(), i32([5000, 700, 4100])
    freed = torch.zeros((3, 5000), dtype=torch.int32, device="cuda")
    rws = i32([1, 2, 0])
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        api.pa_kv_evict(t, rws, lens, w, 1000, 100, lens, freed)
    for _ in range(2):
        gr.replay()
        torch.cuda.synchronize()
        assert lens.tolist() == [1000, 700, 1000]
        for b, (row, n) in enumerate(((1, 5000), (2, 700), (0, 4100))):
            slots, ws, gone = R.evict(t0[row, :n].tolist(), w0[row, :n].tolist(), 1000, 100)
            assert t[row, :len(slots)].tolist() == slots and torch.equal(w[row, :len(ws)].cpu(), torch.tensor(ws))
            assert freed[b, :len(gone)].tolist() == gone


def test_evict_lengths_in_place_past_the_end():
    """Lengths past max_ctx or negative, in place, rows wide enough for several CTAs per request: every CTA of a
    request has to see the length as it was."""
    B, max_ctx = 40, 33000
    t = torch.arange(B * max_ctx, dtype=torch.int32, device="cuda").view(B, max_ctx).contiguous()
    w = torch.rand((B, max_ctx), generator=gen(3)).cuda()
    t0, w0 = t.clone(), w.clone()
    lens = [max_ctx + 1 + b if b % 2 else -b for b in range(B)]
    dev, freed, err = i32(lens), torch.full((B, max_ctx), -1, dtype=torch.int32, device="cuda"), i32([0])
    api.pa_kv_evict(t, i32(list(range(B))), dev, w, 10, 3, dev, freed, err)
    assert api.pa_get_error_word(err) == api.DEVERR_LEN
    assert dev.tolist() == [max_ctx if b % 2 else 0 for b in range(B)]
    assert torch.equal(t, t0) and torch.equal(w, w0) and (freed == -1).all()


def test_padding_without_tokens_may_share_a_row():
    """A padded batch: requests of no tokens name the row of a real one, before and after it."""
    c = Bf16Cache([0, 300, 0, 40], 2, 64, 16, 10).cuda()
    c.dev[3][0] = c.dev[3][2] = c.dev[3][1]
    q = torch.randn((4, 4, 64), generator=c.g).to(torch.bfloat16)
    w = torch.zeros(c.table.shape, device="cuda")
    out, ws = weights_call(c, q.cuda(), 0.1, w)
    assert api.pa_get_error(ws) == 0 and not out[0].any() and not out[2].any()
    for b in (1, 3):
        k, v = c.values(b)
        r = R.attention(q[b][None].double(), k, v, 0.1)
        R.check_out(out[b][None].cpu(), r, 12, "padded batch")
        want = r["p"][0].sum(0)
        tol = (r["p"][0] * (2 * r["ds"][0][:, None] + 2.0 ** -18)).sum(0) + 2.0 ** -22 * want + 1e-30
        assert ((w[int(c.rows[b]), :c.lens[b]].cpu().double() - want).abs() <= tol).all()
    # eviction of the same batch
    table, slots, new = c.dev[2].clone(), c.dev[2][int(c.rows[1])].tolist(), i32([-1] * 4)
    heavy = w[int(c.rows[1])].tolist()
    freed, err = torch.full((4, table.shape[1]), -1, dtype=torch.int32, device="cuda"), i32([0])
    api.pa_kv_evict(table, c.dev[3], i32(c.lens), w, 100, 10, new, freed, err)
    assert api.pa_get_error_word(err) == 0 and new.tolist() == [0, 100, 0, 40]
    kept, _, gone = R.evict(slots[:300], heavy[:300], 100, 10)
    assert table[int(c.rows[1]), :100].tolist() == kept and freed[1, :200].tolist() == gone


# ------------------------------------------------------------ a serving loop

@pytest.mark.parametrize("D,block", [(128, 16), (64, 1), (64, 32)])
def test_captured_chain_in_every_overlap_mode(D, block):
    """Reset, a prompt stored and prefilled, a token appended, decode with weights and eviction, captured together on a
    stream of its own: what the calls give one by one, whatever the overlap."""
    g = gen(D + block)
    Hkv, G, new, page = 2, 4, [150, 37, 1], 32
    B, ctx, size, T = len(new), 200, 16 * page, sum(new)
    perm = torch.randperm(size // page, generator=g)
    table0, at = torch.zeros((B + 1, ctx), dtype=torch.int32), 0
    for b, n in enumerate(new):
        j = torch.arange(n + 1)
        table0[b + 1, :n + 1] = (perm[at + j // page] * page + j % page).int()
        at += n // page + 1
    loc = torch.cat([table0[b + 1, :n] for b, n in enumerate(new)]).cuda()
    last = torch.tensor([int(table0[b + 1, n]) for b, n in enumerate(new)], dtype=torch.int32).cuda()
    rnd = lambda *shape: torch.randn(shape, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    kp, vp, k1, v1 = rnd(T, Hkv, D), rnd(T, Hkv, D), rnd(B, Hkv, D) * 9, rnd(B, Hkv, D) * 9
    qp, qd = rnd(T, Hkv * G, D), rnd(B, Hkv * G, D)
    nb = -(-size // block)
    k, v = (torch.zeros((1, size, Hkv, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    ke, ve = (torch.zeros((1, nb, Hkv), dtype=torch.uint8, device="cuda") for _ in range(2))
    blocks, rws = torch.arange(nb, dtype=torch.int32, device="cuda"), i32(range(1, B + 1))
    qo, lens = i32([0] + torch.tensor(new).cumsum(0).tolist()), i32([n + 1 for n in new])
    table, src, w = table0.cuda(), table0.cuda(), torch.zeros((B + 1, ctx), device="cuda")
    outp, outd, newl = torch.empty_like(qp), torch.empty_like(qd), i32([0] * B)
    freed = torch.zeros((B, ctx), dtype=torch.int32, device="cuda")
    ws1 = api.alloc_workspace(api.pa_prefill_workspace_bytes())
    ws2 = api.alloc_workspace(api.pa_decode_weights_workspace_bytes(B, T + B, Hkv * G, Hkv, D))

    def chain():
        table.copy_(src)
        w.zero_()
        api.pa_kv_reset_fp8_block(ke, ve, blocks)
        api.pa_kv_store_fp8_block(k, v, 0, kp, vp, loc, ke, ve, block)
        api.pa_paged_prefill_attn_fp8_block(qp, k, v, 0, qo, qo, table, rws, 0.1, ke, ve, block, ws1, outp)
        api.pa_kv_store_fp8_block(k, v, 0, k1, v1, last, ke, ve, block)
        api.pa_paged_decode_attn_weights(qd, k, v, 0, table, rws, lens, 0.1, w, ws2, outd, k_exp=ke, v_exp=ve, block=block)
        api.pa_kv_evict(table, rws, lens, w, 100, 10, newl, freed)

    got = (outp, outd, w, table, newl, freed)
    chain()
    torch.cuda.synchronize()
    want = [x.clone() for x in got]
    assert newl.tolist() == [100, 38, 2] and torch.isfinite(outp.float()).all() and float(w[3, :2].sum()) > 7.99
    try:
        for mode in (api.OVERLAP_OFF, api.OVERLAP_SAFE, api.OVERLAP_EARLY_METADATA, api.OVERLAP_EARLY_KV):
            api.pa_set_launch_overlap(mode)
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr):
                chain()
            for _ in range(3):
                for x in got:
                    x.zero_()
                gr.replay()
                torch.cuda.synchronize()
                for x, y in zip(got, want):
                    assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), mode
    finally:
        api.pa_set_launch_overlap(api.OVERLAP_OFF)
    assert api.pa_get_error(ws1) == 0 and api.pa_get_error(ws2) == 0


@pytest.mark.parametrize("block", [0, 1])
def test_serving_loop_with_eviction(block):
    """Three requests, token by token: store, decode with weights, evict when over budget, the freed slots used
    again; the cache, the table, the weights' order and the outputs against the references at every step."""
    Hkv, Hq, D, B, budget, recent, steps = 2, 4, 64, 3, 24, 6, 60
    size, max_ctx, scale = B * (budget + 1), 40, 0.3
    g = gen(77 + block)
    dt = torch.uint8 if block else torch.bfloat16
    k, v = (torch.zeros((1, size, Hkv, D), dtype=dt, device="cuda") for _ in range(2))
    ke, ve = (torch.zeros((1, size, Hkv), dtype=torch.uint8, device="cuda") for _ in range(2))
    host = [np.zeros((size, Hkv, D), np.uint8) if block else torch.zeros((size, Hkv, D), dtype=torch.bfloat16) for _ in range(2)]
    hexp = [np.zeros((size, Hkv), np.uint8) for _ in range(2)]
    table = torch.full((B + 1, max_ctx), -5, dtype=torch.int32, device="cuda")
    weights = torch.zeros((B + 1, max_ctx), device="cuda")
    rws, lens = [2, 0, 3], [0] * B
    mine = [[] for _ in range(B)]                  # the reference's table and weights
    hw = [[] for _ in range(B)]
    free = list(range(size))
    dlens, freed = i32([0] * B), torch.zeros((B, max_ctx), dtype=torch.int32, device="cuda")
    new = i32([0] * B)
    ws = api.alloc_workspace(api.pa_decode_weights_workspace_bytes(B, size + B, Hq, Hkv, D))
    evictions = 0
    for step in range(steps):
        act = [b for b in range(B) if step >= 5 * b]
        loc = [free.pop(0) for _ in act]
        kn, vn = rows((len(act), Hkv, D), g), rows((len(act), Hkv, D), g)
        dloc = i32(loc)
        for b, s in zip(act, loc):
            table[rws[b], lens[b]] = s
            mine[b].append(s)
            hw[b].append(0.0)
            lens[b] += 1
        dlens.copy_(i32(lens))
        if block:
            stale = dloc.clone()
            api.pa_kv_reset_fp8_block(ke, ve, stale)
            api.pa_kv_store_fp8_block(k, v, 0, kn.cuda(), vn.cuda(), dloc, ke, ve, block)
            for i, x in enumerate((kn, vn)):
                hexp[i][loc] = 0
                R.store(host[i], hexp[i], x.double().numpy(), loc, block)
        else:
            api.pa_kv_store(k, v, 0, kn.cuda(), vn.cuda(), dloc)
            host[0][loc], host[1][loc] = kn, vn
        q = torch.randn((B, Hq, D), generator=g).to(torch.bfloat16)
        out = torch.empty_like(q, device="cuda")
        more = dict(k_exp=ke, v_exp=ve, block=block) if block else {}
        api.pa_paged_decode_attn_weights(q.cuda(), k, v, 0, table, i32(rws), dlens, scale, weights, ws, out, **more)
        got_w = weights.cpu()
        for b in range(B):
            if not lens[b]:
                assert torch.count_nonzero(out[b]) == 0
                continue
            at = torch.tensor(mine[b])
            if block:
                kk, vv = (R.values(torch.from_numpy(host[i]), torch.from_numpy(hexp[i]), at, block) for i in range(2))
            else:
                kk, vv = (host[i][at].double() for i in range(2))
            r = R.attention(q[b][None].double(), kk, vv, scale)
            R.check_out(out[b][None].cpu(), r, 12, f"step {step}, request {b}")
            add = r["p"][0].sum(0).tolist()
            hw[b] = [x + y for x, y in zip(hw[b], add)]
            row = got_w[rws[b], :lens[b]].double()
            assert float((row - torch.tensor(hw[b], dtype=torch.float64)).abs().max()) < 1e-4
        api.pa_kv_evict(table, i32(rws), dlens, weights, budget, recent, new, freed)
        for b in range(B):
            # the reference evicts by the library's own accumulated weights: equal choices, not nearly equal ones
            slots, kept, gone = R.evict(mine[b], got_w[rws[b], :lens[b]].tolist(), budget, recent)
            assert int(new[b]) == len(slots) and table[rws[b], :len(slots)].tolist() == slots
            assert freed[b, :len(gone)].tolist() == gone
            if gone:
                evictions += 1
                pos = [mine[b].index(s) for s in slots]
                hw[b] = [hw[b][j] for j in pos]
                mine[b], lens[b] = slots, len(slots)
                free += gone
    assert evictions > 60 and api.pa_get_error(ws) == 0
