"""The block-scaled e4m3 cache on the GPU: the store byte for byte, decode and
prefill attention over it against a plain 64-bit reference with tolerances
counted from the roundings the kernels make."""
import math

import numpy as np
import pytest
import torch

import _block_ref as R
from paged_kv_cache_188_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.lib()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rows(shape, g, spread=0.6):
    """bf16 rows, each (token, head) with a magnitude of its own."""
    x = torch.randn(shape, generator=g) * torch.exp(spread * torch.randn(shape[:-1], generator=g))[..., None]
    return x.to(torch.bfloat16)


def same_bytes(got, want, what):
    nan = (want & 127) == 127
    assert np.array_equal((got & 127) == 127, nan), f"{what}: NaN codes differ"
    bad = (got != want) & ~nan
    assert not bad.any(), f"{what}: {int(bad.sum())} bytes differ, first at {np.argwhere(bad)[0]}"


# -------------------------------------------------------------------- store

@pytest.mark.parametrize("D,Hkv", [(128, 3), (64, 2), (128, 8)])
@pytest.mark.parametrize("block", [1, 2, 4, 16, 32, 128])
def test_store_calls_in_turn(D, Hkv, block):
    """Prompts from the middle of a page, single-token appends and a prompt again, magnitudes rising and falling, the
    last block short; every byte and exponent of both layers after each call."""
    g = gen(D + Hkv * 7 + block)
    size, L, layer = 5 * max(block, 16) + 3, 2, 1
    nb = -(-size // block)
    k = torch.randint(0, 127, (L, size, Hkv, D), generator=g, dtype=torch.uint8)
    v = torch.randint(0, 127, (L, size, Hkv, D), generator=g, dtype=torch.uint8)
    ke = torch.zeros((L, nb, Hkv), dtype=torch.uint8)
    ve = torch.zeros((L, nb, Hkv), dtype=torch.uint8)
    want = [x.numpy().copy() for x in (k, v, ke, ve)]
    k, v, ke, ve = (x.cuda() for x in (k, v, ke, ve))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = max(block, 16)
    calls = [list(range(5, min(size, 2 * p + 7))), [2 * p + 7, 3 * p + 1, 4 * p + 2], [size - 1], [2 * p + 8], [0, 1, 2, 3],
             list(range(3 * p + 2, 4 * p))]
    for i, loc in enumerate(calls):
        kn, vn = rows((len(loc), Hkv, D), g, 1.5) * 2.0 ** (3 * i - 4), rows((len(loc), Hkv, D), g, 1.5) * 4.0 ** (2 - i)
        lt = torch.tensor(loc, dtype=torch.int32)
        api.pa_kv_store_fp8_block(k, v, layer, kn.cuda(), vn.cuda(), lt.cuda(), ke, ve, block, err)
        R.store(want[0][layer], want[2][layer], kn.double().numpy(), loc, block)
        R.store(want[1][layer], want[3][layer], vn.double().numpy(), loc, block)
        for got, w, name in zip((k, v, ke, ve), want, ("k", "v", "k_exp", "v_exp")):
            if name.endswith("exp"):
                assert np.array_equal(got.cpu().numpy(), w), f"{name} after call {i}"
            else:
                same_bytes(got.cpu().numpy(), w, f"{name} after call {i}")
    assert api.pa_get_error_word(err) == 0


@pytest.mark.parametrize("block", [1, 16])
def test_store_special_values_and_bad_slots(block):
    """NaN, infinities, signed zeros, the largest and smallest bf16 magnitudes, rows of zeros; slots out of range are
    skipped and flagged."""
    Hkv, D, size = 2, 64, 64
    x = rows((8, Hkv, D), gen(3))
    x[0, 0, :6] = torch.tensor([math.nan, math.inf, -math.inf, 0.0, -0.0, 3.38e38])
    x[1] = 0.0
    x[2] = 1e-38
    x[3, 1, 0] = math.nan
    x[4] = 9.2e-41
    x[5, 0] = math.inf
    loc = [3, 4, 5, -1, 40, 41, 64, 20]
    k, v = (torch.zeros((1, size, Hkv, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    ke, ve = (torch.zeros((1, size // block, Hkv), dtype=torch.uint8, device="cuda") for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.pa_kv_store_fp8_block(k, v, 0, x.cuda(), x.cuda(), torch.tensor(loc, dtype=torch.int32).cuda(), ke, ve, block, err)
    wk, we = np.zeros((size, Hkv, D), np.uint8), np.zeros((size // block, Hkv), np.uint8)
    R.store(wk, we, x.double().numpy(), loc, block)
    assert np.array_equal(ke[0].cpu().numpy(), we) and np.array_equal(ve[0].cpu().numpy(), we)
    same_bytes(k[0].cpu().numpy(), wk, "k")
    same_bytes(v[0].cpu().numpy(), wk, "v")
    assert api.pa_get_error_word(err) == api.DEVERR_SLOT


def test_reset_marks_listed_blocks_of_every_layer():
    ke = torch.full((3, 7, 2), 9, dtype=torch.uint8, device="cuda")
    ve = ke.clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.pa_kv_reset_fp8_block(ke, ve, torch.tensor([5, 0, 7, -1], dtype=torch.int32, device="cuda"), err)
    want = torch.full((3, 7, 2), 9, dtype=torch.uint8)
    want[:, [0, 5]] = 0
    assert torch.equal(ke.cpu(), want) and torch.equal(ve.cpu(), want)
    assert api.pa_get_error_word(err) == api.DEVERR_SLOT


@pytest.mark.parametrize("e", [253, 254])
def test_store_at_the_largest_exponents(e):
    """Rows stored into a block whose scale is 2^126 or 2^127 already."""
    size, Hkv, D = 16, 1, 64
    x = rows((4, Hkv, D), gen(e)) * 2.0 ** 126
    k, v = (torch.zeros((1, size, Hkv, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    ke, ve = (torch.full((1, 1, Hkv), e, dtype=torch.uint8, device="cuda") for _ in range(2))
    loc = [2, 3, 4, 9]
    api.pa_kv_store_fp8_block(k, v, 0, x.cuda(), x.cuda(), torch.tensor(loc, dtype=torch.int32).cuda(), ke, ve, 16)
    wk, we = np.zeros((size, Hkv, D), np.uint8), np.full((1, Hkv), e, np.uint8)
    R.store(wk, we, x.double().numpy(), loc, 16)
    assert wk.any() and ke.item() == e and ve.item() == e
    same_bytes(k[0].cpu().numpy(), wk, "k")
    same_bytes(v[0].cpu().numpy(), wk, "v")


def test_store_and_reset_of_nothing():
    k = torch.ones((1, 16, 1, 64), dtype=torch.uint8, device="cuda")
    e = torch.ones((1, 1, 1), dtype=torch.uint8, device="cuda")
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    new = torch.zeros((0, 1, 64), dtype=torch.bfloat16, device="cuda")
    api.pa_kv_store_fp8_block(k, k.clone(), 0, new, new, none, e, e.clone(), 16)
    api.pa_kv_reset_fp8_block(e, e.clone(), none)
    assert int(k.sum()) == k.numel() and int(e.sum()) == 1


# ---------------------------------------------------------------- the cache

class Cache:
    """A random block-scaled cache and a page table: unused slots hold NaN codes under a large scale, table entries
    behind a request's length are garbage."""

    def __init__(self, lens, Hkv, D, page, block, seed, layers=2, layer=1, exp_lo=112, exp_hi=124, extra_ctx=5):
        g = gen(seed)
        pages = [-(-n // page) for n in lens]
        n_pages = sum(pages) + 3
        self.size, self.block, self.layer, self.lens = n_pages * page, block, layer, list(lens)
        nb = -(-self.size // block)
        perm = torch.randperm(n_pages, generator=g)
        width = max(max(lens), 1) + extra_ctx
        self.rows = torch.randperm(len(lens) + 2, generator=g)[:len(lens)].int()
        self.table = torch.randint(-self.size, 2 * self.size, (len(lens) + 2, width), generator=g).int()
        self.k = torch.full((layers, self.size, Hkv, D), 127, dtype=torch.uint8)
        self.v = torch.full((layers, self.size, Hkv, D), 255, dtype=torch.uint8)
        self.ke = torch.randint(exp_lo, exp_hi + 1, (layers, nb, Hkv), generator=g).to(torch.uint8)
        self.ve = torch.randint(exp_lo, exp_hi + 1, (layers, nb, Hkv), generator=g).to(torch.uint8)
        at = 0
        self.slots = []
        for b, n in enumerate(lens):
            j = torch.arange(n)
            s = perm[at + j // page] * page + j % page
            at += pages[b]
            self.slots.append(s)
            self.table[self.rows[b], :n] = s.int()
            x = torch.randn((2, n, Hkv, D), generator=g) * 60
            codes = torch.from_numpy(R.encode(x.double().numpy()))
            self.k[layer, s], self.v[layer, s] = codes[0], codes[1]
        self.g = g

    def values(self, b):
        s, i = self.slots[b], self.layer
        return R.values(self.k[i], self.ke[i], s, self.block), R.values(self.v[i], self.ve[i], s, self.block)

    def cuda(self):
        self.dev = [x.cuda() for x in (self.k, self.v, self.table, self.rows, self.ke, self.ve)]
        self.dlens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        return self


def decode(c, q, scale, ws=None, stream=None, out=None):
    k, v, table, rws, ke, ve = c.dev
    ws = api.alloc_workspace(api.pa_decode_fp8_block_workspace_bytes(q.shape[1], k.shape[2], q.shape[2])) if ws is None else ws
    out = torch.full_like(q, math.nan) if out is None else out
    api.pa_paged_decode_attn_fp8_block(q, k, v, c.layer, table, rws, c.dlens, scale, ke, ve, c.block, ws, out, stream=stream)
    return out, ws


def check_decode(c, q, out, scale, what, reqs=None):
    for b in reqs if reqs is not None else range(len(c.lens)):
        if c.lens[b] == 0:
            assert torch.count_nonzero(out[b]) == 0
            continue
        k, v = c.values(b)
        r = R.attention(q[b][None].double(), k, v, scale)
        R.check_out(out[b][None].cpu(), r, 12, f"{what}, request {b} of {c.lens[b]}")


LENS = [1, 2, 127, 128, 129, 0, 300, 16, 1025, 640]


@pytest.mark.parametrize("G,Hkv", [(4, 2), (1, 3), (3, 1), (8, 2), (16, 1), (13, 2)])
@pytest.mark.parametrize("D,page,block", [(128, 16, 16), (128, 1, 1), (64, 16, 16), (64, 3, 1), (128, 32, 32), (64, 2, 2)])
def test_decode_ragged(G, Hkv, D, page, block):
    c = Cache(LENS, Hkv, D, page, block, G * 100 + D + page).cuda()
    q = torch.randn((len(LENS), G * Hkv, D), generator=c.g).to(torch.bfloat16)
    scale = 0.05
    out, ws = decode(c, q.cuda(), scale)
    assert api.pa_get_error(ws) == 0
    check_decode(c, q, out, scale, f"decode G={G} D={D} page={page} block={block}")


@pytest.mark.parametrize("D", [128, 64])
def test_decode_long_and_deterministic(D):
    """30000 tokens over every CTA beside short requests; twice the same bits; the answer does not depend on what
    else is in the batch or in the workspace."""
    c = Cache([30000, 5, 3000], 2, D, 16, 16, 11, layers=1, layer=0).cuda()
    q = torch.randn((3, 8, D), generator=c.g).to(torch.bfloat16)
    out, ws = decode(c, q.cuda(), 0.06)
    again, _ = decode(c, q.cuda(), 0.06)
    ws[2048:].random_(0, 255)         # all but the header and the merge tickets
    third, _ = decode(c, q.cuda(), 0.06, ws=ws)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    assert torch.equal(out.view(torch.int16), third.view(torch.int16))
    check_decode(c, q, out, 0.06, f"long decode D={D}")


def test_decode_batch_of_many():
    """More segments than CTAs, most of them short."""
    g = gen(5)
    lens = [int(x) for x in torch.randint(0, 300, (500,), generator=g)]
    c = Cache(lens, 2, 64, 16, 16, 6, layers=1, layer=0).cuda()
    q = torch.randn((500, 4, 64), generator=c.g).to(torch.bfloat16)
    out, ws = decode(c, q.cuda(), 0.1)
    assert api.pa_get_error(ws) == 0
    check_decode(c, q, out, 0.1, "500 requests")


def test_decode_largest_batch():
    lens = [(i * 7) % 40 for i in range(4096)]
    c = Cache(lens, 1, 128, 4, 4, 9, layers=1, layer=0).cuda()
    q = torch.randn((4096, 16, 128), generator=c.g).to(torch.bfloat16)
    out, ws = decode(c, q.cuda(), 0.05)
    assert api.pa_get_error(ws) == 0
    check_decode(c, q, out, 0.05, "4096 requests", reqs=range(0, 4096, 97))


def test_decode_scales_far_apart():
    """Scales that differ by 2^60 within a request, for K (tiny ones, so that scores stay finite) and for V."""
    c = Cache([700, 130], 2, 128, 16, 16, 21, exp_lo=60, exp_hi=120)
    c.ve.add_(20)
    c.cuda()
    q = torch.randn((2, 8, 128), generator=c.g).to(torch.bfloat16)
    out, _ = decode(c, q.cuda(), 0.05)
    check_decode(c, q, out, 0.05, "far scales")


@pytest.mark.parametrize("G,Hkv,D,lens", [(1, 400, 64, [1, 300, 0, 129]), (1, 700, 128, [40, 200]), (16, 256, 64, [130])])
def test_decode_more_heads_than_workers(G, Hkv, D, lens):
    """Warpgroups that serve several kv heads one after the other; the most query heads."""
    c = Cache(lens, Hkv, D, 16, 16, Hkv, layers=1, layer=0).cuda()
    q = torch.randn((len(lens), Hkv * G, D), generator=c.g).to(torch.bfloat16)
    out, ws = decode(c, q.cuda(), 0.1)
    assert api.pa_get_error(ws) == 0
    check_decode(c, q, out, 0.1, f"{Hkv} kv heads")


@pytest.mark.parametrize("mag", [2.0 ** -100, 2.0 ** 90, "mixed"])
def test_decode_q_magnitudes(mag):
    """Queries far from 1, and heads whose elements differ by 2^20."""
    c = Cache([333], 1, 128, 16, 16, 22).cuda()
    q = torch.randn((1, 4, 128), generator=c.g)
    scale = 0.05
    if mag == "mixed":
        q = q * torch.pow(2.0, torch.randint(-20, 1, q.shape, generator=c.g).float())
    else:
        q, scale = q * mag, 0.05 / mag
    q = q.to(torch.bfloat16)
    out, _ = decode(c, q.cuda(), scale)
    check_decode(c, q, out, scale, f"q magnitude {mag}")


def test_decode_scale_zero_and_equal_weights():
    """scale 0: the mean of V, every weight the same (a bias of the weights' rounding would add up)."""
    c = Cache([5000, 4097], 2, 128, 16, 16, 23).cuda()
    q = torch.randn((2, 8, 128), generator=c.g).to(torch.bfloat16)
    out, _ = decode(c, q.cuda(), 0.0)
    check_decode(c, q, out, 0.0, "scale 0")


def test_decode_one_token_outweighs_all():
    """A score 60 binary orders above the others, in the first, a middle and the last tile."""
    for at in (0, 700, 1299):
        c = Cache([1300], 1, 128, 16, 16, 24)
        q = torch.randn((1, 4, 128), generator=c.g).to(torch.bfloat16)
        s = c.slots[0][at]
        c.k[1, s, 0] = torch.from_numpy(R.encode((q[0, 1].double() * 40).numpy()))
        c.ke[1, int(s) // 16] = 124
        c.cuda()
        out, _ = decode(c, q.cuda(), 0.4)
        check_decode(c, q, out, 0.4, f"one heavy token at {at}")


def test_decode_nan_stays_with_its_head_and_request():
    c = Cache([200, 200], 2, 128, 16, 16, 25)
    c.k[1, c.slots[0][77], 1, 5] = 127
    c.cuda()
    q = torch.randn((2, 8, 128), generator=c.g).to(torch.bfloat16)
    q[1, 2, 3] = math.nan
    q[1, 5, 3] = math.inf
    out, _ = decode(c, q.cuda(), 0.05)
    assert torch.isnan(out[0, 4:].float()).all() and torch.isnan(out[1, 2].float()).all() and torch.isnan(out[1, 5].float()).all()
    k, v = c.values(0)
    R.check_out(out[0, :4][None].cpu(), R.attention(q[0, :4][None].double(), k[:, :1], v[:, :1], 0.05), 12, "beside a NaN")


def test_decode_bad_indices_are_masked_and_flagged():
    c = Cache([300, 260, 10, 50], 1, 128, 16, 16, 26).cuda()
    q = torch.randn((4, 4, 128), generator=c.g).to(torch.bfloat16)
    c.dev[2][c.rows[0].item(), [0, 17, 150]] = torch.tensor([-1, c.size, 2 ** 30], dtype=torch.int32, device="cuda")
    c.dev[2][c.rows[1].item(), 128:256] = -7          # a tile without any row
    c.dev[3][2] = 99                                  # no such table row
    c.dlens[3] = -4
    out, ws = decode(c, q.cuda(), 0.05)
    assert api.pa_get_error(ws) == api.DEVERR_SLOT | api.DEVERR_ROW | api.DEVERR_LEN
    assert torch.count_nonzero(out[2:]) == 0
    for b, gone in ((0, [0, 17, 150]), (1, list(range(128, 256)))):
        keep = [j for j in range(c.lens[b]) if j not in gone]
        k, v = c.values(b)
        R.check_out(out[b][None].cpu(), R.attention(q[b][None].double(), k[keep], v[keep], 0.05), 12, f"masked {b}")
    # a length beyond the table is clamped
    c2 = Cache([100], 1, 64, 16, 16, 27, extra_ctx=0).cuda()
    c2.dlens.fill_(1000)
    q2 = torch.randn((1, 2, 64), generator=c2.g).to(torch.bfloat16)
    out2, ws2 = decode(c2, q2.cuda(), 0.1)
    assert api.pa_get_error(ws2) == api.DEVERR_LEN
    check_decode(c2, q2, out2, 0.1, "clamped length")


def test_decode_cache_beyond_32_bit_offsets():
    """A layer whose bytes start past 2^32, slots at both ends of it."""
    size, Hkv, D = 1 << 22, 8, 128
    k = torch.zeros((2, size, Hkv, D), dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    ke = torch.zeros((2, size // 16, Hkv), dtype=torch.uint8, device="cuda")
    ve = torch.zeros_like(ke)
    g = gen(31)
    n = 200
    slots = torch.cat([torch.arange(100), torch.arange(size - 100, size)]).int()
    x = [rows((n, Hkv, D), g) for _ in range(2)]
    api.pa_kv_store_fp8_block(k, v, 1, x[0].cuda(), x[1].cuda(), slots.cuda(), ke, ve, 16)
    wk = [np.zeros((256, Hkv, D), np.uint8) for _ in range(2)]
    we = [np.zeros((16, Hkv), np.uint8) for _ in range(2)]
    near = [int(s) if s < 112 else 112 + int(s) - (size - 112) for s in slots]
    for i in range(2):
        R.store(wk[i], we[i], x[i].double().numpy(), near, 16)
        same_bytes((k, v)[i][1][slots.long().cuda()].cpu().numpy(), wk[i][near], "stored rows")
    q = torch.randn((1, 32, D), generator=g).to(torch.bfloat16)
    ws = api.alloc_workspace(api.pa_decode_fp8_block_workspace_bytes(32, Hkv, D))
    out = torch.empty_like(q, device="cuda")
    api.pa_paged_decode_attn_fp8_block(q.cuda(), k, v, 1, slots[None].contiguous().cuda(), torch.zeros(1, dtype=torch.int32).cuda(),
                                       torch.tensor([n], dtype=torch.int32).cuda(), 0.09, ke, ve, 16, ws, out)
    vals = [R.values(torch.from_numpy(wk[i]), torch.from_numpy(we[i]), torch.tensor(near), 16) for i in range(2)]
    R.check_out(out.cpu(), R.attention(q.double(), *vals, 0.09), 12, "far layer")


def test_decode_streams_graphs_and_overlap():
    """Two graphs of one workspace replayed in turn, a stream of its own, and the launch-overlap modes: the same bits."""
    c = Cache([900, 4, 77], 2, 128, 16, 16, 41).cuda()
    d = Cache([40, 2000], 2, 128, 1, 1, 42).cuda()
    q1 = torch.randn((3, 8, 128), generator=c.g).to(torch.bfloat16).cuda()
    q2 = torch.randn((2, 8, 128), generator=c.g).to(torch.bfloat16).cuda()
    w1, ws = decode(c, q1, 0.05)
    w2, _ = decode(d, q2, 0.05)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o1, o2 = torch.empty_like(q1), torch.empty_like(q2)
    with torch.cuda.stream(s):
        decode(c, q1, 0.05, ws=ws, out=o1)
    s.synchronize()
    assert torch.equal(o1.view(torch.int16), w1.view(torch.int16))
    try:
        for mode in (api.OVERLAP_OFF, api.OVERLAP_SAFE, api.OVERLAP_EARLY_METADATA, api.OVERLAP_EARLY_KV):
            api.pa_set_launch_overlap(mode)
            graphs = []
            for cc, q, o in ((c, q1, o1), (d, q2, o2)):
                gr = torch.cuda.CUDAGraph()
                with torch.cuda.graph(gr):
                    decode(cc, q, 0.05, ws=ws, out=o)
                    decode(cc, q, 0.05, ws=ws, out=o)
                graphs.append(gr)
            for _ in range(3):
                o1.zero_()
                o2.zero_()
                graphs[0].replay()
                graphs[1].replay()
                torch.cuda.synchronize()
                assert torch.equal(o1.view(torch.int16), w1.view(torch.int16)), mode
                assert torch.equal(o2.view(torch.int16), w2.view(torch.int16)), mode
    finally:
        api.pa_set_launch_overlap(api.OVERLAP_OFF)


def test_decode_wait_limit_zero_aborts_and_recovers():
    c = Cache([3000, 10], 2, 128, 16, 16, 43).cuda()
    q = torch.randn((2, 8, 128), generator=c.g).to(torch.bfloat16).cuda()
    want, ws = decode(c, q, 0.05)
    try:
        api.pa_set_wait_timeout_ns(0)
        decode(c, q, 0.05, ws=ws)
        torch.cuda.synchronize()
    finally:
        api.pa_set_wait_timeout_ns(api.WAIT_TIMEOUT_DEFAULT_NS)
    assert api.pa_get_error(ws) & api.DEVERR_TIMEOUT
    api.pa_workspace_init(ws)
    out, _ = decode(c, q, 0.05, ws=ws)
    assert api.pa_get_error(ws) == 0 and torch.equal(out.view(torch.int16), want.view(torch.int16))


def test_store_then_decode_grows_with_the_request():
    """A request token by token: store, decode, the scale rising on the way."""
    Hkv, D, block = 2, 64, 16
    k, v = (torch.zeros((1, 64, Hkv, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    ke, ve = (torch.zeros((1, 4, Hkv), dtype=torch.uint8, device="cuda") for _ in range(2))
    wk, wv = (np.zeros((64, Hkv, D), np.uint8) for _ in range(2))
    wke, wve = (np.zeros((4, Hkv), np.uint8) for _ in range(2))
    slots = [16 + j for j in range(16)] + [48, 49, 50]
    table = torch.tensor([slots], dtype=torch.int32, device="cuda")
    g, zero = gen(8), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = api.alloc_workspace(api.pa_decode_fp8_block_workspace_bytes(4, Hkv, D))
    for j, s in enumerate(slots):
        x = [rows((1, Hkv, D), g) * (1 + j) for _ in range(2)]
        q = torch.randn((1, 4, D), generator=g).to(torch.bfloat16)
        api.pa_kv_store_fp8_block(k, v, 0, x[0].cuda(), x[1].cuda(), table[0, j:j + 1], ke, ve, block)
        R.store(wk, wke, x[0].double().numpy(), [s], block)
        R.store(wv, wve, x[1].double().numpy(), [s], block)
        out = torch.empty_like(q, device="cuda")
        api.pa_paged_decode_attn_fp8_block(q.cuda(), k, v, 0, table, zero, zero + j + 1, 0.1, ke, ve, block, ws, out)
        at = torch.tensor(slots[:j + 1])
        kk = R.values(torch.from_numpy(wk), torch.from_numpy(wke), at, block)
        vv = R.values(torch.from_numpy(wv), torch.from_numpy(wve), at, block)
        R.check_out(out.cpu(), R.attention(q.double(), kk, vv, 0.1), 12, f"after {j + 1} tokens")
    same_bytes(k[0].cpu().numpy(), wk, "k")


# ------------------------------------------------------------------ prefill

@pytest.mark.parametrize("G", [1, 4, 16])
@pytest.mark.parametrize("D,page,block", [(128, 16, 16), (64, 16, 16), (128, 1, 1), (64, 4, 4), (128, 64, 32)])
def test_prefill_ragged(G, D, page, block):
    new, pre = [1, 31, 130, 0, 300, 128], [0, 5, 300, 17, 257, 129]
    c = Cache([a + b for a, b in zip(new, pre)], 2, D, page, block, G + D + page).cuda()
    q = torch.randn((sum(new), 2 * G, D), generator=c.g).to(torch.bfloat16)
    qo = torch.tensor(np.cumsum([0] + new), dtype=torch.int32).cuda()
    kv = torch.tensor(np.cumsum([0] + c.lens), dtype=torch.int32).cuda()
    ws = api.alloc_workspace(api.pa_prefill_workspace_bytes())
    outs = []
    for _ in range(2):
        out = torch.full_like(q, math.nan, device="cuda")
        k, v, table, rws, ke, ve = c.dev
        api.pa_paged_prefill_attn_fp8_block(q.cuda(), k, v, c.layer, qo, kv, table, rws, 0.05, ke, ve, block, ws, out)
        outs.append(out)
    assert api.pa_get_error(ws) == 0
    assert torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16))
    at = 0
    for b, n in enumerate(new):
        if n:
            kk, vv = c.values(b)
            r = R.attention(q[at:at + n].double(), kk, vv, 0.05, first=pre[b], terms=2.0 ** -19)
            R.check_out(outs[0][at:at + n].cpu(), r, 8, f"prefill G={G} D={D} page={page} block={block} request {b}")
        at += n


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("scale,qmag", [(0.0, 1.0), (-0.05, 1.0), (0.05 * 2.0 ** -60, 2.0 ** 60), (0.4, 1.0)])
def test_prefill_scales_and_query_magnitudes(D, scale, qmag):
    """scale 0 (the mean of V), negative, queries far from 1, and scores that raise the maximum inside a tile."""
    c = Cache([390], 2, D, 16, 16, 62, exp_lo=100, exp_hi=124).cuda()
    q = (torch.randn((260, 8, D), generator=c.g) * torch.pow(2.0, torch.randint(-8, 1, (260, 8, 1), generator=c.g).float()) * qmag).to(torch.bfloat16)
    k, v, table, rws, ke, ve = c.dev
    out = torch.full_like(q, math.nan, device="cuda")
    ws = api.alloc_workspace(api.pa_prefill_workspace_bytes())
    api.pa_paged_prefill_attn_fp8_block(q.cuda(), k, v, 1, torch.tensor([0, 260], dtype=torch.int32).cuda(),
                                        torch.tensor([0, 390], dtype=torch.int32).cuda(), table, rws, scale, ke, ve, 16, ws, out)
    assert api.pa_get_error(ws) == 0
    kk, vv = c.values(0)
    R.check_out(out.cpu(), R.attention(q.double(), kk, vv, scale, first=130, terms=2.0 ** -19), 8, f"prefill scale {scale}")


def test_prefill_bad_slots_read_as_zeros():
    """A slot out of range is flagged; its position has a key and a value of zeros."""
    c = Cache([300], 1, 128, 16, 16, 63).cuda()
    q = torch.randn((40, 4, 128), generator=c.g).to(torch.bfloat16)
    k, v, table, rws, ke, ve = c.dev
    bad = [3, 150, 151, 290]
    table[c.rows[0].item(), bad] = torch.tensor([-1, c.size, 2 ** 30, -9], dtype=torch.int32, device="cuda")
    out = torch.full_like(q, math.nan, device="cuda")
    ws = api.alloc_workspace(api.pa_prefill_workspace_bytes())
    api.pa_paged_prefill_attn_fp8_block(q.cuda(), k, v, 1, torch.tensor([0, 40], dtype=torch.int32).cuda(),
                                        torch.tensor([0, 300], dtype=torch.int32).cuda(), table, rws, 0.05, ke, ve, 16, ws, out)
    assert api.pa_get_error(ws) == api.DEVERR_SLOT
    kk, vv = c.values(0)
    kk[bad], vv[bad] = 0.0, 0.0
    R.check_out(out.cpu(), R.attention(q.double(), kk, vv, 0.05, first=260, terms=2.0 ** -19), 8, "bad slots")


@pytest.mark.parametrize("exp,scale", [(0, 1e-20), (1, 1e-3), (1, 1e-30), (0, 0.0)])
@pytest.mark.parametrize("block", [16, 1])
def test_prefill_keys_of_the_smallest_scales(exp, scale, block):
    """Empty blocks (zeros) and scales of 2^-126: scores of nothing, hidden columns of diagonal tiles stay hidden, and
    each query sees the mean of its values."""
    c = Cache([200], 2, 128, 16, block, 64, exp_lo=118, exp_hi=120).cuda()
    c.ke[...] = exp
    c.dev[4] = c.ke.cuda()
    q = torch.randn((200, 8, 128), generator=c.g).to(torch.bfloat16)
    k, v, table, rws, ke, ve = c.dev
    out = torch.full_like(q, math.nan, device="cuda")
    ws = api.alloc_workspace(api.pa_prefill_workspace_bytes())
    api.pa_paged_prefill_attn_fp8_block(q.cuda(), k, v, 1, torch.tensor([0, 200], dtype=torch.int32).cuda(),
                                        torch.tensor([0, 200], dtype=torch.int32).cuda(), table, rws, scale, ke, ve, block, ws, out)
    assert api.pa_get_error(ws) == 0
    kk, vv = c.values(0)
    R.check_out(out.cpu(), R.attention(q.double(), kk, vv, scale, first=0, terms=2.0 ** -19), 8, f"exponent {exp}")


def test_prefill_last_row_is_decode_within_rounding():
    """The same cache and queries through both paths."""
    c = Cache([700], 2, 128, 16, 16, 61).cuda()
    q = torch.randn((1, 8, 128), generator=c.g).to(torch.bfloat16).cuda()
    out, _ = decode(c, q, 0.05)
    k, v, table, rws, ke, ve = c.dev
    pre = torch.empty_like(q)
    api.pa_paged_prefill_attn_fp8_block(q, k, v, 1, torch.tensor([0, 1], dtype=torch.int32).cuda(),
                                        torch.tensor([0, 700], dtype=torch.int32).cuda(), table, rws, 0.05, ke, ve, 16,
                                        api.alloc_workspace(api.pa_prefill_workspace_bytes()), pre)
    kk, vv = c.values(0)
    r = R.attention(q.cpu().double(), kk, vv, 0.05)
    R.check_out(out.cpu(), r, 12, "decode")
    R.check_out(pre.cpu(), R.attention(q.cpu().double(), kk, vv, 0.05, terms=2.0 ** -19), 8, "prefill")


def test_tensors_of_no_device_are_refused():
    c = Cache([20], 1, 64, 16, 16, 71).cuda()
    q = torch.zeros((1, 2, 64), dtype=torch.bfloat16, device="cuda")
    ws = api.alloc_workspace(api.pa_decode_fp8_block_workspace_bytes(2, 1, 64))
    with pytest.raises(TypeError, match="CUDA tensor"):
        api.pa_paged_decode_attn_fp8_block(q.cpu(), c.dev[0], c.dev[1], 1, c.dev[2], c.dev[3], c.dlens, 0.1, c.dev[4], c.dev[5],
                                           16, ws, q)
    with pytest.raises(ValueError, match="contiguous"):
        api.pa_paged_decode_attn_fp8_block(q, c.dev[0], c.dev[1], 1, c.dev[2][:, ::2], c.dev[3], c.dlens, 0.1, c.dev[4],
                                           c.dev[5], 16, ws, q)
    with pytest.raises(ValueError, match="ceil"):
        api.pa_paged_decode_attn_fp8_block(q, c.dev[0], c.dev[1], 1, c.dev[2], c.dev[3], c.dlens, 0.1, c.dev[4], c.dev[5],
                                           8, ws, q)
