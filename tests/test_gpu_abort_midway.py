"""Calls that give up midway: the wait limit set to times at which some waits of a
call run out and others do not, so that one part of a CTA gives up while another
still has copies on their way.  Each such call returns, and whatever runs on the
same SMs right behind it is right: nothing of the aborted call lands in its
shared memory."""
import math

import numpy as np
import pytest
import torch

from paged_kv_cache_188_gb300 import api
from paged_kv_cache_188_gb300 import workloads as W
from test_gpu_fp8_block import Cache, decode
from test_gpu_weights_evict import Bf16Cache, weights_call

pytestmark = pytest.mark.gpu
LIMITS_NS = [0, 1, 300, 1000, 2000, 3000, 5000, 8000, 12000, 20000]


@pytest.fixture(autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.lib()
    yield
    api.pa_set_wait_timeout_ns(api.WAIT_TIMEOUT_DEFAULT_NS)


def bits(t):
    return t.view(torch.int16)


def _drive(call, want, alloc):
    """For each limit: the call with that limit, and behind it, without a wait between them, the same call with the
    default limit and a workspace of its own.  `call(ws, out)`."""
    gave_up = 0
    for limit in LIMITS_NS:
        ws1, ws2 = alloc(), alloc()
        out1, out2 = torch.full_like(want, math.nan), torch.full_like(want, math.nan)
        torch.cuda.synchronize()
        try:
            api.pa_set_wait_timeout_ns(limit)
            call(ws1, out1)
        finally:
            api.pa_set_wait_timeout_ns(api.WAIT_TIMEOUT_DEFAULT_NS)
        call(ws2, out2)
        torch.cuda.synchronize()
        assert api.pa_get_error(ws2) == 0
        assert torch.equal(bits(out2), bits(want)), f"the call behind one with a limit of {limit} ns"
        err = api.pa_get_error(ws1)
        assert err in (0, api.DEVERR_TIMEOUT)
        if err == 0:
            assert torch.equal(bits(out1), bits(want)), f"limit {limit} ns, nothing reported"
        gave_up += err != 0
        # the workspace of the aborted call, initialised again
        api.pa_workspace_init(ws1)
        call(ws1, out1)
        torch.cuda.synchronize()
        assert api.pa_get_error(ws1) == 0 and torch.equal(bits(out1), bits(want))
    assert gave_up > 0


@pytest.mark.parametrize("D,page,block", [(128, 16, 16), (128, 1, 1), (64, 2, 2)])
def test_block_decode(D, page, block):
    g = torch.Generator().manual_seed(D + page)
    lens = [int(x) for x in torch.randint(1, 2500, (24,), generator=g)]
    c = Cache(lens, 4, D, page, block, 51, layers=1, layer=0).cuda()
    q = torch.randn((len(lens), 16, D), generator=c.g).to(torch.bfloat16).cuda()
    want, _ = decode(c, q, 0.05)
    need = api.pa_decode_fp8_block_workspace_bytes(16, 4, D)
    _drive(lambda ws, out: decode(c, q, 0.05, ws=ws, out=out), want, lambda: api.alloc_workspace(need))


@pytest.mark.parametrize("kind", ["block", "e4m3", "bf16"])
@pytest.mark.parametrize("D", [128, 64])
def test_prefill(kind, D):
    new, pre = [300, 77, 700, 5], [500, 0, 64, 3]
    need = api.pa_prefill_workspace_bytes()
    if kind == "block":
        c = Cache([a + b for a, b in zip(new, pre)], 2, D, 16, 16, 52).cuda()
        q = torch.randn((sum(new), 8, D), generator=c.g).to(torch.bfloat16).cuda()
        qo = torch.tensor(np.cumsum([0] + new), dtype=torch.int32).cuda()
        kv = torch.tensor(np.cumsum([0] + c.lens), dtype=torch.int32).cuda()
        k, v, table, rws, ke, ve = c.dev

        def call(ws, out):
            api.pa_paged_prefill_attn_fp8_block(q, k, v, c.layer, qo, kv, table, rws, 0.05, ke, ve, 16, ws, out)
    else:
        pb = W.make_prefill_batch(new_lens=new, prefix_lens=pre, n_q_heads=8, n_kv_heads=2, head_dim=D, size=2048,
                                  page_size=16, seed=53, device="cuda")
        q = pb.q
        args = (pb.qo_indptr, pb.kv_indptr, pb.kv.req_to_token, pb.kv.req_pool_indices, pb.scale)
        if kind == "bf16":
            api.pa_kv_store(pb.kv.k_buf, pb.kv.v_buf, pb.layer, pb.k_new, pb.v_new, pb.loc)

            def call(ws, out):
                api.pa_paged_prefill_attn(q, pb.kv.k_buf, pb.kv.v_buf, pb.layer, *args, ws, out)
        else:
            n_layers, size, Hkv, _ = pb.kv.k_buf.shape
            ks = torch.full((n_layers, Hkv), 4.5 / 448, dtype=torch.float32, device="cuda")
            k8 = torch.zeros((n_layers, size, Hkv, D), dtype=torch.uint8, device="cuda")
            v8 = torch.zeros_like(k8)
            every = torch.arange(size, dtype=torch.int32, device="cuda")
            api.pa_kv_store_fp8(k8, v8, pb.layer, pb.kv.k_buf[pb.layer], pb.kv.v_buf[pb.layer], every, ks, ks)
            api.pa_kv_store_fp8(k8, v8, pb.layer, pb.k_new, pb.v_new, pb.loc, ks, ks)

            def call(ws, out):
                api.pa_paged_prefill_attn_fp8(q, k8, v8, pb.layer, *args, ks, ks, ws, out)
    want = torch.empty_like(q)
    call(api.alloc_workspace(need), want)
    _drive(call, want, lambda: api.alloc_workspace(need))


@pytest.mark.parametrize("bf16", [True, False])
def test_weights_table_of_an_aborted_call(bf16):
    """A call that gave up adds nothing to the table, and neither does one on its workspace before that is initialised
    again; then the same call is right."""
    lens = [3000, 40, 777, 0, 1500]
    c = (Bf16Cache(lens, 2, 128, 16, 54) if bf16 else Cache(lens, 2, 128, 16, 16, 54)).cuda()
    q = torch.randn((len(lens), 8, 128), generator=c.g).to(torch.bfloat16).cuda()
    w0 = torch.rand(c.table.shape, generator=c.g).cuda()
    w1 = w0.clone()
    want, _ = weights_call(c, q, 0.05, w1)
    assert not torch.equal(w1, w0)
    need = api.pa_decode_weights_workspace_bytes(len(lens), sum(lens), 8, 2, 128)
    gave_up = 0
    for limit in LIMITS_NS:
        ws, w, out = api.alloc_workspace(need), w0.clone(), torch.full_like(want, math.nan)
        torch.cuda.synchronize()
        try:
            api.pa_set_wait_timeout_ns(limit)
            weights_call(c, q, 0.05, w, ws=ws, out=out)
        finally:
            api.pa_set_wait_timeout_ns(api.WAIT_TIMEOUT_DEFAULT_NS)
        torch.cuda.synchronize()
        err = api.pa_get_error(ws)
        assert err in (0, api.DEVERR_TIMEOUT) and (limit > 0 or err)
        if err:
            gave_up += 1
            assert torch.equal(w, w0), f"limit {limit} ns: the table changed"
            # entries of the score and log-sum-exp areas are the aborted call's, whatever they are
            weights_call(c, q, 0.05, w, ws=ws, out=out)
            torch.cuda.synchronize()
            assert torch.equal(w, w0) and api.pa_get_error(ws) == api.DEVERR_TIMEOUT
            api.pa_workspace_init(ws)
            weights_call(c, q, 0.05, w, ws=ws, out=out)
            torch.cuda.synchronize()
            assert api.pa_get_error(ws) == 0
        assert torch.equal(w, w1) and torch.equal(bits(out), bits(want)), f"limit {limit} ns"
    assert gave_up > 0
