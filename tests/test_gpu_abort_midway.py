"""Calls that give up midway: the wait limit set to times at which some waits of a
call run out and others do not, so that one part of a CTA gives up while another
still has copies on their way.  Each such call returns, and whatever runs on the
same SMs right behind it is right: nothing of the aborted call lands in its
shared memory."""
import math

import pytest
import torch

from paged_kv_cache_188_gb300 import api
from test_gpu_fp8_block import Cache, decode

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
