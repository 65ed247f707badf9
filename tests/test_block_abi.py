"""CPU checks of the block-scaled cache, attention-weight and eviction entry
points: arguments are refused on the host, before any launch, and the plain
64-bit reference the GPU tests use is pinned against torch and by hand."""
import ctypes
import math

import numpy as np
import pytest
import torch

import _block_ref as R
from paged_kv_cache_188_gb300 import api
from paged_kv_cache_188_gb300 import build as B

FAKE = 0x10000000
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    B.build()
    return api.lib()


def shape(size=64, hkv=2, d=64, n_layers=2):
    return api.KvShape(n_layers, size, hkv, d)


def ptr(x):
    return P(x) if x else None


def test_store_refusals(lib):
    def call(s=None, layer=0, k=FAKE, ke=FAKE, ve=FAKE, block=16, n=4, loc=FAKE, err=0):
        return lib.pa_kv_store_fp8_block(ptr(k), P(FAKE), s or shape(), layer, P(FAKE), P(FAKE), ptr(loc), n, ptr(ke),
                                         ptr(ve), block, ptr(err), None)
    assert call(layer=2) == 2 and call(layer=-1) == 2 and call(n=-1) == 2
    for block in (0, -1, 3, 24, 256):
        assert call(block=block) == 2
    assert call(s=shape(d=96)) == 4
    assert call(k=0) == 1 and call(ke=0) == 1 and call(ve=0) == 1 and call(loc=0) == 1
    assert call(k=FAKE + 8) == 3 and call(loc=FAKE + 2) == 3 and call(err=FAKE + 1) == 3
    assert call(n=0, k=0, ke=0) == 0


def test_reset_refusals(lib):
    call = lambda nl=2, nb=4, h=2, n=1, ke=FAKE, bl=FAKE, err=0: lib.pa_kv_reset_fp8_block(  # noqa: E731
        ptr(ke), P(FAKE), nl, nb, h, ptr(bl), n, ptr(err), None)
    assert call(nl=0) == 2 and call(nb=0) == 2 and call(h=0) == 2 and call(n=-1) == 2
    assert call(ke=0) == 1 and call(bl=0) == 1
    assert call(bl=FAKE + 2) == 3 and call(err=FAKE + 2) == 3
    assert call(n=0, ke=0) == 0


def test_decode_refusals(lib):
    need = api.pa_decode_fp8_block_workspace_bytes(8, 2, 64)

    def call(q=FAKE, batch=1, hq=8, s=None, layer=0, max_ctx=16, ke=FAKE, block=16, ws=FAKE, wsb=need, out=FAKE, sl=FAKE):
        return lib.pa_paged_decode_attn_fp8_block(ptr(q), batch, hq, P(FAKE), P(FAKE), s or shape(), layer, P(FAKE), 1,
                                                  max_ctx, P(FAKE), ptr(sl), 0.1, ptr(ke), P(FAKE), block, ptr(ws), wsb,
                                                  ptr(out), None)
    assert call(batch=-1) == 2 and call(batch=4097) == 2 and call(hq=7) == 2 and call(layer=2) == 2
    assert call(max_ctx=0) == 2 and call(block=0) == 2 and call(block=48) == 2
    assert call(batch=4096, max_ctx=2 ** 30) == 2             # tiles beyond 32 bits
    assert call(s=shape(d=96)) == 4 and call(hq=64) == 4
    big = api.KvShape(1, 64, 4097, 64)                        # more query heads than are supported
    assert call(s=big, hq=4097, wsb=1 << 40) == 4
    assert call(q=0) == 1 and call(ke=0) == 1 and call(ws=0) == 1 and call(out=0) == 1
    assert call(q=FAKE + 4) == 3 and call(ws=FAKE + 16) == 3 and call(sl=FAKE + 1) == 3
    assert call(wsb=need - 1) == 5
    assert call(batch=0, q=0, ke=0) == 0


def test_weights_refusals(lib):
    need = api.pa_decode_weights_workspace_bytes(1, 128, 8, 2, 64)

    def call(batch=1, ke=0, ve=0, block=0, w=FAKE, wsb=need):
        return lib.pa_paged_decode_attn_weights(P(FAKE), batch, 8, P(FAKE), P(FAKE), shape(), 0, P(FAKE), 1, 16, P(FAKE),
                                                P(FAKE), 0.1, ptr(ke), ptr(ve), block, ptr(w), P(FAKE), wsb, P(FAKE), None)
    assert call(w=0) == 1 and call(w=FAKE + 2) == 3
    assert call(ke=FAKE) == 2 and call(ve=FAKE) == 2          # exponents with a bf16 cache
    assert call(block=16) == 1 and call(block=16, ke=FAKE) == 1
    assert call(block=3, ke=FAKE, ve=FAKE) == 2
    assert call(batch=64) == 5                                # not one tile per request
    assert call(wsb=api.pa_decode_fp8_block_workspace_bytes(8, 2, 64)) == 5
    assert call(batch=0, w=0) == 0


def test_workspace_sizes(lib):
    assert api.pa_decode_fp8_block_workspace_bytes(0, 2, 64) == 0
    assert api.pa_decode_fp8_block_workspace_bytes(7, 2, 64) == 0
    small = api.pa_decode_weights_workspace_bytes(1, 1, 32, 8, 128)
    assert small >= api.pa_decode_fp8_block_workspace_bytes(32, 8, 128) + 32 * 128 * 4
    assert api.pa_decode_weights_workspace_bytes(64, 10 ** 6, 32, 8, 128) > small + 10 ** 6 * 32 * 4
    assert api.pa_decode_weights_workspace_bytes(-1, 0, 32, 8, 128) == 0


def test_prefill_refusals(lib):
    wsb = api.pa_prefill_workspace_bytes()

    def call(d=128, hq=8, ke=FAKE, block=16, n=10):
        return lib.pa_paged_prefill_attn_fp8_block(P(FAKE), n, hq, P(FAKE), P(FAKE), shape(d=d), 0, P(FAKE), P(FAKE), 1,
                                                   P(FAKE), 1, 16, P(FAKE), 0.1, ptr(ke), P(FAKE), block, P(FAKE), wsb,
                                                   P(FAKE), None)
    assert call(d=96) == 4 and call(hq=6) == 4 and call(hq=7) == 2 and call(block=5) == 2
    assert call(ke=0) == 1
    assert call(n=0, ke=0) == 0


def test_evict_refusals(lib):
    def call(batch=1, max_ctx=64, budget=8, recent=2, t=FAKE, w=FAKE, nl=FAKE, fr=FAKE, err=0):
        return lib.pa_kv_evict(ptr(t), 4, max_ctx, P(FAKE), P(FAKE), batch, ptr(w), budget, recent, ptr(nl), ptr(fr),
                               ptr(err), None)
    assert call(batch=-1) == 2 and call(budget=0) == 2 and call(recent=-1) == 2 and call(recent=9) == 2
    assert call(max_ctx=2 ** 31 - 1) == 2
    assert call(t=0) == 1 and call(w=0) == 1 and call(nl=0) == 1 and call(fr=0) == 1
    assert call(w=FAKE + 2) == 3 and call(err=FAKE + 2) == 3
    assert call(batch=0, t=0) == 0


def test_wrappers_refuse_before_the_library(monkeypatch):
    monkeypatch.setattr(api, "_device", lambda: 0)
    u8 = torch.zeros((1, 32, 2, 64), dtype=torch.uint8)
    e = torch.zeros((1, 2, 2), dtype=torch.uint8)
    with pytest.raises(TypeError, match="uint8 or float8_e4m3fn"):
        api.pa_kv_store_fp8_block(u8.bfloat16(), u8.bfloat16(), 0, None, None, None, e, e, 16)
    with pytest.raises(TypeError, match="CUDA tensor"):
        api.pa_kv_store_fp8_block(u8, u8, 0, None, None, None, e, e, 16)
    with pytest.raises(ValueError, match="power of two"):
        api.pa_kv_store_fp8_block(u8, u8, 0, None, None, None, e, e, 12)
    with pytest.raises(TypeError, match="CUDA tensor"):
        api.pa_kv_evict(torch.zeros((1, 4), dtype=torch.int32), None, None, None, 1, 0, None, None)
    with pytest.raises(ValueError, match="needs k_exp"):
        api.pa_paged_decode_attn_weights(None, u8, u8, 0, None, None, None, 0.1, None, None, None, block=16)


# ------------------------------------------------ the reference itself

def test_reference_codes_match_torch():
    codes = torch.arange(256).to(torch.uint8)
    t = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(t), np.isnan(R.E4M3)) and np.array_equal(t[~np.isnan(t)], R.E4M3[~np.isnan(t)])
    x = torch.cat([torch.randn(20000, generator=torch.Generator().manual_seed(1)) * 60,
                   torch.tensor(R.E4M3[:126]), torch.tensor((R.E4M3[:125] + R.E4M3[1:126]) / 2)]).clamp(-448, 448)
    want = x.to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.encode(x.to(torch.float32).double().numpy()), want)


def test_reference_exponents_by_hand():
    assert [R.need(a) for a in (0.0, 448.0, 449.0, 224.0, 225.0, 896.0, 3.5, 3.515625)] == [0, 127, 128, 126, 127, 128, 120, 121]
    assert R.need(2.0 ** -149) == 1


def test_reference_store_by_hand():
    buf, exp = np.zeros((4, 1, 2), np.uint8), np.zeros((2, 1), np.uint8)
    R.store(buf, exp, np.array([[[448.0, 1.0]]]), [0], 2)
    assert exp[0, 0] == 127 and list(R.E4M3[buf[0, 0]]) == [448.0, 1.0]
    # a row twice as large: the scale doubles, the earlier row is kept at half its codes
    R.store(buf, exp, np.array([[[896.0, -3.0]]]), [1], 2)
    assert exp[0, 0] == 128 and list(R.E4M3[buf[0, 0]]) == [224.0, 0.5] and list(R.E4M3[buf[1, 0]]) == [448.0, -1.5]
    assert exp[1, 0] == 0


def test_reference_evict_by_hand():
    nan = math.nan
    assert R.evict([9, 8, 7, 6, 5], [1.0, 3.0, nan, 3.0, 0.0], 3, 1) == ([8, 6, 5], [3.0, 3.0, 0.0], [9, 7])
    assert R.evict([9, 8, 7], [2.0, 2.0, 2.0], 1, 0) == ([9], [2.0], [8, 7])
    assert R.evict([9, 8], [1.0, 2.0], 2, 2) == ([9, 8], [1.0, 2.0], [])
