"""CPU checks of the drafted tokens' entry points: arguments are refused on the
host, before any launch, and the plain references the GPU tests use are pinned
by hand, against torch and against the distribution they must leave."""
import ctypes

import numpy as np
import pytest
import torch

import _spec_ref as S
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


def test_tree_refusals(lib):
    need = api.pa_tree_workspace_bytes(8, 2, 64)

    def call(q=FAKE, t=4, hq=8, s=None, layer=0, qo=FAKE, r=1, max_ctx=16, sl=FAKE, mask=FAKE, words=1, ke=0, ve=0, block=0,
             ws=FAKE, wsb=need, out=FAKE):
        return lib.pa_paged_tree_attn(ptr(q), t, hq, P(FAKE), P(FAKE), s or shape(), layer, ptr(qo), r, P(FAKE), 1, max_ctx,
                                      P(FAKE), ptr(sl), ptr(mask), words, 0.1, ptr(ke), ptr(ve), block, ptr(ws), wsb,
                                      ptr(out), None)
    assert call(t=-1) == 2 and call(r=-1) == 2 and call(r=4097) == 2 and call(hq=7) == 2 and call(layer=2) == 2
    assert call(layer=-1) == 2 and call(max_ctx=0) == 2 and call(block=48, ke=FAKE, ve=FAKE) == 2
    assert call(mask=0) == 2 and call(words=0) == 2 and call(words=-1) == 2       # a mask and its words go together
    assert call(ke=FAKE) == 2 and call(ve=FAKE) == 2                              # exponents with a bf16 cache
    assert call(t=2 ** 31 - 1, max_ctx=2 ** 31 - 200) == 2                        # tiles beyond 32 bits
    assert call(s=shape(d=96)) == 4 and call(hq=64) == 4
    assert call(q=0) == 1 and call(qo=0) == 1 and call(sl=0) == 1 and call(ws=0) == 1 and call(out=0) == 1
    assert call(block=16) == 1 and call(block=16, ke=FAKE) == 1
    assert call(q=FAKE + 4) == 3 and call(ws=FAKE + 16) == 3 and call(sl=FAKE + 1) == 3 and call(mask=FAKE + 2) == 3
    assert call(wsb=need - 1) == 5
    assert call(t=0, q=0, out=0) == 0 and call(r=0, qo=0) == 0


def test_tree_workspace(lib):
    assert api.pa_tree_workspace_bytes(0, 2, 64) == 0 and api.pa_tree_workspace_bytes(7, 2, 64) == 0
    assert 0 < api.pa_tree_workspace_bytes(32, 8, 128) <= 128 << 20


def test_verify_refusals(lib):
    def call(p=FAKE, f=0, v=100, tok=FAKE, par=FAKE, t=4, qo=FAKE, r=1, ua=FAKE, us=FAKE, acc=FAKE, mp=4, na=FAKE, nt=FAKE,
             err=0):
        return lib.pa_tree_verify(ptr(p), ptr(f), v, ptr(tok), ptr(par), t, ptr(qo), r, ptr(ua), ptr(us), ptr(acc), mp,
                                  ptr(na), ptr(nt), ptr(err), None)
    assert call(v=0) == 2 and call(v=2 ** 24 + 1) == 2 and call(t=-1) == 2 and call(r=-1) == 2 and call(r=65537) == 2
    assert call(mp=0) == 2 and call(mp=-1) == 2
    for name in ("p", "tok", "par", "qo", "ua", "us", "acc", "na", "nt"):
        assert call(**{name: 0}) == 1, name
    assert call(p=FAKE + 4) == 3 and call(f=FAKE + 8) == 3 and call(tok=FAKE + 2) == 3 and call(err=FAKE + 1) == 3
    assert call(r=0, p=0, qo=0) == 0


def test_accept_refusals(lib):
    def call(t=FAKE, rows=2, max_ctx=32, sl=FAKE, nt=4, r=1, acc=FAKE, mp=4, na=FAKE, nl=FAKE + 4096, fr=FAKE, k=0, v=0,
             s=None, eb=0, err=0):
        return lib.pa_kv_accept(ptr(t), rows, max_ctx, P(FAKE), ptr(sl), P(FAKE), nt, r, ptr(acc), mp, ptr(na), ptr(nl),
                                ptr(fr), ptr(k), ptr(v), s or shape(), eb, ptr(err), None)
    assert call(rows=0) == 2 and call(max_ctx=0) == 2 and call(nt=-1) == 2 and call(r=-1) == 2 and call(mp=0) == 2
    for name in ("t", "sl", "acc", "na", "nl", "fr"):
        assert call(**{name: 0}) == 1, name
    assert call(t=FAKE + 2) == 3 and call(err=FAKE + 2) == 3 and call(nl=FAKE + 1) == 3
    move = dict(k=FAKE, v=FAKE, eb=2)
    assert call(**dict(move, v=0)) == 1 and call(**dict(move, k=0)) == 1
    assert call(**dict(move, eb=4)) == 2 and call(**dict(move, s=shape(n_layers=0))) == 2
    assert call(**dict(move, nl=FAKE)) == 2                   # the lengths in place
    assert call(**dict(move, nl=FAKE + 8, r=3)) == 2          # or overlapping
    assert call(**dict(move, s=shape(hkv=1, d=4))) == 4       # rows of 8 bytes
    assert call(**dict(move, k=FAKE + 8)) == 3
    assert call(r=0, t=0) == 0 and call(**dict(move, r=0, t=0)) == 0


def test_wrappers_refuse_before_the_library(monkeypatch):
    monkeypatch.setattr(api, "_device", lambda: 0)
    u8 = torch.zeros((1, 32, 2, 64), dtype=torch.uint8)
    with pytest.raises(ValueError, match="needs k_exp"):
        api.pa_paged_tree_attn(None, u8, u8, 0, None, None, None, None, 0.1, None, None, block=16)
    with pytest.raises(TypeError, match="k_buf must be torch.bfloat16"):
        api.pa_paged_tree_attn(None, u8, u8, 0, None, None, None, None, 0.1, None, None)
    with pytest.raises(TypeError, match="CUDA tensor"):
        api.pa_tree_verify(torch.zeros((2, 4)), None, None, None, None, None, None, None, None)
    with pytest.raises(TypeError, match="target_probs must be torch.float32"):
        api.pa_tree_verify(torch.zeros((2, 4)).double(), None, None, None, None, None, None, None, None)
    with pytest.raises(TypeError, match="CUDA tensor"):
        api.pa_kv_accept(torch.zeros((1, 4), dtype=torch.int32), None, None, None, None, None, None, None)


# ------------------------------------------------ the references themselves

def test_reference_attention_matches_torch():
    g = torch.Generator().manual_seed(1)
    m, n, Hq, Hkv, D = 5, 12, 4, 2, 8
    q, k, v = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((m, Hq, D), (n, Hkv, D), (n, Hkv, D)))
    seen = S.tree_seen([-1, 0, 0, 1, 2])
    assert seen.tolist() == [[1, 0, 0, 0, 0], [1, 1, 0, 0, 0], [1, 0, 1, 0, 0], [1, 1, 0, 1, 0], [1, 0, 1, 0, 1]]
    full = torch.cat([torch.ones((m, n - m), dtype=torch.bool), seen], 1)
    want = torch.nn.functional.scaled_dot_product_attention(
        q.transpose(0, 1), k.repeat_interleave(2, 1).transpose(0, 1), v.repeat_interleave(2, 1).transpose(0, 1),
        attn_mask=full, scale=0.3).transpose(0, 1)
    assert torch.allclose(S.attention(q, k, v, 0.3, seen)["out"], want, atol=1e-12)
    # what is not seen does not matter, not even a NaN
    k[n - 2] = float("nan")
    got = S.attention(q, k, v, 0.3, seen)["out"]
    assert torch.isfinite(got[:3]).all() and torch.isnan(got[3]).any()


def test_reference_mask_words():
    seen = S.chain_seen(40)
    w = S.mask_words(seen, 2)
    assert w[31, 0] == -1 and w[31, 1] == 0 and w[39, 1] == 0xFF and w[0, 0] == 1


def test_reference_verify_by_hand():
    p = np.array([[0.5, 0.25, 0.25], [0.0, 1.0, 0.0], [0.25, 0.25, 0.5]], np.float32)
    f = np.array([[0.25, 0.5, 0.25]] * 3, np.float32)
    tree = [-1, 0, 0]
    # token 1 is kept where u * 0.5 < 0.25
    assert S.verify(p, f, [0, 1, 2], tree, [0, 0.49, 0], 0.5, 9) == ([0, 1], 1)
    # else what is left of w is [0.25, 0, 0], Z = 0.25: token 2 cannot be kept, token 0 follows
    assert S.verify(p, f, [0, 1, 2], tree, [0, 0.5, 0.0], 0.99, 9) == ([0], 0)
    # chosen tokens: 1 refused leaves Z = 0.75, then 2 is kept where u * 0.75 < 0.25
    assert S.verify(p, None, [0, 1, 2], tree, [0, 0.25, 0.33], 0.75, 9) == ([0, 2], 2)
    assert S.verify(p, None, [0, 1, 2], tree, [0, 0.25, 0.34], 0.99, 9) == ([0], 0)
    # a path that is full ends, whatever its children
    assert S.verify(p, f, [0, 1, 2], tree, [0, 0.0, 0], 0.5, 1) == ([0], 1)
    # no mass at all
    assert S.verify(np.zeros((1, 3), np.float32), None, [0], [-1], [0], 0.5, 9) == ([0], -1)
    # the draft is the target: a refusal (u rounded up to 1) leaves nothing, the target's row is drawn from
    assert S.verify(p[:2] * 0 + np.float32(1 / 3), p[:2] * 0 + np.float32(2 / 3), [0, 1], [-1, 0], [0, 0.9], 0.5, 9)[0] == [0]


@pytest.mark.parametrize("seed", range(6))
def test_reference_verify_in_fp32_and_in_rationals(seed):
    g = torch.Generator().manual_seed(seed)
    n, V = 9, 17
    par = S.random_parents(n, g)
    p, f = S.softmax_rows(n, V, g, 1.5), S.softmax_rows(n, V, g, 1.5)
    for _ in range(20):
        tok = torch.randint(V, (n,), generator=g).tolist()
        u, ul = torch.rand(n, generator=g).tolist(), float(torch.rand((), generator=g))
        for draft in (f, None):
            assert S.verify(p, draft, tok, par, u, ul, n) == S.verify_exact(p, draft, tok, par, u, ul)


@pytest.mark.parametrize("drawn", [True, False])
def test_reference_verify_leaves_the_targets_distribution(drawn):
    """The first token behind the root, kept or drawn, has the target's probabilities (chi-square, 5 sigma)."""
    g = torch.Generator().manual_seed(7)
    V, N = 4, 6000
    p = np.array([[0.45, 0.3, 0.2, 0.05]] * 3, np.float32)
    f = np.array([[0.1, 0.2, 0.3, 0.4]] * 3, np.float32)
    u, ul = torch.rand((N, 3), generator=g).numpy(), torch.rand(N, generator=g).numpy()
    draws = torch.multinomial(torch.from_numpy(f[0]), 2 * N, True, generator=g).view(N, 2).tolist()
    got = np.zeros(V)
    for i in range(N):
        tok = [0] + (draws[i] if drawn else [3, 1])
        path, after = S.verify(p, f if drawn else None, tok, [-1, 0, 0], u[i], ul[i], 3)
        got[tok[path[1]] if len(path) > 1 else after] += 1
    want = N * p[0].astype(np.float64)
    chi = ((got - want) ** 2 / want).sum()
    assert chi < 3 + 5 * np.sqrt(6), (got, want)


def test_reference_accept_by_hand():
    row = [10, 11, 12, 13, 14, 15, 99]
    assert S.accept(row, 2, 4, [0, 2]) == ([10, 11, 12, 14, 14, 15, 99], 4, [13, 15])
    assert S.accept_move(row, 2, 4, [0, 2]) == ([(12, 12), (14, 13)], 4, [14, 15])
