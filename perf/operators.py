"""Operators of a KV cache held in 8 bits and of a cache kept to a budget.

``store``    new K/V rows into an e4m3 cache whose scale is a power of two per (block of slots, kv head)
``decode``   one new token per request, attention over that cache through the page table
``prefill``  packed prompts after cached prefixes, causal attention over that cache
``weights``  decode attention that also adds each cached token's attention weight to a running table
``evict``    keeps the heaviest and the most recent tokens of each request, in the page table and the weights

``listed()`` and ``draw()`` give cases, ``prepare()`` their inputs on the GPU, ``run()`` one pass: in elementary
torch operations, or (``own``) by the library's calls.  ``exact()`` gives the results from the definitions in 64 bits.

The cache: bytes [layers, size, Hkv, D]; scale exponents [layers, size / block, Hkv], one byte e each, a row's value is
e4m3(byte) * 2^(e - 127); e = 0 is a block that nothing was stored in.
"""
import math
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn
MAX_E4M3 = 448.0
SINKS = 4          # first tokens that draw much attention, as measured in real models' heads


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the new tokens of 64 running requests, in blocks that are partly filled
        dict(name="store_append_64", op="store", T=64, Hkv=8, D=128, block=16, reset=False),
        # 8000 prompt tokens into pages handed out afresh
        dict(name="store_prompt_8000", op="store", T=8000, Hkv=8, D=128, block=16, reset=True),
        # one user, a short chat: latency
        dict(name="decode_1x1k", op="decode", B=1, n=1000, least=1000, Hq=32, Hkv=8, D=128, page=16, block=16),
        # one user, a long document
        dict(name="decode_1x32k", op="decode", B=1, n=32768, least=32768, Hq=32, Hkv=8, D=128, page=16, block=16),
        # a server's batch of mixed lengths
        dict(name="decode_48_ragged", op="decode", B=48, n=8192, least=500, Hq=32, Hkv=8, D=128, page=16, block=16),
        # token-granular pages, small heads, a scale for each token
        dict(name="decode_96_page1_d64", op="decode", B=96, n=4000, least=1, Hq=16, Hkv=2, D=64, page=1, block=1),
        # two short prompts behind a cached prefix
        dict(name="prefill_2_short", op="prefill", R=2, new=150, prefix=333, Hq=8, Hkv=2, D=64, page=16, block=16),
        # a packed batch of prompts, some with prefixes
        dict(name="prefill_16", op="prefill", R=16, new=2048, prefix=960, Hq=32, Hkv=8, D=128, page=16, block=16),
        # one user over a bf16 cache, weights kept for eviction
        dict(name="weights_1x8k_bf16", op="weights", B=1, n=8192, least=8192, Hq=32, Hkv=8, D=128, page=16, block=0),
        # a batch over the 8-bit cache, weights kept for eviction
        dict(name="weights_32_e4m3", op="weights", B=32, n=8192, least=700, Hq=32, Hkv=8, D=128, page=16, block=16),
        # one long request cut to a quarter
        dict(name="evict_1x32k", op="evict", B=1, n=32768, least=32768, budget=8192, recent=1024),
        # a batch brought back to its budget; requests below it stay as they are
        dict(name="evict_64_ragged", op="evict", B=64, n=16000, least=300, budget=2000, recent=333),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def draw(rng):
    op = rng.choice(["store", "decode", "prefill", "weights", "evict"])
    heads = rng.choice([(8, 2), (16, 2), (32, 8), (32, 2), (4, 4), (8, 1)])
    D = rng.choice([64, 128])
    block = rng.choice([1, 2, 4, 8, 16, 32, 64, 128])
    page = block * rng.choice([1, 1, 2])
    if op == "store":
        reset = rng.random() < 0.5
        return dict(op=op, T=_log(rng, 1, 7900 if reset else min(7900, 131072 // block)), Hkv=rng.choice([1, 2, 4, 7, 8]),
                    D=D, block=block, reset=reset)
    if op == "prefill":
        R = _log(rng, 1, 12)
        return dict(op=op, R=R, new=_log(rng, 1, 1700), prefix=rng.choice([0, rng.randint(1, 900)]), Hq=heads[0],
                    Hkv=heads[1], D=D, page=page, block=block)
    if op == "evict":
        B, n = _log(rng, 1, 48), _log(rng, 2, 16000)
        budget = rng.randint(1, n)
        return dict(op=op, B=B, n=n, least=max(1, n // rng.choice([1, 3, 40])), budget=budget,
                    recent=rng.randint(0, budget))
    bf16 = op == "weights" and rng.random() < 0.5
    B = _log(rng, 1, 40)
    n = _log(rng, 1, min(32000, (50000 if bf16 else 100000) // B))
    case = dict(op=op, B=B, n=n, least=max(1, n // rng.choice([1, 4, 50])), Hq=heads[0], Hkv=heads[1], D=D, page=page,
                block=block)
    if bf16:
        case["block"] = 0
        case["page"] = rng.choice([1, 16])
    return case


def _lens(n, least, B):
    """Lengths between `least` and n, the first one n, spread over their logarithm: the same for every seed."""
    rng = random.Random(n * 1000003 + B * 101 + least)
    return [n] + [_log(rng, least, n) for _ in range(B - 1)]


def _prompts(case):
    rng = random.Random(case["new"] * 7919 + case["R"] * 31 + case["prefix"])
    new = [case["new"]] + [_log(rng, max(1, case["new"] // 16), case["new"]) for _ in range(case["R"] - 1)]
    return new, [case["prefix"]] + [rng.randint(0, case["prefix"]) for _ in range(case["R"] - 1)]


# ----------------------------------------------------------------- inputs

class State:
    pass


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _table(lens, page, gen, rows_extra=3, max_ctx=None):
    """Slots of each request's tokens: whole pages in random order, rows of the table in random order, -1 behind
    the last token.  Returns (table, rows, size)."""
    B, dev = len(lens), "cuda"
    n = torch.tensor(lens, device=dev)
    pages = (n + page - 1) // page
    first = torch.cumsum(pages, 0) - pages
    n_pages = int(sum(-(-x // page) for x in lens)) + 8
    perm = torch.randperm(n_pages, generator=gen, device=dev)
    width = max_ctx or max(max(lens), 1)
    j = torch.arange(width, device=dev)
    p = (first[:, None] + j // page).clamp(max=n_pages - 1)
    slots = torch.where(j < n[:, None], perm[p] * page + j % page, -1)
    rows = torch.randperm(B + rows_extra, generator=gen, device=dev)[:B]
    table = torch.full((B + rows_extra, width), -1, dtype=torch.int32, device=dev)
    table[rows] = slots.to(torch.int32)
    return table, rows.to(torch.int32), n_pages * page


def _rows(shape, gen):
    """K or V rows: normal values, each token and head with a magnitude of its own."""
    x = torch.randn(shape, generator=gen, device="cuda")
    return (x * torch.exp(0.6 * torch.randn(shape[:-1], generator=gen, device="cuda"))[..., None]).to(torch.bfloat16)


def _need(amax):
    """Smallest exponent byte e with amax <= 448 * 2^(e - 127); 0 for an amax of 0."""
    m, e = torch.frexp(amax)
    return torch.where(amax > 0, (e + 118 + (m > 0.875)).clamp(1, 254), 0)


def _scale(e):
    """2^(e - 127) in fp32, from its bits (0 for e = 0): torch's own powers of two need not be exact on the GPU."""
    return (e.int() << 23).view(torch.float32)


def _encode(x, e):
    """Rows x in fp32 as e4m3 of x / 2^(e - 127): nearest even, saturating, NaN kept."""
    y = x * _scale(254 - e.int())[..., None]
    return y.clamp(-MAX_E4M3, MAX_E4M3).to(E4M3)


def _block_cache(size, Hkv, D, block, gen):
    """A full one-layer cache of `_rows`: bytes and scale exponents."""
    x = _rows((size, Hkv, D), gen).float()
    nb = -(-size // block)
    pad = torch.zeros((nb * block, Hkv), device="cuda")
    pad[:size] = x.abs().amax(-1)
    e = _need(pad.view(nb, block, Hkv).amax(1))
    b = _encode(x, e.repeat_interleave(block, 0)[:size])
    return b.view(torch.uint8)[None].contiguous(), e.to(torch.uint8)[None].contiguous()


def prepare(case, seed):
    gen, s, op = _gen(seed), State(), case["op"]
    s.op, s.block = op, case.get("block", 0)
    if op == "store":
        T, Hkv, D, block = case["T"], case["Hkv"], case["D"], case["block"]
        # an append: one token to each of T requests, the block's earlier rows there; a prompt: whole pages
        n_blocks = (T if not case["reset"] else -(-T // block)) + 5
        size = n_blocks * block
        perm = torch.randperm(n_blocks, generator=gen, device="cuda")
        if case["reset"]:
            t = torch.arange(T, device="cuda")
            s.loc = (perm[t // block] * block + t % block).to(torch.int32)
            s.fresh = perm[:-(-T // block)].to(torch.int32)
        else:
            s.loc = (perm[:T] * block + torch.randint(block, (T,), generator=gen, device="cuda")).to(torch.int32)
            s.fresh = None
        s.k, s.k_exp = _block_cache(size, Hkv, D, block, gen)
        s.v, s.v_exp = _block_cache(size, Hkv, D, block, gen)
        s.k_new, s.v_new = _rows((T, Hkv, D), gen), _rows((T, Hkv, D), gen)
        return s
    if op == "evict":
        lens = _lens(case["n"], case["least"], case["B"])
        s.table, s.rows, _ = _table(lens, 1, gen)
        s.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        # accumulated weights: many small, few large, ties among the untouched, the first tokens heavy
        w = torch.exp(2.5 * torch.randn(s.table.shape, generator=gen, device="cuda") - 4)
        w = torch.where(torch.rand(w.shape, generator=gen, device="cuda") < 0.1, 0.0, w)
        w[:, :SINKS] += 30.0
        s.weights = w
        s.budget, s.recent = case["budget"], case["recent"]
        s.new_lens = torch.empty_like(s.lens)
        s.freed = torch.full((case["B"], s.table.shape[1]), -1, dtype=torch.int32, device="cuda")
        return s
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
    s.scale = 1.0 / math.sqrt(D)
    if op == "prefill":
        new, pre = _prompts(case)
        s.new, s.pre = new, pre
        totals = [a + b for a, b in zip(new, pre)]
        s.table, s.rows, size = _table(totals, page, gen)
        cum = lambda v: torch.tensor([sum(v[:i]) for i in range(len(v) + 1)], dtype=torch.int32, device="cuda")  # noqa: E731
        s.qo, s.kv = cum(new), cum(totals)
        s.q = torch.randn((sum(new), Hq, D), generator=gen, device="cuda").to(torch.bfloat16)
        s.workspace = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    else:
        lens = _lens(case["n"], case["least"], case["B"])
        s.lens_host = lens
        s.table, s.rows, size = _table(lens, page, gen)
        s.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s.q = torch.randn((case["B"], Hq, D), generator=gen, device="cuda").to(torch.bfloat16)
        s.workspace = torch.zeros((64 << 20) + 4 * Hq * (sum(lens) + 64 * len(lens)), dtype=torch.uint8, device="cuda")
        s.weights = torch.rand(s.table.shape, generator=gen, device="cuda") if op == "weights" else None
    if s.block:
        s.k, s.k_exp = _block_cache(size, Hkv, D, s.block, gen)
        s.v, s.v_exp = _block_cache(size, Hkv, D, s.block, gen)
    else:
        s.k, s.v = _rows((1, size, Hkv, D), gen), _rows((1, size, Hkv, D), gen)
        s.k_exp = s.v_exp = None
    s.out = torch.empty_like(s.q)
    return s


# ------------------------------------------------------------------- runs

def run(s):
    if own:
        return _own(s)
    return {"store": _store, "evict": _evict, "prefill": _prefill, "decode": _decode, "weights": _decode}[s.op](s)


def _own(s):
    from paged_kv_cache_188_gb300 import api
    if s.op == "store":
        if s.fresh is not None:
            api.pa_kv_reset_fp8_block(s.k_exp, s.v_exp, s.fresh)
        api.pa_kv_store_fp8_block(s.k, s.v, 0, s.k_new, s.v_new, s.loc, s.k_exp, s.v_exp, s.block)
        return _cache_of(s)
    if s.op == "evict":
        api.pa_kv_evict(s.table, s.rows, s.lens, s.weights, s.budget, s.recent, s.new_lens, s.freed)
        return _evicted(s)
    if s.op == "prefill":
        api.pa_paged_prefill_attn_fp8_block(s.q, s.k, s.v, 0, s.qo, s.kv, s.table, s.rows, s.scale, s.k_exp, s.v_exp,
                                            s.block, s.workspace, s.out)
        return s.out
    if s.op == "decode":
        api.pa_paged_decode_attn_fp8_block(s.q, s.k, s.v, 0, s.table, s.rows, s.lens, s.scale, s.k_exp, s.v_exp,
                                           s.block, s.workspace, s.out)
        return s.out
    api.pa_paged_decode_attn_weights(s.q, s.k, s.v, 0, s.table, s.rows, s.lens, s.scale, s.weights, s.workspace, s.out,
                                     k_exp=s.k_exp, v_exp=s.v_exp, block=s.block)
    return {"out": s.out, "weights": s.weights}


def _cache_of(s):
    return {"k": s.k.view(E4M3), "v": s.v.view(E4M3), "k_exp": s.k_exp, "v_exp": s.v_exp}


def _evicted(s):
    return {"table": s.table, "weights": s.weights, "lens": s.new_lens, "freed": s.freed}


def _store(s):
    if s.fresh is not None:
        s.k_exp[:, s.fresh.long()] = 0
        s.v_exp[:, s.fresh.long()] = 0
    _store_rows(s.k[0], s.k_exp[0], s.k_new.float(), s.loc.long(), s.block)
    _store_rows(s.v[0], s.v_exp[0], s.v_new.float(), s.loc.long(), s.block)
    return _cache_of(s)


def _store_rows(buf, exp, x, loc, block):
    blocks, at = torch.unique(loc // block, return_inverse=True)
    amax = torch.where(x.isfinite(), x.abs(), 0.0).amax(-1)
    need = torch.zeros((blocks.numel(), x.shape[1]), device=x.device).index_reduce_(0, at, amax, "amax")
    old = exp[blocks].int()
    new = torch.maximum(old, _need(need))
    # earlier rows of a block whose scale grows are read back and rounded to the new scale
    slots = (blocks[:, None] * block + torch.arange(block, device=x.device)).flatten()
    rows = buf.view(E4M3)[slots].float().view(-1, block, *x.shape[1:])
    grown = ((old > 0) & (new > old))[:, None, :, None]
    again = _encode(rows * _scale(old)[:, None, :, None], new[:, None])
    was = buf[slots].view(-1, block, *x.shape[1:])
    buf[slots] = torch.where(grown, again.view(torch.uint8), was).flatten(0, 1)
    buf[loc] = _encode(x, new[at]).view(torch.uint8)
    exp[blocks] = new.to(torch.uint8)


def _values(buf, exp, slots, block):
    """Rows at `slots` (-1: zeros) in fp32."""
    at = slots.clamp(min=0).long()
    if exp is None:
        x = buf[0][at].float()
    else:
        x = buf[0].view(E4M3)[at].float() * _scale(exp[0][at // block])[..., None]
    return torch.where((slots >= 0)[..., None, None], x, 0.0)


def _decode(s):
    B, Hq, D = s.q.shape
    slots = s.table[s.rows.long()]                                  # -1 behind each request's last token
    k, v = _values(s.k, s.k_exp, slots, s.block), _values(s.v, s.v_exp, slots, s.block)
    Hkv = k.shape[2]
    live = (torch.arange(slots.shape[1], device=slots.device) < s.lens[:, None])[:, None, None]
    q = s.q.float().view(B, Hkv, Hq // Hkv, D)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * s.scale            # [B, Hkv, G, n]
    x = torch.where(live, x, -math.inf)
    p = torch.where(live, torch.exp(x - x.amax(-1, keepdim=True)), 0.0)
    p = p / p.sum(-1, keepdim=True).clamp(min=0.5)                  # 1 or more where anything is live
    out = torch.matmul(p, v.permute(0, 2, 1, 3)).view(B, Hq, D).to(torch.bfloat16)
    if s.op == "decode":
        return out
    s.weights[s.rows.long()] += p.sum((1, 2))
    return {"out": out, "weights": s.weights}


def _prefill(s):
    T, Hq, D = s.q.shape
    R, most = len(s.new), max(s.new)
    slots = s.table[s.rows.long()]
    k, v = _values(s.k, s.k_exp, slots, s.block), _values(s.v, s.v_exp, slots, s.block)
    Hkv, n = k.shape[2], slots.shape[1]
    count = (s.qo[1:] - s.qo[:-1]).long()
    prefix = (s.kv[1:] - s.kv[:-1]).long() - count
    i = torch.arange(most, device=s.q.device)
    valid = i < count[:, None]                                      # [R, most]
    q = s.q[(s.qo[:-1].long()[:, None] + i).clamp(max=T - 1)].float()
    q = q.view(R, most, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(R, Hkv, -1, D)
    x = (torch.matmul(q, k.permute(0, 2, 3, 1)) * s.scale).view(R, Hkv, -1, most, n)
    seen = torch.arange(n, device=s.q.device) <= (prefix[:, None] + i)[..., None]
    x = torch.where(seen[:, None, None], x, -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    del x
    p = p / p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(R, Hkv, -1, n), v.permute(0, 2, 1, 3)).view(R, Hkv, Hq // Hkv, most, D)
    return out.permute(0, 3, 1, 2, 4).reshape(R, most, Hq, D)[valid].to(torch.bfloat16)


def _evict(s):
    rows, n = s.rows.long(), s.lens.long()
    slots, w = s.table[rows], s.weights[rows]
    j = torch.arange(slots.shape[1], device=slots.device)
    live, cut = j < n[:, None], n > s.budget
    key = torch.where(w.isnan(), -math.inf, w).clamp(max=torch.finfo(torch.float32).max)
    key = torch.where(j >= (n - s.recent)[:, None], math.inf, key)
    # live tokens before the others; ties go to the lowest position
    order = torch.sort(key, dim=1, descending=True, stable=True).indices
    order = order.gather(1, torch.sort(live.gather(1, order).int(), dim=1, descending=True, stable=True).indices)
    rank = torch.empty_like(order).scatter_(1, order, j.expand_as(order))
    keep = live & ((rank < s.budget) | ~cut[:, None])
    to = torch.cumsum(keep, 1) - 1
    b = torch.arange(len(rows), device=rows.device)[:, None].expand_as(keep)
    table, weights = slots.clone(), torch.where(live & cut[:, None], 0.0, w)
    table[b[keep], to[keep]] = slots[keep]
    weights[b[keep], to[keep]] = w[keep]
    gone = live & ~keep
    s.freed[b[gone], (torch.cumsum(gone, 1) - 1)[gone]] = slots[gone]
    s.table[rows], s.weights[rows] = table, weights
    s.new_lens.copy_(torch.where(cut, s.budget, n))
    return _evicted(s)


# ------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "store":
        row = case["Hkv"] * case["D"]
        blocks = case["T"] if not case["reset"] else -(-case["T"] // case["block"])
        return {"bytes": 2 * case["T"] * row * 3 + 4 * case["T"] + 4 * blocks * case["Hkv"], "flops": 4 * case["T"] * row}
    if op == "evict":
        lens = _lens(case["n"], case["least"], case["B"])
        kept = [min(n, case["budget"]) for n in lens]
        cut = [n for n in lens if n > case["budget"]]
        # table and weights read; those kept written, the weights behind them zeroed, the freed slots listed
        moved = 8 * sum(cut) + 8 * case["budget"] * len(cut) + 8 * sum(n - case["budget"] for n in cut)
        return {"bytes": moved + 16 * len(kept), "flops": 2 * sum(cut)}
    per = case["D"] * 2 + (2.0 / case["block"] if case["block"] else case["D"] * 2)
    if op == "prefill":
        new, pre = _prompts(case)
        keys = sum(new) + sum(pre)
        pairs = sum(n * p + n * (n + 1) // 2 for n, p in zip(new, pre))
        return {"bytes": keys * (case["Hkv"] * per + 4) + 4 * sum(new) * case["Hq"] * case["D"],
                "flops": 4 * case["D"] * case["Hq"] * pairs}
    total = sum(_lens(case["n"], case["least"], case["B"]))
    extra = 8 * total if op == "weights" else 0
    return {"bytes": total * (case["Hkv"] * per + 4) + 4 * case["B"] * case["Hq"] * case["D"] + 8 * case["B"] + extra,
            "flops": 4 * total * case["Hq"] * case["D"]}


# ------------------------------------------------------------------ exact

def _two(k):
    """2^k in doubles, exact, for whole numbers k of magnitude up to 320."""
    powers = torch.tensor([2.0 ** i for i in range(-320, 321)], dtype=torch.float64, device=k.device)
    return powers[k.long() + 320]


def _value64(codes):
    """e4m3 bytes as doubles, from the format: sign, 4 exponent bits (bias 7), 3 bits of mantissa."""
    c = codes.long()
    e, m = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * _two(e - 10))
    return torch.where((c & 127) == 127, math.nan, torch.where(c >= 128, -mag, mag))


def _round64(x):
    """Doubles to the nearest e4m3 value, ties to even, saturating."""
    a = x.abs().clamp(max=448.0)
    step = _two(torch.frexp(a.clamp(min=2.0 ** -6)).exponent - 4)
    return torch.copysign(torch.round(a / step) * step, x)


def _exact_store(case, seed):
    s = prepare(case, seed)
    got = {}
    for name, buf, exp, new in (("k", s.k[0], s.k_exp[0], s.k_new), ("v", s.v[0], s.v_exp[0], s.v_new)):
        e = exp.double()
        if s.fresh is not None:
            e[s.fresh.long()] = 0
        loc, block = s.loc.long(), s.block
        top = torch.zeros_like(e)
        for r in range(block):                                     # the slots of a call differ: one row of a block at a time
            at = (loc % block == r).nonzero()[:, 0]
            top[loc[at] // block] = torch.maximum(top[loc[at] // block], new[at].double().abs().amax(-1))
        want = torch.where(top > 0, (torch.frexp(top / 448.0).exponent - (torch.frexp(top / 448.0).mantissa == 0.5).int()) + 127, 0.0).clamp(0, 254)
        want = torch.maximum(e, torch.where(top > 0, want.clamp(min=1), want))
        val = _value64(buf)
        old = e.repeat_interleave(block, 0)[:buf.shape[0], :, None]
        now = want.repeat_interleave(block, 0)[:buf.shape[0], :, None]
        val = torch.where((old > 0) & (now > old), _round64(val * _two(old - now)), val)
        val[loc] = _round64(new.double() / _two(now[loc] - 127))
        got[name] = val[None]
    return {"k": got["k"], "v": got["v"], "k_exp": None, "v_exp": None}


def _rows64(buf, exp, slots, block):
    at = slots.long()
    if exp is None:
        return buf[0][at].double()
    return _value64(buf[0][at]) * _two(exp[0][at // block].int() - 127)[..., None]


def exact(case, seed):
    if case["op"] == "store":
        return _exact_store(case, seed)
    if case["op"] == "evict":
        return None                                                # table entries and moved numbers: nothing is computed
    s = prepare(case, seed)
    out = torch.zeros(s.q.shape, dtype=torch.float64, device="cuda")
    weights = s.weights.double() if s.op == "weights" else None
    for b, row in enumerate(s.rows.tolist()):
        n = s.new[b] + s.pre[b] if s.op == "prefill" else s.lens_host[b]
        k = _rows64(s.k, s.k_exp, s.table[row, :n], s.block)
        v = _rows64(s.v, s.v_exp, s.table[row, :n], s.block)
        lo = int(s.qo[b]) if s.op == "prefill" else b
        m = s.new[b] if s.op == "prefill" else 1
        q = s.q[lo:lo + m].double()
        G = q.shape[1] // k.shape[1]
        hidden = torch.arange(n, device="cuda") > torch.arange(n - m, n, device="cuda")[:, None]
        for h in range(q.shape[1]):
            x = (q[:, h] @ k[:, h // G].T) * s.scale
            p = torch.softmax(x.masked_fill(hidden, -math.inf), -1)
            out[lo:lo + m, h] = p @ v[:, h // G]
            if weights is not None:
                weights[row, :n] += p[0]
    return {"out": out, "weights": weights} if weights is not None else out
