"""Operators of a speculative decoding step over a paged KV cache.

``tree``     attention of each request's drafted tokens (a tree, or a chain) over its cached tokens and over the drafted
             ones that its mask lets it see, bf16 cache or e4m3 cache with a power-of-two scale per (block of slots, head)
``verify``   which of the drafted tokens are kept, from the target's (and the draft's) probabilities and given random
             numbers, and the token that follows them
``accept``   the kept tokens' slots move up behind the context and the others are handed back: in the page table, or
             by moving the K/V rows of every layer

``listed()`` and ``draw()`` give cases, ``prepare()`` their inputs on the GPU, ``run()`` one pass: in elementary
torch operations, or (``own``) by the library's calls.  ``exact()`` gives the results from the definitions in 64 bits.

A request's drafted tokens ("nodes") are its last cached tokens; node 0 is the root, the newest token that is certain;
parents[i] < i.  The cache: [layers, size, Hkv, D] in bf16, or bytes with scale exponents [layers, size / block, Hkv], a
byte e each: a row's value is e4m3(byte) * 2^(e - 127).
"""
import math
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn
STEP = 2.0 ** -48       # probabilities are summed in whole numbers of this: the same total in any order


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one user, a short chat, a small tree: latency
        dict(name="tree_1x1k", op="tree", B=1, n=1000, least=1000, nodes=8, chain=False, Hq=32, Hkv=8, D=128, page=16, block=0),
        # one user, a long document, a wide tree
        dict(name="tree_1x32k", op="tree", B=1, n=32768, least=32768, nodes=64, chain=False, Hq=32, Hkv=8, D=128, page=16, block=0),
        # a server's batch of mixed lengths, trees of up to 32 nodes
        dict(name="tree_32_ragged", op="tree", B=32, n=8192, least=500, nodes=32, chain=False, Hq=32, Hkv=8, D=128, page=16, block=0),
        # token-granular pages, small heads, drafted chains
        dict(name="tree_96_page1_d64", op="tree", B=96, n=4000, least=1, nodes=5, chain=True, Hq=16, Hkv=2, D=64, page=1, block=0),
        # one user over the 8-bit cache
        dict(name="tree_1x8k_e4m3", op="tree", B=1, n=8192, least=8192, nodes=16, chain=False, Hq=32, Hkv=8, D=128, page=16, block=16),
        # a batch over the 8-bit cache
        dict(name="tree_48_e4m3", op="tree", B=48, n=8192, least=500, nodes=24, chain=False, Hq=32, Hkv=8, D=128, page=16, block=16),
        # one user's drafted chain: latency
        dict(name="verify_1_chain", op="verify", B=1, nodes=6, V=32000, chain=True, sampled=True),
        # a batch's chains, drawn from the draft's probabilities, a large vocabulary
        dict(name="verify_64_chain", op="verify", B=64, nodes=6, V=131072, chain=True, sampled=True),
        # trees of the draft's likeliest tokens (no draft probabilities), rows that start anywhere
        dict(name="verify_32_tree", op="verify", B=32, nodes=48, V=100003, chain=False, sampled=False),
        # trees whose siblings were drawn from the draft: every refused one takes its share off the target
        dict(name="verify_16_drawn", op="verify", B=16, nodes=24, V=65536, chain=False, sampled=True),
        # slots kept in the page table after a batch's step
        dict(name="accept_64_table", op="accept", B=64, n=2000, least=100, nodes=32, layers=0, Hkv=8, D=128, page=1),
        # whole pages stay together: rows moved in all layers
        dict(name="accept_32_move", op="accept", B=32, n=300, least=40, nodes=32, layers=16, Hkv=8, D=128, page=16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "verify", "accept"])
    if op == "verify":
        B = _log(rng, 1, 48)
        nodes, V = _log(rng, 1, 40), _log(rng, 100, 130000)
        while B * nodes * V > 50_000_000:
            V = max(100, V // 2 - rng.randint(0, 9))
        return dict(op=op, B=B, nodes=nodes, V=V, chain=rng.random() < 0.4, sampled=rng.random() < 0.5)
    if op == "accept":
        layers = rng.choice([0, rng.randint(1, 15)])
        return dict(op=op, B=_log(rng, 1, 30), n=_log(rng, 40, 290 if layers else 1900), least=40, nodes=_log(rng, 1, 30),
                    layers=layers, Hkv=rng.choice([1, 2, 7, 8]), D=rng.choice([64, 128]), page=rng.choice([1, 16]))
    heads = rng.choice([(8, 2), (16, 2), (32, 8), (14, 2), (9, 3), (4, 4), (8, 1)])
    block = rng.choice([0, 0, 1, 4, 16, 64])
    B = _log(rng, 1, 30)
    n = _log(rng, 1, min(32000, 90000 // B))
    return dict(op=op, B=B, n=n, least=max(1, n // rng.choice([1, 4, 50])), nodes=_log(rng, 1, 60), chain=rng.random() < 0.3,
                Hq=heads[0], Hkv=heads[1], D=rng.choice([64, 128]), page=max(block, rng.choice([1, 16])), block=block)


def _lens(case):
    """Contexts between `least` and n, the first one n, spread over their logarithm, and each request's nodes: the same
    for every seed."""
    B, n = case["B"], case.get("n", 0)
    rng = random.Random(n * 1000003 + B * 101 + case["nodes"] * 7)
    context = [n] + [_log(rng, case["least"], n) for _ in range(B - 1)] if n else [0] * B
    nodes = [case["nodes"]] + [rng.randint((case["nodes"] + 1) // 2, case["nodes"]) for _ in range(B - 1)]
    return context, nodes


# ----------------------------------------------------------------- inputs

class State:
    pass


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _starts(counts):
    out = [0]
    for c in counts:
        out.append(out[-1] + c)
    return _ints(out)


def _parents(nodes, chain, rng):
    """Parents of one request's nodes (-1: the root): a chain, or a tree that branches most near its root."""
    if chain:
        return [i - 1 for i in range(nodes)]
    return [-1] + [int(rng.random() ** 1.5 * i) for i in range(1, nodes)]


def _tree_mask(parents, words):
    """Each node's own bit and its ancestors', in 32-bit words."""
    rows = []
    for p in parents:
        seen = []
        for i, a in enumerate(p):
            seen.append((1 << i) | (seen[a] if a >= 0 else 0))
        rows += seen
    signed = lambda x: x - (1 << 32) if x >> 31 else x  # noqa: E731
    return _ints([[signed(x >> (32 * w) & 0xFFFFFFFF) for w in range(words)] for x in rows])


def _table(lens, page, gen, rows_extra=3):
    """Slots of each request's tokens: whole pages in random order, rows of the table in random order, -1 behind
    the last token.  Returns (table, rows, size)."""
    B, dev = len(lens), "cuda"
    n = torch.tensor(lens, device=dev)
    pages = (n + page - 1) // page
    first = torch.cumsum(pages, 0) - pages
    n_pages = int(sum(-(-x // page) for x in lens)) + 8
    perm = torch.randperm(n_pages, generator=gen, device=dev)
    j = torch.arange(max(lens), device=dev)
    p = (first[:, None] + j // page).clamp(max=n_pages - 1)
    slots = torch.where(j < n[:, None], perm[p] * page + j % page, -1)
    rows = torch.randperm(B + rows_extra, generator=gen, device=dev)[:B]
    table = torch.full((B + rows_extra, max(lens)), -1, dtype=torch.int32, device=dev)
    table[rows] = slots.to(torch.int32)
    return table, rows.to(torch.int32), n_pages * page


def _rows(shape, gen):
    """K or V rows: normal values, each token and head with a magnitude of its own."""
    x = torch.randn(shape, generator=gen, device="cuda")
    return (x * torch.exp(0.6 * torch.randn(shape[:-1], generator=gen, device="cuda"))[..., None]).to(torch.bfloat16)


def _scale(e):
    """2^(e - 127) in fp32, from its bits (0 for e = 0)."""
    return (e.int() << 23).view(torch.float32)


def _block_cache(size, Hkv, D, block, gen):
    """A full one-layer e4m3 cache of `_rows`: bytes and scale exponents."""
    x = _rows((size, Hkv, D), gen).float()
    nb = -(-size // block)
    top = torch.zeros((nb * block, Hkv), device="cuda")
    top[:size] = x.abs().amax(-1)
    m, e = torch.frexp(top.view(nb, block, Hkv).amax(1))
    e = torch.where(m > 0, (e + 118 + (m > 0.875)).clamp(1, 254), 0)      # the smallest with amax <= 448 * 2^(e - 127)
    b = (x * _scale(254 - e.int()).repeat_interleave(block, 0)[:size, :, None]).clamp(-448, 448).to(E4M3)
    return b.view(torch.uint8)[None].contiguous(), e.to(torch.uint8)[None].contiguous()


def _prepare_tree(s, case, gen, rng):
    context, nodes = _lens(case)
    lens = [a + b for a, b in zip(context, nodes)]
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    s.block, s.scale = case["block"], 1.0 / math.sqrt(D)
    s.lens_host, s.nodes_host = lens, nodes
    s.table, s.rows, size = _table(lens, case["page"], gen)
    s.lens, s.qo = _ints(lens), _starts(nodes)
    s.mask = None if case["chain"] else _tree_mask([_parents(n, False, rng) for n in nodes], -(-max(nodes) // 32))
    s.q = torch.randn((sum(nodes), Hq, D), generator=gen, device="cuda").to(torch.bfloat16)
    if s.block:
        s.k, s.k_exp = _block_cache(size, Hkv, D, s.block, gen)
        s.v, s.v_exp = _block_cache(size, Hkv, D, s.block, gen)
    else:
        s.k, s.v = _rows((1, size, Hkv, D), gen), _rows((1, size, Hkv, D), gen)
        s.k_exp = s.v_exp = None
    s.workspace = torch.zeros(128 << 20, dtype=torch.uint8, device="cuda")
    s.out = torch.empty_like(s.q)


def _prepare_verify(s, case, gen, rng):
    _, nodes = _lens(dict(case, n=0))
    T, V = sum(nodes), case["V"]
    s.nodes_host, s.qo = nodes, _starts(nodes)
    parents = [_parents(n, case["chain"], rng) for n in nodes]
    s.parents = _ints([a for p in parents for a in p])
    # a few likely tokens in a flat tail; the draft sees them roughly
    logits = torch.randn((T, V), generator=gen, device="cuda")
    top = torch.randint(V, (T, 24), generator=gen, device="cuda")
    logits.scatter_add_(1, top, 6 + 6 * torch.rand(top.shape, generator=gen, device="cuda"))
    s.p = torch.softmax(logits, 1)
    logits.scatter_add_(1, top, torch.randn(top.shape, generator=gen, device="cuda"))
    q = torch.softmax(logits, 1)
    del logits
    # the tokens: drawn from the draft behind their parent, or its likeliest ones, in the order of the siblings
    at, rank, base = [], [], 0
    for p in parents:
        seen = {}
        for a in p:
            at.append(base + max(a, 0))
            rank.append(seen.get(a, 0))
            seen[a] = rank[-1] + 1
        base += len(p)
    at, rank = torch.tensor(at, device="cuda"), torch.tensor(rank, device="cuda")
    most = min(V, int(rank.max()) + 1)
    if case["sampled"]:
        u = torch.rand((T, 1), generator=gen, device="cuda", dtype=torch.float64)
        cum = torch.cumsum(q, 1, dtype=torch.float64)
        x = torch.searchsorted(cum[at], u * cum[at, -1:]).clamp(max=V - 1)[:, 0]
        s.q = q
    else:
        x = torch.topk(q, most, dim=1).indices[at, rank.clamp(max=most - 1)]
        s.q = None
    s.tokens = x.to(torch.int32)
    s.u_accept = torch.rand(T, generator=gen, device="cuda")
    s.u_sample = torch.rand(len(nodes), generator=gen, device="cuda")
    s.accepted = torch.empty((len(nodes), max(nodes)), dtype=torch.int32, device="cuda")
    s.count = torch.empty(len(nodes), dtype=torch.int32, device="cuda")
    s.next = torch.empty(len(nodes), dtype=torch.int32, device="cuda")


def _prepare_accept(s, case, gen, rng):
    context, nodes = _lens(case)
    lens = [a + b for a, b in zip(context, nodes)]
    s.table, s.rows, size = _table(lens, case["page"], gen)
    s.lens, s.qo, s.nodes_host = _ints(lens), _starts(nodes), nodes
    # paths as verification leaves them: the root, then deeper nodes
    most = max(nodes)
    paths = []
    for n in nodes:
        p = _parents(n, False, rng)
        path, i = [], rng.randrange(n)
        while i >= 0:
            path.append(i)
            i = p[i]
        paths.append(path[::-1])
    s.accepted = _ints([p + [-1] * (most - len(p)) for p in paths])
    s.count = _ints([len(p) for p in paths])
    s.paths_host = paths
    s.new_lens = torch.empty_like(s.lens)
    s.freed = torch.full((sum(nodes),), -1, dtype=torch.int32, device="cuda")
    s.k = s.v = None
    if case["layers"]:
        shape = (case["layers"], size, case["Hkv"], case["D"])
        s.k, s.v = _rows(shape, gen), _rows(shape, gen)


def prepare(case, seed):
    s = State()
    s.op = case["op"]
    {"tree": _prepare_tree, "verify": _prepare_verify, "accept": _prepare_accept}[s.op](s, case, _gen(seed), random.Random(seed))
    return s


# ------------------------------------------------------------------- runs

def run(s):
    if own:
        return _own(s)
    return {"tree": _tree, "verify": _verify, "accept": _accept}[s.op](s)


def _own(s):
    from paged_kv_cache_188_gb300 import api
    if s.op == "tree":
        api.pa_paged_tree_attn(s.q, s.k, s.v, 0, s.qo, s.table, s.rows, s.lens, s.scale, s.workspace, s.out,
                               tree_mask=s.mask, k_exp=s.k_exp, v_exp=s.v_exp, block=s.block)
        return s.out
    if s.op == "verify":
        api.pa_tree_verify(s.p, s.tokens, s.parents, s.qo, s.u_accept, s.u_sample, s.accepted, s.count, s.next,
                           draft_probs=s.q)
        return _verified(s)
    api.pa_kv_accept(s.table, s.rows, s.lens, s.qo, s.accepted, s.count, s.new_lens, s.freed, k_buf=s.k, v_buf=s.v)
    return _kept(s)


def _verified(s):
    return {"accepted": s.accepted, "count": s.count, "next": s.next}


def _kept(s):
    out = {"table": s.table, "lens": s.new_lens, "freed": s.freed}
    if s.k is not None:
        out["k"], out["v"] = s.k, s.v
    return out


def _values(buf, exp, slots, block):
    """Rows at `slots` (-1: zeros) in fp32."""
    at = slots.clamp(min=0).long()
    if exp is None:
        x = buf[0][at].float()
    else:
        x = buf[0].view(E4M3)[at].float() * _scale(exp[0][at // block])[..., None]
    return torch.where((slots >= 0)[..., None, None], x, 0.0)


def _tree(s):
    T, Hq, D = s.q.shape
    R, most = len(s.nodes_host), max(s.nodes_host)
    slots = s.table[s.rows.long()]
    k, v = _values(s.k, s.k_exp, slots, s.block), _values(s.v, s.v_exp, slots, s.block)
    Hkv, n = k.shape[2], slots.shape[1]
    count = (s.qo[1:] - s.qo[:-1]).long()
    context = s.lens.long() - count
    i = torch.arange(most, device=s.q.device)
    valid = i < count[:, None]                                          # [R, most]
    at = (s.qo[:-1].long()[:, None] + i).clamp(max=T - 1)
    q = s.q[at].float().view(R, most, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(R, Hkv, -1, D)
    j = torch.arange(n, device=s.q.device) - context[:, None]           # a token's node, negative in the context
    if s.mask is None:
        node = j[:, None] <= i[:, None]
    else:
        word = s.mask[at].gather(2, (j.clamp(min=0) >> 5).clamp(max=s.mask.shape[1] - 1)[:, None].expand(R, most, n))
        node = (word >> (j.clamp(min=0) & 31)[:, None]) & 1 != 0
    seen = torch.where(j[:, None] < 0, True, node & (j < count[:, None])[:, None])[:, None, None]
    x = (torch.matmul(q, k.permute(0, 2, 3, 1)) * s.scale).view(R, Hkv, -1, most, n)
    x = torch.where(seen, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(x - torch.where(top == -math.inf, 0.0, top)), 0.0)
    del x
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, 1.0, total)                         # a row that sees nothing: zeros
    out = torch.matmul(p.view(R, Hkv, -1, n), v.permute(0, 2, 1, 3)).view(R, Hkv, Hq // Hkv, most, D)
    return out.permute(0, 3, 1, 2, 4).reshape(R, most, Hq, D)[valid].to(torch.bfloat16)


def _steps(r):
    """Probabilities as whole numbers of STEP."""
    return torch.round(r.double() / STEP).long()


def _verify(s):
    R, V = len(s.nodes_host), s.p.shape[1]
    first, count = s.qo[:-1].long(), (s.qo[1:] - s.qo[:-1]).long()
    b = torch.arange(R, device=s.p.device)
    cur, kept = torch.zeros_like(first), torch.ones_like(first)
    s.accepted.fill_(-1)
    s.accepted[:, 0] = 0
    r, z = s.p[first].clamp(min=0), torch.ones(R, device=s.p.device)
    for i in range(1, max(s.nodes_host)):
        at = (first + i).clamp(max=s.p.shape[0] - 1)
        x = s.tokens[at].long()
        child = (i < count) & (s.parents[at] == cur)
        have = r[b, x]
        share = z if s.q is None else z * s.q[first + cur, x]
        take = child & (s.u_accept[at] * share < have)
        leave = child & ~take
        if s.q is None:
            z = torch.where(leave, (z - have).clamp(min=0), z)
            r[b, x] = torch.where(leave, 0.0, have)
        else:
            less = (r - z[:, None] * s.q[first + cur]).clamp(min=0)
            r = torch.where(leave[:, None], less, r)
            z = torch.where(leave, (_steps(less).sum(1).double() * STEP).float(), z)
        cur = torch.where(take, i, cur)
        r = torch.where(take[:, None], s.p[at].clamp(min=0), r)
        z = torch.where(take, 1.0, z)
        s.accepted[b, kept.clamp(max=s.accepted.shape[1] - 1)] = torch.where(
            take, i, s.accepted[b, kept.clamp(max=s.accepted.shape[1] - 1)].long()).int()
        kept += take
    w = _steps(r)
    w = torch.where(w.sum(1, keepdim=True) > 0, w, _steps(s.p[first + cur].clamp(min=0)))
    cum = torch.cumsum(w, 1)
    # floor(u * total) in whole numbers: u = m 2^-(24 + k), m below 2^24, the total in halves of 24 bits
    m, k = torch.frexp(s.u_sample)
    m, k = (m * 2.0 ** 24).long(), (-k).clamp(0, 63)
    total = cum[:, -1]
    goal = (m * (total >> 24) + ((m * (total & 0xFFFFFF)) >> 24)) >> k
    s.next.copy_((cum <= goal[:, None]).sum(1))
    s.count.copy_(kept)
    return _verified(s)


def _accept(s):
    rows, count = s.rows.long(), (s.qo[1:] - s.qo[:-1]).long()
    context = s.lens.long() - count
    most, width = s.accepted.shape[1], s.table.shape[1]
    i = torch.arange(most, device=rows.device)
    slots = s.table[rows].gather(1, (context[:, None] + i).clamp(max=width - 1))      # [R, most] of the nodes
    have, stay = i < count[:, None], i < s.count[:, None]
    path = s.accepted.clamp(min=0).long()
    kept = torch.zeros_like(slots, dtype=torch.bool)
    b = torch.arange(len(rows), device=rows.device)[:, None].expand_as(path)
    kept[b[stay], path[stay]] = True
    s.new_lens.copy_(context + s.count)
    if s.k is None:
        gone = have & ~kept
        to = (context[:, None] + i)[stay]
        s.table[rows[:, None].expand_as(path)[stay], to] = slots.gather(1, path)[stay]
        s.freed[(s.qo[:-1, None] + torch.cumsum(gone, 1) - 1)[gone].long()] = slots[gone]
        return _kept(s)
    gone = have & ~stay
    s.freed[(s.qo[:-1, None] + i - s.count[:, None])[gone].long()] = slots[gone]
    src, dst = slots.gather(1, path)[stay].long(), slots[stay].long()
    for buf in (s.k, s.v):
        buf[:, dst] = buf[:, src]
    return _kept(s)


# ------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    context, nodes = _lens(dict(case, n=case.get("n", 0)))
    T = sum(nodes)
    if op == "verify":
        # the last kept node's row, and the draft's where its child was refused (nearly always); per node a gather of each
        per = 4 * case["V"] * (2 if case["sampled"] else 1)
        return {"bytes": len(nodes) * per + T * (16 + (8 if case["sampled"] else 4)),
                "flops": len(nodes) * case["V"] * (3 if case["sampled"] else 1)}
    if op == "accept":
        if not case["layers"]:
            return {"bytes": 4 * T + 4 * T + 16 * len(nodes), "flops": T}
        # a path holds about the logarithm of its tree's nodes; all but its root move
        moved = sum(max(0.0, math.log2(n)) for n in nodes)
        return {"bytes": int(8 * moved * case["layers"] * case["Hkv"] * case["D"]) + 8 * T, "flops": T}
    D, block = case["D"], case["block"]
    per = 2 * D + 2.0 / block if block else 4 * D
    total = sum(context) + T
    pairs = sum(n * (c + n) for c, n in zip(context, nodes))
    return {"bytes": total * (case["Hkv"] * per + 4) + 4 * T * case["Hq"] * D + 4 * T, "flops": 4 * pairs * case["Hq"] * D}


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


def _rows64(buf, exp, slots, block):
    at = slots.long()
    if exp is None:
        return buf[0][at].double()
    return _value64(buf[0][at]) * _two(exp[0][at // block].int() - 127)[..., None]


def _exact_tree(s):
    out = torch.zeros(s.q.shape, dtype=torch.float64, device="cuda")
    masks = None if s.mask is None else s.mask.cpu().tolist()
    lo = 0
    for row, n, m in zip(s.rows.tolist(), s.lens_host, s.nodes_host):
        k, v = _rows64(s.k, s.k_exp, s.table[row, :n], s.block), _rows64(s.v, s.v_exp, s.table[row, :n], s.block)
        hidden = torch.zeros((m, n), dtype=torch.bool)
        for i in range(m):
            for j in range(m):
                hidden[i, n - m + j] = j > i if masks is None else not masks[lo + i][j // 32] >> (j % 32) & 1
        hidden = hidden.cuda()
        q = s.q[lo:lo + m].double()
        G = q.shape[1] // k.shape[1]
        for h in range(q.shape[1]):
            x = (q[:, h] @ k[:, h // G].T) * s.scale
            out[lo:lo + m, h] = torch.softmax(x.masked_fill(hidden, -math.inf), -1) @ v[:, h // G]
        lo += m
    return out


def _exact_verify(s):
    lo, parents, tokens = 0, s.parents.tolist(), s.tokens.tolist()
    u, us = s.u_accept.double().tolist(), s.u_sample.double().tolist()
    accepted = torch.full(s.accepted.shape, -1, dtype=torch.int64)
    count, after = [], []
    for b, n in enumerate(s.nodes_host):
        path, r, taken = [0], s.p[lo].double(), 1.0
        for i in range(1, n):
            if parents[lo + i] != path[-1]:
                continue
            x = tokens[lo + i]
            if s.q is None:
                draft = torch.zeros_like(r)
                draft[x] = 1.0
            else:
                draft = s.q[lo + path[-1]].double()
            if u[lo + i] * taken * float(draft[x]) < float(r[x]):
                path.append(i)
                r, taken = s.p[lo + i].double(), 1.0
            else:
                less = (r - taken * draft).clamp(min=0)
                if s.q is None:
                    taken = taken - float(r[x])
                    r = less
                    r[x] = 0
                else:
                    r, taken = less, float(less.sum())
        if float(r.sum()) == 0:
            r = s.p[lo + path[-1]].double()
        cum = torch.cumsum(r, 0)
        after.append(int((cum <= us[b] * float(cum[-1])).sum()))
        accepted[b, :len(path)] = torch.tensor(path)
        count.append(len(path))
        lo += n
    return {"accepted": accepted.cuda(), "count": torch.tensor(count, device="cuda"), "next": torch.tensor(after, device="cuda")}


def exact(case, seed):
    if case["op"] == "accept":
        return None                                                # table entries and moved rows: nothing is computed
    s = prepare(case, seed)
    return _exact_tree(s) if case["op"] == "tree" else _exact_verify(s)
