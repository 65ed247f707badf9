"""Plain 64-bit reference of the block-scaled e4m3 cache, of attention with
weights over it (or over a bf16 cache), and of eviction.  Host only, from the
definitions; shares nothing with the library."""
import math

import numpy as np
import torch

POWERS = np.array([0.0] + [math.ldexp(1.0, e - 127) for e in range(1, 255)] + [math.nan])   # scale of an exponent byte


def e4m3_table():
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        v[c] = math.nan if c & 127 == 127 else x
    v[128:] = -v[:128]
    return v


E4M3 = e4m3_table()


def encode(x):
    """Doubles to e4m3 bytes: nearest, ties to the even code, saturating, NaN to 0x7F."""
    x = np.asarray(x, np.float64)
    mags = E4M3[:127]
    a = np.minimum(np.abs(x), 448.0)
    a0 = np.nan_to_num(a)
    hi = np.clip(np.searchsorted(mags, a0), 1, 126)
    lo = hi - 1
    dl, dh = a0 - mags[lo], mags[hi] - a0
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(np.isnan(x), 127, code)
    return (code + np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def need(amax):
    """Smallest e in [1, 254] with amax <= 448 * 2^(e - 127); 0 for 0."""
    if amax == 0:
        return 0
    e = 1
    while amax > 448.0 * POWERS[e]:
        e += 1
    return e


def store(buf, exp, x, loc, block):
    """One call of the store on one layer: buf uint8 [size, Hkv, D], exp uint8 [n_blocks, Hkv], x doubles."""
    size, Hkv, _ = buf.shape
    groups = {}
    for t, s in enumerate(loc):
        if 0 <= s < size:
            groups.setdefault(int(s) // block, []).append(t)
    for blk, ts in groups.items():
        for h in range(Hkv):
            rows = x[ts, h]
            fin = np.abs(rows[np.isfinite(rows)])
            old = int(exp[blk, h])
            e = max(old, need(float(fin.max()) if fin.size else 0.0))
            mine = {int(loc[t]) for t in ts}
            if e > old > 0:
                for s in range(blk * block, min(size, (blk + 1) * block)):
                    if s not in mine:
                        buf[s, h] = encode(E4M3[buf[s, h]] * math.ldexp(1.0, old - e))
            for t in ts:
                buf[int(loc[t]), h] = encode(np.ldexp(x[t, h], 127 - e))
            exp[blk, h] = e


def values(buf, exp, slots, block):
    """Rows at `slots` in doubles: buf uint8 [size, Hkv, D] with exponents, or bf16 rows (exp None)."""
    if exp is None:
        return buf[slots].double()
    return torch.from_numpy(E4M3)[buf[slots].long()] * torch.from_numpy(POWERS)[exp[slots // block].long()][..., None]


def attention(q, k, v, scale, first=None, terms=2.0 ** -22):
    """q [m, Hq, D] over k, v [n, Hkv, D]; row i sees positions 0 .. first + i (first None: all).  Returns the
    output [m, Hq, D], the weights [m, Hq, n], and per output row and head what its error is measured in:
    sum_j p_j |v_j| [m, Hq, D], max_j p_j, max |v|, and the error of a score (natural units) that
    fp32 products allow."""
    m, Hq, _ = q.shape
    n, Hkv, _ = k.shape
    G = Hq // Hkv
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    x = torch.einsum("mhd,nhd->mhn", q, kk) * scale
    mag = torch.einsum("mhd,nhd->mhn", q.abs(), kk.abs()) * abs(scale)
    top = q.abs().amax(-1)[..., None] * kk.abs().sum(-1).T[None] * abs(scale)
    if first is not None:
        hide = torch.arange(n)[None] > first + torch.arange(m)[:, None]
        x = x.masked_fill(hide[:, None], -math.inf)
        mag, top = mag.masked_fill(hide[:, None], 0), top.masked_fill(hide[:, None], 0)
    p = torch.softmax(x, -1)
    # products summed in fp32 with truncation (2^-20 of their magnitudes), what q's two terms leave out (`terms` of
    # the row's largest element: 2^-22 where the second term is kept 16 times larger, 2^-19 where it is not), the
    # exponent's argument in fp32
    ds = (2.0 ** -20 * mag + terms * top + 2.0 ** -22 * x.abs().nan_to_num(posinf=0.0)).amax(-1)
    return dict(out=torch.einsum("mhn,nhd->mhd", p, vv), p=p, mean=torch.einsum("mhn,nhd->mhd", p, vv.abs()),
                pmax=p.amax(-1), vmax=float(v.abs().max()) if n else 0.0, ds=ds, n=n)


def check_out(got, r, p_bits, what):
    """|got - ref| within one bf16 rounding of the result, the weights' rounding (2^-p_bits each, relative) and
    the scores' error, both on sum p |v|; weights below 2^-14 of the tile's largest lose absolute 2^-26 of it."""
    rel = 2.0 ** -p_bits + 2 * r["ds"][..., None] + 2.0 ** -18
    tol = 2.0 ** -8 * r["out"].abs() + rel * r["mean"] * 1.01 + r["n"] * 2.0 ** -26 * (r["pmax"] * r["vmax"])[..., None] + 1e-37
    bad = (got.double() - r["out"]).abs() - tol
    assert torch.isfinite(got.double()).all(), f"{what}: non-finite output"
    assert float(bad.max()) <= 0, f"{what}: off by {float(bad.max()):.3e} more than {float(tol.flatten()[bad.argmax()]):.3e}"


def evict(slots, w, budget, recent):
    """One request: (kept slots, kept weights, freed slots)."""
    n = len(slots)
    if n <= budget:
        return list(slots), list(w), []
    cand = n - recent
    key = [(-math.inf if math.isnan(x) else float(x)) for x in w[:cand]]
    best = sorted(range(cand), key=lambda j: (-key[j], j))[:budget - recent]
    keep = sorted(best + list(range(cand, n)))
    gone = sorted(set(range(n)) - set(keep))
    return [slots[j] for j in keep], [w[j] for j in keep], [slots[j] for j in gone]
