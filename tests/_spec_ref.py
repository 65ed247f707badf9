"""Plain references of drafted tokens' attention, verification and acceptance, on
the host from the definitions: attention in doubles, verification in fp32 steps as documented
and in exact rationals.  Shares nothing with the library."""
from fractions import Fraction

import numpy as np
import torch


def tree_seen(parents):
    """[n, n]: node i sees itself and its ancestors."""
    n = len(parents)
    seen = torch.zeros((n, n), dtype=torch.bool)
    for i, a in enumerate(parents):
        if a >= 0:
            seen[i] = seen[a]
        seen[i, i] = True
    return seen


def chain_seen(n):
    return torch.ones((n, n), dtype=torch.bool).tril()


def mask_words(seen, words):
    """The bits of `seen` [n, n] as int32 [n, words]."""
    out = np.zeros((len(seen), words), np.uint32)
    for i in range(len(seen)):
        for k in range(len(seen)):
            if seen[i, k]:
                out[i, k // 32] |= np.uint32(1 << (k % 32))
    return torch.from_numpy(out.view(np.int32).copy())


def attention(q, k, v, scale, seen, terms=0.0):
    """q [m, Hq, D] of the last m of n cached tokens, k, v [n, Hkv, D] in doubles, seen [m, m]: the output and what its
    error is measured in (as the other references': sum p |v|, the largest score error `ds` that fp32 products allow and
    q's terms, which leave out up to `terms` of its row's largest element).
    A row that is not seen enters nothing, whatever it holds."""
    m, Hq, D = q.shape
    n, Hkv, _ = k.shape
    G = Hq // Hkv
    full = torch.ones((m, n), dtype=torch.bool)
    full[:, n - m:] = seen
    out = torch.zeros((m, Hq, D), dtype=torch.float64)
    mean, ds, pmax = torch.zeros_like(out), torch.zeros((m, Hq), dtype=torch.float64), torch.zeros((m, Hq), dtype=torch.float64)
    vmax = 0.0
    for i in range(m):
        at = full[i].nonzero()[:, 0]
        if len(at) == 0:
            continue
        kk, vv = k[at].repeat_interleave(G, 1), v[at].repeat_interleave(G, 1)
        x = torch.einsum("hd,nhd->hn", q[i], kk) * scale
        mag = torch.einsum("hd,nhd->hn", q[i].abs(), kk.abs()) * abs(scale)
        p = torch.softmax(x, -1)
        out[i] = torch.einsum("hn,nhd->hd", p, vv)
        mean[i] = torch.einsum("hn,nhd->hd", p, vv.abs())
        pmax[i] = p.amax(-1)
        top = q[i].abs().amax(-1)[:, None] * kk.abs().sum(-1).T * abs(scale)
        ds[i] = (2.0 ** -20 * mag + 2.0 ** -22 * x.abs() + terms * top).amax(-1)
        vmax = max(vmax, float(vv.abs().max()))
    return dict(out=out, mean=mean, ds=ds, pmax=pmax, vmax=vmax, n=n, p=None)


def _fixed(w):
    """Probabilities (fp32) in whole steps of 2^-48, nearest even (exact: their products with 2^48 are doubles)."""
    return np.rint(w.astype(np.float64) * 2.0 ** 48).astype(np.int64)


def _clean(row):
    return np.where(row > 0, row, np.float32(0))


def _draw(c, u):
    """The first index at which the running sum of the whole numbers c passes u times their sum; -1 for none."""
    total = int(c.sum())
    if total == 0:
        return -1
    goal = Fraction(float(u)) * total
    return int(np.searchsorted(np.cumsum(c), goal.numerator // goal.denominator, side="right"))


def verify(p, f, tokens, parents, u, u_last, max_path):
    """One request: (path, next token), in fp32 with each operation rounded and sums in steps of 2^-48.  p, f: fp32
    arrays [n, V] (f None: chosen tokens)."""
    F, V = np.float32, p.shape[1]
    path, w, Z = [0], _clean(p[0]), F(1)
    for i in range(1, len(tokens)):
        if len(path) == max_path:
            break
        a, x = parents[i], tokens[i]
        if a != path[-1] or not 0 <= x < V:
            continue
        fr = None if f is None else _clean(f[a])
        share = F(u[i]) * (Z * fr[x] if fr is not None else Z)
        if share < w[x]:
            path.append(i)
            w, Z = _clean(p[i]), F(1)
        elif fr is not None:
            w = np.maximum(w - Z * fr, F(0))
            Z = F(float(_fixed(w).sum()) * 2.0 ** -48)
        else:
            Z = max(Z - w[x], F(0))
            w = w.copy()
            w[x] = 0
    after = _draw(_fixed(w), u_last)
    return path, after if after >= 0 else _draw(_fixed(_clean(p[path[-1]])), u_last)


def verify_exact(p, f, tokens, parents, u, u_last):
    """The same in rationals, without any rounding."""
    n, V = p.shape
    num = lambda row: [Fraction(float(x)) for x in row]  # noqa: E731
    path, w, Z = [0], num(p[0]), Fraction(1)
    for i in range(1, n):
        if parents[i] != path[-1]:
            continue
        x = tokens[i]
        draft = num(f[path[-1]]) if f is not None else [Fraction(int(v == x)) for v in range(V)]
        if Fraction(float(u[i])) * Z * draft[x] < w[x]:
            path.append(i)
            w, Z = num(p[i]), Fraction(1)
        elif f is not None:
            w = [max(w[v] - Z * draft[v], Fraction(0)) for v in range(V)]
            Z = sum(w)
        else:
            Z -= w[x]
            w[x] = Fraction(0)
    if sum(w) == 0:
        w = num(p[path[-1]])
    goal, run = Fraction(float(u_last)) * sum(w), Fraction(0)
    for v in range(V):
        run += w[v]
        if run > goal:
            return path, v
    return path, -1


def accept(row, context, n, path):
    """Table form of one request: (new row, new length, freed)."""
    nodes = list(row[context:context + n])
    new = list(row)
    for k, e in enumerate(path):
        new[context + k] = nodes[e]
    return new, context + len(path), [nodes[i] for i in range(n) if i not in set(path)]


def accept_move(row, context, n, path):
    """Move form: (list of (from slot, to slot), new length, freed)."""
    return ([(row[context + e], row[context + k]) for k, e in enumerate(path)], context + len(path),
            list(row[context + len(path):context + n]))


def random_parents(n, g, chain=False, wide=1.5):
    if chain:
        return [i - 1 for i in range(n)]
    return ([-1] + [int(float(torch.rand((), generator=g)) ** wide * i) for i in range(1, n)])[:n]


def softmax_rows(T, V, g, sharp=3.0):
    return torch.softmax(sharp * torch.randn((T, V), generator=g, dtype=torch.float64), -1).float().numpy()


