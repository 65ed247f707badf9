"""The plain form of the verification, in torch operations on the host: the token that
it draws is the definition's, whatever places the random number has."""
import importlib.util
import os
from fractions import Fraction

import numpy as np
import pytest
import torch

import _spec_ref as S

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "more_operators.py")


@pytest.fixture(scope="module")
def plain():
    spec = importlib.util.spec_from_file_location("more_operators", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def drawn(plain, p, u):
    """The token that follows the root, for each row of p and number of u."""
    s, R = plain.State(), len(u)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    s.nodes_host, s.qo = [1] * R, torch.arange(R + 1, dtype=torch.int32)
    s.p, s.q, s.tokens, s.parents, s.u_accept, s.u_sample = p, None, i32(R), i32(R) - 1, torch.zeros(R), u
    s.accepted, s.count, s.next = i32(R)[:, None].clone(), i32(R), i32(R)
    return plain._verify(s)["next"].tolist()


def want(p, u):
    return [S.verify(row[None], None, [0], [-1], [0], x, 1)[1] for row, x in zip(p.numpy(), u.numpy())]


@pytest.mark.parametrize("seed", range(4))
def test_token_at_the_border(plain, seed):
    """Numbers next to a running sum, which below 1/2 have places finer than 2^-24."""
    g = torch.Generator().manual_seed(seed)
    V, R = 3001, 200
    row = torch.from_numpy(S.softmax_rows(1, V, g, 1.0))[0]
    steps = S._fixed(row.numpy())
    cum, total = np.cumsum(steps), int(steps.sum())
    u = []
    for v in torch.randint(V // 2, (R,), generator=g).tolist():
        x = np.float32(float(Fraction(int(cum[v]), total)))
        while Fraction(float(x)) * total < int(cum[v]):        # the smallest number that the token v does not reach
            x = np.nextafter(x, np.float32(1))
        u.append(x)
    u = torch.tensor(np.array(u))
    assert ((u * 2 ** 24) != (u * 2 ** 24).floor()).sum() > R // 2
    p = row.repeat(R, 1)
    assert drawn(plain, p, u) == want(p, u)


def test_token_of_numbers_of_32_bits(plain):
    """32 random bits rounded to fp32, as a device's generator gives them; the ends of [0, 1)."""
    g = torch.Generator().manual_seed(9)
    V, R = 20000, 400
    bits = torch.randint(1 << 32, (R,), generator=g, dtype=torch.int64)
    u = (bits.double() * 2.0 ** -32).float().clamp(max=1 - 2.0 ** -24)
    u[:4] = torch.tensor([0.0, 2.0 ** -32, 2.0 ** -149, 1 - 2.0 ** -24])
    p = torch.from_numpy(S.softmax_rows(1, V, g, 0.5)).repeat(R, 1)
    assert drawn(plain, p, u) == want(p, u)
