"""kv_verify_drafts where one token has most of the weight, at the borders between tokens: what is left
of it after refusals takes more than 24 bits, and numbers on either side of a border fall on either side."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import paged_kv_cache_39_gb300 as kv
from operator_refs import BF16, dev
from step_refs import i32, verify

pytestmark = pytest.mark.gpu
UNIT = Fraction(1, 2 ** 45)


def fractions(t):
    return [[Fraction(x) for x in row] for row in t.double().tolist()]


def peaked(refusals, V, dtype, rng):
    """(p, q, tokens) of a row: one token of 0.25 to 1, draft probabilities of many sizes, and tokens that a
    number of nearly 1 refuses; the last one keeps a weight."""
    p = rng.uniform(0, 1, V)
    top = int(rng.integers(0, V - 1))
    whole = rng.uniform(0.25, 1.0)
    p[top] = 0
    p *= (1 - whole) / p.sum()
    p[top] = whole
    q = rng.uniform(1, 2, V) * 2.0 ** -rng.integers(6, 26, V)
    tokens = rng.choice([i for i in range(V - 1) if i != top], refusals, replace=False)
    q[V - 1] = 2.0 ** -30
    p[V - 1] += 0.01
    q[tokens] = 0.8 / refusals
    p[tokens] *= 0.01
    return torch.from_numpy(np.stack([p, q])).to(dtype), tokens.tolist()


def left_over(p, q, refusals):
    s, z = p, Fraction(1)
    for _ in range(refusals):
        s = [max(a - z * b, Fraction(0)) for a, b in zip(s, q)]
        z = sum(s)
    return s


def around(border):
    """The two neighbouring fp32 numbers with the border between them."""
    u = np.float32(float(border))
    if Fraction(float(u)) > border:
        return np.nextafter(u, np.float32(0)), u
    return u, np.nextafter(u, np.float32(1))


def cases(count, refusals, V, dtype, seed):
    """Requests with a row 0 and `refusals` children of it, and their outcome by the rule.  Left out are
    borders an fp32 number is too near to.  A weight is off by less than a unit and a sum by V of
    them; a refusal takes that of the sum before it, times q (which sums to less than 2), along."""
    rng = np.random.default_rng(seed)
    m = refusals + 1
    target, draft, tokens, uniform, want = [], [], [], [], []
    near = 0
    while len(want) < count:
        pq, x = peaked(refusals, V, dtype, rng)
        p, q = fractions(pq)
        s = left_over(p, q, refusals)
        sums = np.cumsum(np.asarray(s, object))
        # behind the largest one but the last: a border that its own error moves
        for u in around(sums[int(np.argmax(s[:-1]))] / sums[-1]):
            if min(abs(Fraction(float(u)) * sums[-1] - c) for c in sums) < 3 ** refusals * V * UNIT:
                near += 1
                continue
            numbers = [float(u)] + [1 - 2.0 ** -24] * refusals
            rows = [p] + [[Fraction(1, V)] * V] * refusals
            out, path = verify(rows, [q] + rows[1:], [0] + x, [-1] + [0] * refusals, [Fraction(n) for n in numbers])
            assert path == [0]
            want.append(out[0])
            target += [pq[0]] + [torch.full((V,), 1 / V, dtype=dtype)] * refusals
            draft += [pq[1]] + [torch.full((V,), 1 / V, dtype=dtype)] * refusals
            tokens += [0] + x
            uniform += numbers
    assert near <= count // 50
    parents = ([-1] + [0] * refusals) * len(want)
    return (torch.stack(target).to(dev()), i32(tokens), i32(np.arange(len(want) + 1) * m),
            torch.tensor(uniform, dtype=torch.float32, device=dev()), torch.stack(draft).to(dev()), i32(parents)), want


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("V", [5, 24, 301])
@pytest.mark.parametrize("refusals", [1, 2, 3])
@pytest.mark.parametrize("count", [20, 400])       # clusters of CTAs, a CTA each
def test_numbers_beside_a_border(refusals, V, dtype, count):
    args, want = cases(count, refusals, V, dtype, 1000 * refusals + V + count)
    err = kv.new_error_word(dev())
    got, path, kept = kv.kv_verify_drafts(*args, err=err)
    assert not kept.any() and err.item() == 0
    wrong = [i for i, (a, b) in enumerate(zip(got[::refusals + 1].tolist(), want)) if a != b]
    assert not wrong, f"{len(wrong)} of {count} beside the border, first {wrong[:5]}"


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("rows", [1, 200])
def test_rows_that_are_no_probabilities_end(dtype, rows):
    """2^20 tokens of 1 each: their sum passes 64 bits, the last token is any or none."""
    V = 2 ** 20
    p = torch.ones((rows, V), dtype=dtype, device=dev())
    u = torch.linspace(0, 0.99, rows, device=dev())
    got, _, kept = kv.kv_verify_drafts(p, i32([0] * rows), i32(np.arange(rows + 1)), u)
    assert not kept.any() and ((got >= -1) & (got < V)).all()
