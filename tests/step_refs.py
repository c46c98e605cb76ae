"""Plain implementations of the operators of a step with drafted rows, from their rules: 64 bits
for what is computed, exact arithmetic for what is decided."""
from fractions import Fraction

import numpy as np
import torch

from operator_refs import BF16, F64, dev


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).to(dev())


def starts(rows):
    return np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)


def random_tree(m, rng, width=4):
    """Parents of a tree of m rows; row 0's is not read."""
    return ([-1] + [int(rng.integers(max(0, i - width), i)) for i in range(1, m)])[:m]


def ancestors(parents):
    """Bit j of entry i: row j is row i or above it (a row without a parent before it is a root)."""
    mask = []
    for i, p in enumerate(parents):
        mask.append(1 << i | (mask[p] if i > 0 and 0 <= p < i else 0))
    return mask


def as_int64(masks):
    return torch.from_numpy(np.asarray(masks, np.uint64).view(np.int64)).to(dev())


def block_table(lengths, T, rng, spare=3, extra=1):
    """A table of permuted blocks for `lengths` positions, and the pool's size."""
    need = [-(-int(n) // T) for n in lengths]
    B = sum(need) + 1 + spare
    order = rng.permutation(np.arange(1, B))
    table = np.zeros((len(need), max(max(need, default=1), 1) + extra), np.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    return table, B


def attend(q, k, v, seen, scale):
    """(o, bound) of rows q [m, Hq, D] over k, v [n, H, D]; seen [m, n] says what each row sees.

    The bound: a logit sums D products, is scaled and has the maximum taken off, D + 4
    roundings of 32 bits (2^-23 each: the matrix unit may cut off) of the products' magnitudes;
    exp2 is within 2^-21; both move a weight and the sum of the weights by that relative
    amount.  Weights are rounded to bf16 (2^-8) for their product with V, sums run over n keys in 32
    bits, the output is rounded to bf16; a weight below 2^-126 of the largest may be lost."""
    m, hq, d = q.shape
    n, h = k.shape[0], k.shape[1]
    if m == 0 or n == 0:
        z = torch.zeros((m, hq, d), dtype=F64, device=q.device)
        return z, z.clone()
    q, k, v = q.to(F64).view(m, h, hq // h, d), k.to(F64), v.to(F64)
    seen = torch.as_tensor(seen, device=q.device)
    gone = ~seen.any(0)
    k, v = k.clone(), v.clone()
    k[gone] = 0
    v[gone] = 0
    x = torch.einsum("mhgd,nhd->hgmn", q, k) * scale
    size = torch.einsum("mhgd,nhd->hgmn", q.abs(), k.abs()) * scale
    x = x.masked_fill(~seen, -float("inf"))
    top = x.amax(-1, keepdim=True)
    w = torch.where(seen, torch.exp(x - torch.where(top.isfinite(), top, 0.0)), 0.0)
    total = w.sum(-1, keepdim=True)
    w = torch.where(total > 0, w / total, 0.0)
    o = torch.einsum("hgmn,nhd->mhgd", w, v)
    a = torch.einsum("hgmn,nhd->mhgd", w, v.abs())
    seen_size = torch.where(seen, size, 0.0).amax(-1)
    slack = 2 * ((d + 4) * 2.0 ** -23 * seen_size + 2.0 ** -20) + n * 2.0 ** -23
    slack = slack.permute(2, 0, 1)[..., None]
    bound = o.abs() * 2.0 ** -8 + a * (2.0 ** -8 + slack) + n * 2.0 ** -126 * v.abs().max()
    return o.reshape(m, hq, d), bound.reshape(m, hq, d)


def verify(target, draft, tokens, parents, uniform):
    """(tokens, path) of one request in exact arithmetic: target and draft [m][V] fractions (draft
    may be None), numbers as fractions."""
    m, V = len(target), len(target[0])
    at, path, out = 0, [0], []
    while True:
        s, z, nxt = list(target[at]), Fraction(1), None
        for c in range(1, m):
            if parents[c] != at or not 0 <= parents[c] < c or not 0 <= tokens[c] < V:
                continue
            x = tokens[c]
            q = draft[at] if draft is not None else [Fraction(int(i == x)) for i in range(V)]
            if uniform[c] * q[x] * z < s[x]:
                nxt = c
                break
            if draft is None:
                z, s[x] = max(z - s[x], Fraction(0)), Fraction(0)
            else:
                s = [max(a - z * b, Fraction(0)) for a, b in zip(s, q)]
                z = sum(s)
        if nxt is None:
            break
        at = nxt
        path.append(at)
        out.append(tokens[at])
    if sum(s) == 0:
        s = list(target[at])
    want, run = uniform[0] * sum(s), Fraction(0)
    last = -1
    for i, x in enumerate(s):
        run += x
        if run > want:
            last = i
            break
    return out + [last], path
