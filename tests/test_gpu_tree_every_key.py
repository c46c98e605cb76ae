"""Every key of a context counts once in kv_attention_tree: at the boundaries of units, blocks, CTAs'
shares and parts of a join, with contexts of up to 131072 tokens."""
import numpy as np
import pytest
import torch

import paged_kv_cache_39_gb300 as kv
from key_patterns import marks, shares, turns, wrong
from operator_refs import BF16, dev, normal
from step_refs import block_table, i32, starts

pytestmark = pytest.mark.gpu
UNIT = 32       # keys that share a channel: one of them is 2^-5 of its channel's share, a rounding 2^-8

HEADS = [(32, 8, 128), (8, 1, 128), (6, 2, 64), (40, 5, 64)]
BATCHES = [
    ([1], [1009], None), ([8], [1001], None), ([5], [40007], None), ([64], [30011], None),
    ([3, 1, 1, 16, 2, 64], [20000, 1, 0, 3, 5001, 64], None),
    ([1] * 40, [9001 + 37 * i for i in range(40)], None),
    ([16, 1], [131072, 100003], None),
    ([9, 33, 2, 1], [30000, 20011, 700, 64], [37, 19999, 320, 0]),
]


def cache(ctx, rows, T, h, D, seed):
    rng = np.random.default_rng(seed)
    table, B = block_table([c + m for c, m in zip(ctx, rows)], T, rng)
    slots = [torch.from_numpy(table[r, np.arange(c + m) // T].astype(np.int64) * T + np.arange(c + m) % T).to(dev())
             for r, (c, m) in enumerate(zip(ctx, rows))]
    return i32(table), torch.cat(slots), B


def fill(to, at, ctx, rows, unit, D, turn):
    """The marks of every request's positions, in all heads."""
    n = max(c + m for c, m in zip(ctx, rows))
    mark = torch.from_numpy(marks(n, unit, D, turn)).to(dev()).to(BF16)
    x = torch.cat([mark[:c + m] for c, m in zip(ctx, rows)])
    to[0].flatten(0, 1)[at] = x[:, None].expand(-1, to.shape[3], -1)


@pytest.mark.parametrize("rows,ctx,start", BATCHES)
@pytest.mark.parametrize("hq,h,D", HEADS)
@pytest.mark.parametrize("T", [16, 20])       # TMA boxes, rows one by one
def test_shares(rows, ctx, start, hq, h, D, T):
    """Queries of zero: every key has the same weight."""
    table, at, B = cache(ctx, rows, T, h, D, len(ctx))
    kc = normal((1, B, T, h, D), 1)
    vc = torch.zeros((1, B, T, h, D), dtype=BF16, device=dev())
    q = torch.zeros((sum(rows), hq, D), dtype=BF16, device=dev())
    call = kv.kv_attention_tree(q, kc, vc, table, i32(starts(rows)), i32(ctx), max_rows=max(rows),
                                span_start=None if start is None else i32(start), prepare=True)
    first = [0] * len(ctx) if start is None else start
    for t in range(turns(max(c + m for c, m in zip(ctx, rows)), UNIT, D)):
        fill(vc, at, ctx, rows, UNIT, D, t)
        want = np.concatenate([shares(c + 1 + np.arange(m), UNIT, D, t, first=s) for c, m, s in zip(ctx, rows, first)])
        got = call().double().cpu().numpy()
        bad = wrong(got, np.repeat(want[:, None], hq, 1))
        assert not bad.any(), f"turn {t}: {bad.sum()} of {bad.size} wrong, first at {np.argwhere(bad)[0]}"


@pytest.mark.parametrize("rows,ctx", [([1], [1009]), ([8], [1001]), ([5], [9007]), ([64], [7011]),
                                      ([3, 1, 1, 16, 2, 64], [7000, 1, 0, 3, 5001, 64])])
@pytest.mark.parametrize("hq,h,D", HEADS)
@pytest.mark.parametrize("T", [16, 20])
def test_picks_each_key(rows, ctx, hq, h, D, T):
    """Each query's logit is 90 or more (in log2) above the others' at one key: its output is that value row."""
    table, at, B = cache(ctx, rows, T, h, D, len(ctx))
    kc, vc = torch.zeros((1, B, T, h, D), dtype=BF16, device=dev()), normal((1, B, T, h, D), 2)
    n, group = sum(rows), hq // h
    row, head = np.arange(n)[:, None], np.arange(hq)[None]
    channel = (row + 31 * head) % D
    q = torch.zeros((n, hq, D), dtype=BF16, device=dev())
    q[torch.from_numpy(row).to(dev()), torch.from_numpy(head).to(dev()), torch.from_numpy(channel).to(dev())] = 1024
    call = kv.kv_attention_tree(q, kc, vc, table, i32(starts(rows)), i32(ctx), max_rows=max(rows), prepare=True)
    seen = np.concatenate([c + 1 + np.arange(m) for c, m in zip(ctx, rows)])[:, None]
    first = np.repeat(starts([c + m for c, m in zip(ctx, rows)])[:-1], rows)[:, None]
    values = vc[0].flatten(0, 1)
    for t in range(turns(max(c + m for c, m in zip(ctx, rows)), 1, D)):
        fill(kc, at, ctx, rows, 1, D, t)
        key = t * D + channel
        visible = torch.from_numpy(key < seen).to(dev())
        place = at[torch.from_numpy(np.where(key < seen, first + key, 0)).to(dev())]
        want = values[place, torch.from_numpy(head // group).to(dev()).expand_as(place)]
        assert torch.equal(call()[visible], want[visible]), f"turn {t}"
