"""Every key of a context counts once: at the boundaries of units, tiles, warps' shares, parts of a
split and blocks, in both attentions."""
import numpy as np
import pytest
import torch

import operator_refs as ref
import paged_kv_cache_39_gb300 as kv
from key_patterns import marks, shares, turns, wrong
from operator_refs import BF16, dev, normal
from test_gpu_attention_q4 import layout
from test_gpu_cache_q4 import i32, random_cache

pytestmark = pytest.mark.gpu


def check(got, want, what):
    got = got.double().cpu().numpy()
    bad = wrong(got, want)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} wrong, first at {np.argwhere(bad)[0]}"


@pytest.mark.parametrize("ctx,start", [
    ([1], None), ([31, 32, 33], None), ([1009], None), ([4100], None), ([40007], None),
    ([20000, 1, 0, 3, 5001, 64], None), ([9001] + [1 + 37 * i % 90 for i in range(40)], None),
    ([3000, 2000, 700, 64], [37, 1999, 320, 0]),
])
@pytest.mark.parametrize("hq,h,D,T", [(32, 8, 128, 16), (4, 1, 128, 24), (8, 1, 128, 16), (33, 1, 128, 16),
                                      (6, 2, 64, 8), (16, 1, 64, 32)])
def test_attention_q4(ctx, start, hq, h, D, T):
    start = [0] * len(ctx) if start is None else start
    table, B = layout(ctx, T, len(ctx))
    kc, vc = random_cache(1, B, T, h, D, 1), random_cache(1, B, T, h, D, 2)
    n = max(ctx)
    q = torch.zeros((len(ctx), hq, D), dtype=BF16, device=dev())
    slots = [table[r, np.arange(c) // T].astype(np.int64) * T + np.arange(c) % T for r, c in enumerate(ctx)]
    at = torch.from_numpy(np.concatenate(slots)).to(dev())
    call = kv.kv_attention_q4(q, kc, vc, i32(table), i32(start), i32(ctx), T, prepare=True)
    one = 7 * float(torch.tensor(1 / 7).to(BF16))       # what a value of 1 is held as
    for t in range(turns(n, 32, D)):
        rows = np.concatenate([marks(c, 32, D, t) for c in ctx])
        rows = torch.from_numpy(rows).to(dev()).to(BF16)[:, None].expand(-1, h, -1).contiguous()
        kv.kv_cache_write_q4(rows, rows, random_cache(1, B, T, h, D, 3), vc, at, T)
        want = np.stack([shares([c], 32, D, t, first=s)[0] if c > s else np.zeros(D)
                         for c, s in zip(ctx, start)]) * one
        check(call(), np.repeat(want[:, None], hq, 1), f"turn {t}")


@pytest.mark.parametrize("new,total", [
    ([1000], [1000]), ([257], [257]), ([129, 1, 300], [129, 400, 640]),      # one wave
    ([600] * 40, [600] * 40), ([200] * 30, [500 + 7 * i for i in range(30)]),  # many
    ([16], [10000]), ([100], [3001]), ([20, 3], [2049, 1500]), ([5], [641]),   # clusters
])
@pytest.mark.parametrize("hq,h,d", [(32, 8, 128), (4, 4, 64), (6, 2, 80)])
def test_attention_prompt(new, total, hq, h, d):
    starts = lambda x: np.concatenate([[0], np.cumsum(x)])  # noqa: E731
    qs, ks = starts(new), starts(total)
    q = torch.zeros((qs[-1], hq, d), dtype=BF16, device=dev())
    k = normal((ks[-1], h, d), 1)
    v = torch.zeros((ks[-1], h, d), dtype=BF16, device=dev())
    seen = np.concatenate([np.arange(m) + n - m + 1 for m, n in zip(new, total)])
    call = kv.kv_attention_prompt(q, k, v, i32(qs), i32(ks), prepare=True)
    for t in range(turns(max(total), 1, d)):
        rows = np.concatenate([marks(n, 1, d, t) for n in total])
        v.copy_(torch.from_numpy(rows).to(dev())[:, None].expand(-1, h, -1))
        check(call(), np.repeat(shares(seen, 1, d, t)[:, None], hq, 1), f"turn {t}")


@pytest.mark.parametrize("new,total", [([257], [257]), ([129, 1, 300], [129, 400, 640]), ([300] * 40, [300] * 40),
                                       ([130], [3001]), ([20, 3], [2049, 1500])])
@pytest.mark.parametrize("hq,h,d", [(32, 8, 128), (4, 4, 64), (6, 2, 80)])
def test_attention_prompt_picks_each_key(new, total, hq, h, d):
    """Each query's logit is 90 or more above the others' at one key: its output is that value row."""
    starts = lambda x: np.concatenate([[0], np.cumsum(x)])  # noqa: E731
    qs, ks = starts(new), starts(total)
    row, head = np.arange(qs[-1])[:, None], np.arange(hq)[None]
    channel = (row + 31 * head) % d
    q = torch.zeros((qs[-1], hq, d), dtype=BF16, device=dev())
    q[torch.from_numpy(row).to(dev()), torch.from_numpy(head).to(dev()), torch.from_numpy(channel).to(dev())] = 1024
    k, v = torch.zeros((ks[-1], h, d), dtype=BF16, device=dev()), normal((ks[-1], h, d), 2)
    seen = np.concatenate([np.arange(m) + n - m + 1 for m, n in zip(new, total)])[:, None]
    first = np.repeat(ks[:-1], new)[:, None]
    call = kv.kv_attention_prompt(q, k, v, i32(qs), i32(ks), prepare=True)
    for t in range(turns(max(total), 1, d)):
        rows = np.concatenate([marks(n, 1, d, t) for n in total])
        k.copy_(torch.from_numpy(rows).to(dev())[:, None].expand(-1, h, -1))
        key = t * d + channel
        visible = torch.from_numpy(key < seen).to(dev())
        at = torch.from_numpy(np.where(key < seen, first + key, 0)).to(dev())
        want = v[at, torch.from_numpy(head // (hq // h)).to(dev()).expand_as(at)]
        assert torch.equal(call()[visible], want[visible]), f"turn {t}"


@pytest.mark.parametrize("ctx", [[1009], [33, 700, 1, 2100]])
@pytest.mark.parametrize("hq,h,D,T", [(32, 8, 128, 16), (8, 1, 128, 24), (16, 1, 64, 32)])
def test_attention_q4_picks_each_unit(ctx, hq, h, D, T):
    """Each query's logits are 85 or more above the others' in one unit of 32 keys: its output is the
    mean of their values, each off by its weight's rounding (fp16, 2^-11) and the sum's (32 bits)."""
    table, B = layout(ctx, T, len(ctx))
    kc, vc = random_cache(1, B, T, h, D, 1), random_cache(1, B, T, h, D, 2)
    slots = [table[r, np.arange(c) // T].astype(np.int64) * T + np.arange(c) % T for r, c in enumerate(ctx)]
    at = torch.from_numpy(np.concatenate(slots)).to(dev())
    group, units = hq // h, -(-max(ctx) // 32)
    q = torch.zeros((len(ctx), hq, D), dtype=BF16, device=dev())
    call = kv.kv_attention_q4(q, kc, vc, i32(table), i32([0] * len(ctx)), i32(ctx), T, prepare=True)
    values = [ref.values(vc, T, D, 0, s) for s in slots]
    for t in range(turns(max(ctx), 32, D)):
        rows = torch.from_numpy(np.concatenate([marks(c, 32, D, t) for c in ctx])).to(dev()).to(BF16)
        rows = rows[:, None].expand(-1, h, -1).contiguous()
        kv.kv_cache_write_q4(rows, rows, kc, random_cache(1, B, T, h, D, 3), at, T)
        for u0 in range(t * D, min(units, t * D + D), group):
            q.zero_()
            for g in range(min(group, units - u0)):
                q[:, g::group, (u0 + g) % D] = 1024
            got = call().double()
            for r, c in enumerate(ctx):
                for g in range(group):
                    lo = 32 * (u0 + g)
                    if lo >= min(c, 32 * D * (t + 1)):
                        continue
                    x = values[r][lo:min(c, lo + 32)]
                    want, size = x.mean(0), x.abs().mean(0)
                    d = (got[r, g::group] - want).abs()
                    assert (d <= want.abs() * 2.0 ** -8 + size * (2.0 ** -11 + 2.0 ** -16)).all(), (r, u0 + g)
