"""kv_attention_q4 where value scales differ: every channel group against its own size, at fp16's
step for the weights."""
import numpy as np
import pytest
import torch

import operator_refs as ref
import paged_kv_cache_39_gb300 as kv
from operator_refs import BF16, dev, normal
from test_gpu_attention_q4 import layout
from test_gpu_cache_q4 import i32, random_cache

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -11   # weight times scale, rounded to fp16


def scales_of(cache, T, D):
    """A copy of a cache's scales as float64 [layers, blocks, heads, T, groups]."""
    return cache[..., T * D // 2:].clone().view(BF16).to(ref.F64).unflatten(-1, (T, D // 32))


def set_scales(cache, T, D, s):
    cache[..., T * D // 2:] = s.to(BF16).flatten(-2).contiguous().view(torch.uint8)


def check(q, kc, vc, table, n, T, D, start=0):
    """One request of positions [start, n), at the default scale."""
    got = kv.kv_attention_q4(q, kc, vc, i32(table), i32([start]), i32([n]), T)
    p = np.arange(start, n)
    slots = table[0, p // T].astype(np.int64) * T + p % T
    k, v = ref.values(kc, T, D, 0, slots), ref.values(vc, T, D, 0, slots)
    seen, scale = [len(slots)], D ** -0.5
    o, bound = ref.attend(q, k, v, seen, scale, STEP)
    # The product's operand of a token in a group is weight times scale, times a power of two that
    # puts the group's largest one at 2^7 or above: one below 2^-14, fp16's normal range, is off by
    # 2^-25 at most, 2^-32 of the largest, and that counts times a code of up to 8.
    s = scales_of(vc, T, D)[0][torch.as_tensor(slots // T, device=dev()), :,
                               torch.as_tensor(slots % T, device=dev())].abs()       # [n, h, groups]
    h, g = s.shape[1:]
    x = torch.einsum("hgd,nhd->hgn", q[0].to(ref.F64).view(h, -1, D), k) * scale
    w = torch.softmax(x, -1)
    top = torch.stack([(w * s[:, :, j].T[:, None]).amax(-1) for j in range(g)], -1)  # [h, heads, g]
    bound = bound + len(slots) * 2.0 ** -29 * top.repeat_interleave(32, -1).reshape(1, -1, D)
    ref.check(got, o, bound, f"n={n} D={D}")


def make(n, T, hq, h, D, seed):
    table, B = layout([n], T, seed)
    return (table, random_cache(1, B, T, h, D, seed + 1), random_cache(1, B, T, h, D, seed + 2),
            normal((1, hq, D), seed + 3))


@pytest.mark.parametrize("hq,h", [(4, 1), (8, 1), (16, 1), (6, 2), (33, 1)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("apart", [0, 12, 20, 30])
def test_groups_far_apart(apart, D, hq, h):
    """A head's groups lie powers of two apart, in either order, in every token."""
    n, T = 1000, 16
    table, kc, vc, q = make(n, T, hq, h, D, apart + hq)
    s = scales_of(vc, T, D)
    for order in (1, -1):
        e = torch.arange(D // 32, device=dev()) * apart
        e = e if order > 0 else e.flip(0)
        set_scales(vc, T, D, s * 2.0 ** -e.double())
        check(q, kc, vc, table, n, T, D)


@pytest.mark.parametrize("n", [1, 15, 33, 700, 9001])
@pytest.mark.parametrize("hq,h,D", [(32, 8, 128), (8, 1, 128), (16, 1, 64)])
def test_ordinary_scales(n, hq, h, D):
    table, kc, vc, q = make(n, 16, hq, h, D, n)
    check(q, kc, vc, table, n, 16, D)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("spread", [6, 20, 40])
def test_scales_of_every_token_by_themselves(spread, D):
    n, T = 600, 16
    table, kc, vc, q = make(n, T, 8, 2, D, spread)
    g = torch.Generator(device="cuda").manual_seed(spread)
    s = scales_of(vc, T, D)
    e = torch.randint(-spread, spread + 1, s.shape, generator=g, device="cuda").double()
    s = s * 2.0 ** e
    s[torch.rand(s.shape, generator=g, device="cuda") < 0.2] = 0
    set_scales(vc, T, D, s)
    check(q, kc, vc, table, n, T, D)


@pytest.mark.parametrize("D", [64, 128])
def test_groups_that_appear_or_leave_along_the_context(D):
    """Zero, then tiny, then huge, then tiny again, group by group at other places."""
    n, T = 2500, 16
    table, kc, vc, q = make(n, T, 8, 2, D, 5)
    s = scales_of(vc, T, D)
    size = torch.zeros((n, D // 32), device=dev(), dtype=ref.F64)
    for j in range(D // 32):
        for i, f in enumerate((0.0, 2.0 ** -50, 2.0 ** 30, 2.0 ** -20, 1.0)):
            lo = 97 * j + 480 * i
            size[lo:, j] = f
    p = torch.arange(n, device=dev())
    blk = torch.as_tensor(table[0], device=dev()).long()[p // T]
    s[0, blk, :, p % T] *= size[:, None]
    set_scales(vc, T, D, s)
    check(q, kc, vc, table, n, T, D)
    check(q, kc, vc, table, 1200, T, D, start=470)


@pytest.mark.parametrize("slope", [0.05, -0.05, 1.0])
@pytest.mark.parametrize("D", [64, 128])
def test_logits_that_grow_or_fall(D, slope):
    """References rise again and again (or weights vanish), with groups 2^-20 apart."""
    n, T, h = 900, 16, 2
    table, kc, vc, q = make(n, T, 8, h, D, 6)
    row = (torch.arange(n, device=dev())[:, None, None] * slope * torch.ones((n, h, D), device=dev())).to(BF16)
    p = np.arange(n)
    slots = torch.as_tensor(table[0, p // T].astype(np.int64) * T + p % T, device=dev())
    kv.kv_cache_write_q4(row, row, kc, vc.clone(), slots, T)
    set_scales(vc, T, D, scales_of(vc, T, D) * 2.0 ** (-20 * torch.arange(D // 32, device=dev()).double()))
    check(torch.full_like(q, 0.25), kc, vc, table, n, T, D)


def test_a_heavy_token_among_many_light_ones():
    """One token's weight is 2^24 times the others', which together are not small beside it."""
    n, T, D = 1 << 18, 32, 64
    table, kc, vc, q = make(n, T, 4, 1, D, 7)
    k = torch.zeros((n, 1, D), dtype=BF16, device=dev())
    v = torch.ones_like(k)
    k[3], v[3] = 16.0, -1.0
    p = np.arange(n)
    slots = torch.as_tensor(table[0, p // T].astype(np.int64) * T + p % T, device=dev())
    kv.kv_cache_write_q4(k, v, kc, vc, slots, T)
    # 16 q sum(1) / 8 = 24 ln 2
    q = torch.full((1, 4, D), 24 * np.log(2) * 8 / (16 * D), device=dev()).to(BF16)
    check(q, kc, vc, table, n, T, D)
