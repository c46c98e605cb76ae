"""kv_attention_q4 against its formula in 64 bits."""
import numpy as np
import pytest
import torch

import operator_refs as ref
import paged_kv_cache_39_gb300 as kv
from operator_refs import BF16, dev, normal
from test_gpu_cache_q4 import i32, random_cache

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -8   # the weights keep at least bf16's bits


def layout(ctx, T, seed, spare=3):
    """A table of permuted blocks for contexts `ctx`, and the pool's size."""
    rng = np.random.default_rng(seed)
    need = [-(-int(n) // T) for n in ctx]
    B = sum(need) + 1 + spare
    order = rng.permutation(np.arange(1, B))
    table = np.zeros((len(ctx), max(max(need), 1) + 1), np.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    return table, B


def expect(q, kc, vc, table, start, end, T, D, layer, scale):
    B = kc.shape[1]
    outs, bounds, bits = [], [], 0
    for r in range(q.shape[0]):
        slots = []
        if start[r] < 0 or end[r] < start[r]:
            bits |= kv.ERR_BITS["BAD_POSITION"]
        else:
            for lb in range(start[r] // T, -(-int(end[r]) // T)):
                lo, hi = max(start[r], lb * T), min(end[r], (lb + 1) * T)
                if hi <= lo:
                    continue
                if lb >= table.shape[1]:
                    bits |= kv.ERR_BITS["BAD_POSITION"]
                    continue
                b = int(table[r, lb])
                if b < 0 or b >= B:
                    bits |= kv.ERR_BITS["BAD_BLOCK"]
                elif b > 0:
                    slots.append(b * T + np.arange(lo % T, lo % T + hi - lo))
        slots = np.concatenate(slots) if slots else np.zeros(0, np.int64)
        k, v = ref.values(kc, T, D, layer, slots), ref.values(vc, T, D, layer, slots)
        o, b = ref.attend(q[r:r + 1], k, v, [len(slots)], scale, STEP,
                          unit=ref.units(vc, T, D, layer, slots))
        outs.append(o)
        bounds.append(b)
    return torch.cat(outs), torch.cat(bounds), bits


def run(ctx, T, hq, h, D, seed=0, start=None, table=None, scale=None, layer=1, q_scale=1.0):
    t, B = layout(ctx, T, seed)
    table = t if table is None else table(t, B)
    kc, vc = random_cache(2, B, T, h, D, seed + 1), random_cache(2, B, T, h, D, seed + 2)
    q = normal((len(ctx), hq + 3, D), seed + 3, q_scale)[:, 1:hq + 1]   # strided rows
    start = np.zeros(len(ctx), np.int64) if start is None else np.asarray(start)
    err = kv.new_error_word(dev())
    got = kv.kv_attention_q4(q, kc, vc, i32(table), i32(start), i32(ctx), T, layer=layer, scale=scale, err=err)
    o, b, bits = expect(q, kc, vc, table, start, np.asarray(ctx), T, D, layer,
                        D ** -0.5 if scale is None else scale)
    ref.check(got, o, b, f"T={T} hq={hq} h={h} D={D}")
    assert err.item() == bits
    return got


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hq,h", [(1, 1), (4, 4), (8, 2), (6, 2), (8, 1), (24, 3), (16, 1), (35, 5), (33, 1)])
def test_head_groups(hq, h, D):
    run([1, 5, 16, 17, 33, 100, 257], 16, hq, h, D, seed=hq)


@pytest.mark.parametrize("T", [8, 16, 24, 48, 528])
def test_block_sizes(T):
    run([1, T - 1, T, T + 1, 3 * T + 5, 700], T, 8, 2, 128, seed=T)


@pytest.mark.parametrize("D", [64, 128])
def test_long_and_short_together(D):
    run([20000, 1, 0, 3, 5001, 64], 16, 8, 2, D, seed=7)


def test_one_long_request():
    run([40007], 16, 8, 2, 128, seed=8)


def test_many_requests():
    rng = np.random.default_rng(9)
    run(list(rng.integers(0, 300, 300)), 16, 4, 1, 64, seed=9)


def test_spans_that_start_late_are_empty_or_invalid():
    ctx = [100, 100, 100, 50, 77, 40]
    got = run(ctx, 16, 8, 2, 128, seed=10, start=[0, 37, 99, 50, -1, 41])
    assert not got[3].any() and not got[4].any() and not got[5].any()


def test_null_bad_and_missing_table_entries():
    def spoil(t, B):
        t[0, :3] = 0                  # recycled blocks
        t[1, 1] = B                   # outside the pool
        t[2, 0] = -5
        t[3, :] = 0                   # nothing left
        return t[:, :5].copy()        # positions 80.. have no entry
    got = run([80, 64, 33, 60, 100], 16, 8, 2, 128, seed=11, table=spoil)
    assert not got[3].any()


@pytest.mark.parametrize("scale,q_scale", [(0.5, 1.0), (None, 30.0), (1e-4, 1.0), (None, 1e-3)])
def test_scales(scale, q_scale):
    run([300, 40], 16, 8, 2, 128, seed=12, scale=scale, q_scale=q_scale)


def test_values_of_very_different_size():
    """Value scales from 2^-40 to 2^40 within one context, and scales of zero."""
    T, D, h, n = 16, 128, 2, 200
    table, B = layout([n], T, 1)
    kc, vc = random_cache(1, B, T, h, D, 1), random_cache(1, B, T, h, D, 2)
    g = torch.Generator(device="cuda").manual_seed(3)
    e = torch.randint(-40, 41, (1, B, h, T * D // 32), generator=g, device="cuda")
    s = torch.ldexp(torch.ones((), device="cuda"), e).to(BF16)
    s[torch.rand(s.shape, generator=g, device="cuda") < 0.2] = 0
    vc[..., T * D // 2:] = s.view(torch.uint8)
    q = normal((1, 8, D), 4)
    got = kv.kv_attention_q4(q, kc, vc, i32(table), i32([0]), i32([n]), T)
    o, b, _ = expect(q, kc, vc, table, [0], [n], T, D, 0, D ** -0.5)
    ref.check(got, o, b)
    vc[..., T * D // 2:] = 0                       # every value is zero
    got = kv.kv_attention_q4(q, kc, vc, i32(table), i32([0]), i32([n]), T)
    assert not got.any()


def test_tiny_and_huge_value_scales():
    T, D, h, n = 16, 64, 1, 100
    table, B = layout([n], T, 1)
    for f in (2.0 ** -100, 2.0 ** 100):
        kc, vc = random_cache(1, B, T, h, D, 1), random_cache(1, B, T, h, D, 2)
        s = vc[..., T * D // 2:].clone().view(BF16)
        vc[..., T * D // 2:] = (s.float() * f).to(BF16).view(torch.uint8)
        q = normal((1, 4, D), 4)
        got = kv.kv_attention_q4(q, kc, vc, i32(table), i32([0]), i32([n]), T)
        o, b, _ = expect(q, kc, vc, table, [0], [n], T, D, 0, D ** -0.5)
        ref.check(got, o, b)


def test_rows_nobody_attends_may_hold_anything():
    """Tokens outside the span, in null blocks and other requests' are NaN and infinite."""
    T, D, h = 16, 128, 2
    table, B = layout([40, 40], T, 5)
    kc, vc = random_cache(1, B, T, h, D, 1), random_cache(1, B, T, h, D, 2)
    q = normal((2, 8, D), 4)
    args = (i32(table), i32([10, 0]), i32([37, 0]), T)
    want = kv.kv_attention_q4(q, kc, vc, *args)
    used = set(int(table[0, p // T]) * T + p % T for p in range(10, 37))
    for c, bad in ((kc, float("nan")), (vc, float("inf"))):
        s = c[..., T * D // 2:].clone().view(BF16).unflatten(-1, (T, D // 32))
        for b in range(B):
            for off in range(T):
                if b * T + off not in used:
                    s[0, b, :, off] = bad
        c[..., T * D // 2:] = s.flatten(-2).contiguous().view(torch.uint8)
    got = kv.kv_attention_q4(q, kc, vc, *args)
    assert torch.equal(got, want) and torch.isfinite(got.float()).all() and not got[1].any()


def test_not_finite_where_attended_is_seen():
    T, D, h = 16, 128, 2
    table, B = layout([40], T, 5)
    kc, vc = random_cache(1, B, T, h, D, 1), random_cache(1, B, T, h, D, 2)
    b = int(table[0, 1])
    vc[0, b, 1, T * D // 2 + 2:T * D // 2 + 4] = torch.tensor([0xc0, 0x7f], dtype=torch.uint8, device=dev())
    got = kv.kv_attention_q4(normal((1, 8, D), 4), kc, vc, i32(table), i32([0]), i32([40]), T).float()
    assert torch.isnan(got[0, 4:, 32:64]).all()
    got[0, 4:, 32:64] = 0
    assert torch.isfinite(got).all()


def test_results_repeat_bit_for_bit():
    ctx = [5000, 300, 1, 8000]
    table, B = layout(ctx, 16, 1)
    kc, vc = random_cache(1, B, 16, 8, 128, 1), random_cache(1, B, 16, 8, 128, 2)
    q = normal((4, 32, 128), 3)
    call = kv.kv_attention_q4(q, kc, vc, i32(table), i32([0] * 4), i32(ctx), 16, prepare=True)
    first = call().clone()
    for _ in range(20):
        call.result.fill_(9)
        assert torch.equal(call(), first)


def test_two_streams_and_a_graph():
    ctx = [3000, 700, 1500]
    table, B = layout(ctx, 16, 1)
    kc, vc = random_cache(1, B, 16, 8, 128, 1), random_cache(1, B, 16, 8, 128, 2)
    qs = [normal((3, 32, 128), s) for s in (3, 4)]
    args = (kc, vc, i32(table), i32([0] * 3), i32(ctx), 16)
    want = [kv.kv_attention_q4(q, *args).clone() for q in qs]
    calls = [kv.kv_attention_q4(q, *args, prepare=True) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    graphs = []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c()
        graphs.append(g)
    for _ in range(10):
        for s, g, c in zip(streams, graphs, calls):
            with torch.cuda.stream(s):
                c.result.zero_()
                g.replay()
        torch.cuda.synchronize()
        for c, w in zip(calls, want):
            assert torch.equal(c.result, w)


@pytest.mark.parametrize("D,hq,h", [(128, 32, 8), (64, 16, 2), (128, 9, 1)])
@pytest.mark.parametrize("count", [1, 7, 8, 28, 29, 60, 300])
def test_one_long_context_among_short_ones(count, D, hq, h):
    """Its parts are many for the few warps that join them, whatever the others need."""
    ctx = [1 + 37 * i % 90 for i in range(count)]
    ctx[count // 2] = 9001
    run(ctx, 16, hq, h, D, seed=count + D)
