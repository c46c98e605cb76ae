"""kv_cache_keep_path bit for bit."""
import numpy as np
import pytest
import torch

import paged_kv_cache_39_gb300 as kv
from operator_refs import BF16, dev, normal
from step_refs import block_table, i32, starts

pytestmark = pytest.mark.gpu


def random_path(m, rng):
    k = int(rng.integers(0, m))
    return [0] + sorted(int(x) for x in rng.choice(np.arange(1, m), k, replace=False)) if m > 1 else [0]


def expect(cache, table, T, ctx, paths):
    want = cache.clone()
    for r, path in enumerate(paths):
        if path is None:
            continue
        for i, j in enumerate(path):
            a, b = ctx[r] + j, ctx[r] + i
            want[:, table[r, b // T], b % T] = cache[:, table[r, a // T], a % T]
    return want


def run(rows, ctx, paths, L=3, T=16, h=2, D=64, seed=0, table=None, kept=None, flat=None, bits=0, skipped=()):
    rng = np.random.default_rng(seed)
    t, B = block_table([c + m for c, m in zip(ctx, rows)], T, rng)
    table = t if table is None else table(t, B)
    kc, vc = normal((L, B, T, h, D), seed + 1), normal((L, B, T, h, D), seed + 2)
    if flat is None:
        flat = [x for m, p in zip(rows, paths) for x in p + [-1] * (m - len(p))]
    if kept is None:
        kept = [len(p) - 1 if m else 0 for m, p in zip(rows, paths)]
    real = [None if r in skipped or rows[r] == 0 else p for r, p in enumerate(paths)]
    want = [expect(c, table, T, ctx, real) for c in (kc, vc)]
    err = kv.new_error_word(dev())
    assert kv.kv_cache_keep_path(kc, vc, i32(table), i32(starts(rows)), i32(ctx), i32(flat), i32(kept), err=err) is None
    assert torch.equal(kc.view(torch.int16), want[0].view(torch.int16))
    assert torch.equal(vc.view(torch.int16), want[1].view(torch.int16))
    assert err.item() == bits


@pytest.mark.parametrize("T", [1, 5, 8, 16, 48])
@pytest.mark.parametrize("h,D,L", [(2, 64, 3), (1, 8, 1), (8, 128, 2), (5, 80, 4), (3, 256, 1)])
def test_random_paths(T, h, D, L):
    rng = np.random.default_rng(T + D)
    rows = [1, 2, 9, 0, 64, 33, 17, 5]
    run(rows, [0, 7, 100, 3, 15, 16, 31, 64], [random_path(m, rng) if m else [] for m in rows], L=L, T=T, h=h, D=D, seed=T)


def test_whole_paths_and_the_longest_moves():
    run([64, 64, 64, 64], [3, 30, 9, 1],
        [list(range(64)), [0] + list(range(2, 64)), [0, 63], [0] + list(range(1, 64, 2))], seed=1)


def test_many_requests_and_many_layers():
    rng = np.random.default_rng(2)
    rows = [int(x) for x in rng.integers(1, 20, 500)]
    run(rows, list(rng.integers(0, 60, 500)), [random_path(m, rng) for m in rows], L=2, h=1, D=64, seed=3)
    run([12, 3], [70, 5], [[0, 2, 5, 9, 11], [0, 2]], L=40, h=4, D=128, seed=4)


def test_values_that_are_not_finite_move_bit_for_bit():
    T, L = 16, 2
    kc = torch.randint(-32768, 32767, (L, 5, T, 2, 64), dtype=torch.int16, device=dev(),
                       generator=torch.Generator(device="cuda").manual_seed(5)).view(BF16)
    vc = kc.flip(0).contiguous()
    want = [c.clone() for c in (kc, vc)]
    for w in want:
        w[:, 2, 5] = w[:, 2, 9].clone()
        w[:, 2, 6] = w[:, 3, 1].clone()
    kv.kv_cache_keep_path(kc, vc, i32([[2, 3]]), i32([0, 14]), i32([4]), i32([0, 5, 13] + [-1] * 11), i32([2]))
    for c, w in zip((kc, vc), want):
        assert torch.equal(c.view(torch.int16), w.view(torch.int16))


def test_paths_and_counts_that_are_none():
    rows, ctx = [5, 5, 5, 5, 5, 5], [4, 4, 4, 4, 4, 4]
    flat = [0, 2, 3, -1, -1,   0, 2, 2, -1, -1,   1, 2, 3, -1, -1,   0, 2, 5, -1, -1,   0, 2, 3, 4, -1,   0, 3, 4, -1, -1]
    paths = [[0, 2, 3], [0], [0], [0], [0], [0, 3, 4]]
    run(rows, ctx, paths, flat=flat, kept=[2, 2, 2, 2, 5, 2], bits=kv.ERR_BITS["BAD_TREE"], skipped=(1, 2, 3, 4), seed=6)
    run([3], [4], [[0]], kept=[-1], bits=kv.ERR_BITS["BAD_TREE"], skipped=(0,), seed=7)


def test_bad_blocks_and_positions():
    path = [0, 2, 12]
    flat_rows = [13, 13, 13, 13]

    def spoil(t, B):
        t[0, 0] = 0             # where a row would go
        t[1, 0] = B
        t[2, 0] = -4
        return t
    bits = kv.ERR_BITS["NULL_WRITE"] | kv.ERR_BITS["BAD_BLOCK"]
    run(flat_rows, [4, 4, 4, 4], [path] * 4, table=spoil, bits=bits, skipped=(0, 1, 2), seed=8)
    run([13, 13], [4, 1], [path] * 2, table=lambda t, B: t[:, :1].copy(), bits=kv.ERR_BITS["BAD_POSITION"],
        skipped=(0,), seed=9)
    run([13, 2], [4, 20], [path, [0]], kept=[2, 0], seed=10, bits=0)
    T = 16
    kc, vc = normal((1, 4, T, 1, 64), 11), normal((1, 4, T, 1, 64), 12)
    was = kc.clone()
    err = kv.new_error_word(dev())
    kv.kv_cache_keep_path(kc, vc, i32([[1, 2]]), i32([0, 3]), i32([-1]), i32([0, 2, -1]), i32([1]), err=err)
    assert err.item() == kv.ERR_BITS["BAD_POSITION"] and torch.equal(kc, was)


def test_rows_out_of_order():
    T = 16
    kc, vc = normal((1, 6, T, 1, 64), 13), normal((1, 6, T, 1, 64), 14)
    was = kc.clone()
    err = kv.new_error_word(dev())
    kv.kv_cache_keep_path(kc, vc, i32([[1], [2], [3]]), i32([0, 3, 2, 9]), i32([2, 2, 2]), i32([0, 2, -1]), i32([0, 1, 1]), err=err)
    assert err.item() == kv.ERR_BITS["BAD_QSL"] and torch.equal(kc, was)


def test_nothing_to_do():
    kc = torch.zeros((1, 4, 16, 1, 64), dtype=BF16, device=dev())
    kv.kv_cache_keep_path(kc, kc.clone(), i32(np.zeros((0, 2))), i32([0]), i32([]), i32([]), i32([]))
    kv.kv_cache_keep_path(kc, kc.clone(), i32([[1, 2]]), i32([0, 0]), i32([3]), i32([]), i32([0]))
