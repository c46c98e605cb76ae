"""kv_tree_layout against its rule."""
import numpy as np
import pytest
import torch

import paged_kv_cache_39_gb300 as kv
from operator_refs import dev
from step_refs import ancestors, as_int64, i32, random_tree, starts

pytestmark = pytest.mark.gpu


def expect(trees, ctx):
    masks = [x for p in trees for x in ancestors(p)]
    base = np.repeat(np.asarray(ctx, np.int64), [len(p) for p in trees])
    depth = np.asarray([bin(x).count("1") - 1 for x in masks])
    place = np.concatenate([np.arange(len(p)) for p in trees] or [np.zeros(0, int)])
    return as_int64(masks), torch.from_numpy(base + depth).to(dev()), torch.from_numpy(base + place).to(dev())


def check(trees, ctx, chain=False, err_bits=0, tail=0):
    rows = [len(p) for p in trees]
    n = sum(rows)
    flat = i32([x for p in trees for x in p] + [7] * tail)
    outs = [torch.full((n + tail,), -5, dtype=torch.int64, device=dev()) for _ in range(3)]
    err = kv.new_error_word(dev())
    got = kv.kv_tree_layout(None if chain else flat, i32(starts(rows)), i32(ctx), num_rows=n + tail,
                            tree_mask=outs[0], positions=outs[1], cache_positions=outs[2], err=err)
    for g, o, w in zip(got, outs, expect(trees, ctx)):
        assert g is o
        assert torch.equal(g[:n], w)
        assert (g[n:] == -5).all()
    assert err.item() == err_bits


@pytest.mark.parametrize("rows", [[1], [2], [8], [31], [32], [33], [63], [64], [1, 64, 0, 17, 0, 33, 2]])
def test_random_trees(rows):
    rng = np.random.default_rng(sum(rows))
    check([random_tree(m, rng) for m in rows], rng.integers(0, 2 ** 31 - 1, len(rows)))


def test_many_requests():
    rng = np.random.default_rng(3)
    check([random_tree(int(m), rng, 64) for m in rng.integers(0, 65, 777)], rng.integers(0, 9999, 777))


@pytest.mark.parametrize("chain", [False, True])
def test_chains(chain):
    check([list(range(-1, m - 1)) for m in (64, 1, 5, 33)], [0, 7, 100, 2 ** 31 - 1], chain=chain)


def test_stars_and_rows_behind_the_last_request():
    check([[-1] + [0] * 63, [-1, 0]], [5, 6], tail=9)


def test_parents_that_are_no_rows_before():
    trees = [[-1, 0, 2, 1, 3], [99, 0, 1, 64, 3], [-1, -1, 1]]  # row 0's is not read
    check(trees, [10, 20, 30], err_bits=kv.ERR_BITS["BAD_TREE"])


def test_negative_context():
    err = kv.new_error_word(dev())
    mask, pos, place = kv.kv_tree_layout(None, i32([0, 2, 4]), i32([-1, 3]), num_rows=4, err=err)
    assert mask.tolist() == [1, 3, 1, 3]
    assert pos.tolist() == place.tolist() == [-1, -1, 3, 4]
    assert err.item() == kv.ERR_BITS["BAD_POSITION"]


def test_rows_out_of_order_out_of_range_or_too_many():
    for qs in ([0, 3, 2, 6], [-1, 3, 4, 6], [0, 2, 4, 7], [0, 65, 65, 66]):
        n = 6 if qs[1] < 65 else 66
        outs = [torch.full((n,), -5, dtype=torch.int64, device=dev()) for _ in range(3)]
        err = kv.new_error_word(dev())
        kv.kv_tree_layout(None, i32(qs), i32([10, 20, 30]), num_rows=n, tree_mask=outs[0],
                          positions=outs[1], cache_positions=outs[2], err=err)
        assert err.item() == kv.ERR_BITS["BAD_QSL"]
        good = [r for r in range(3) if 0 <= qs[r] <= qs[r + 1] <= n and qs[r + 1] - qs[r] <= 64]
        want = [{-5} for _ in range(n)]
        for r in good:
            for i in range(qs[r + 1] - qs[r]):       # a row that two requests claim: either's
                want[qs[r] + i] = want[qs[r] + i] - {-5} | {10 * (r + 1) + i}
        assert all(x in w for x, w in zip(outs[2].tolist(), want))


def test_no_rows_and_no_requests():
    assert [x.numel() for x in kv.kv_tree_layout(None, i32([0, 0]), i32([3]), num_rows=0)] == [0, 0, 0]
    kv.kv_tree_layout(None, i32([0]), i32([]), num_rows=0)
