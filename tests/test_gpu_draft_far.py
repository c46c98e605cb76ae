"""A step with drafted rows at the ends of its range: caches and probabilities past 2^31 elements,
groups of heads that share tiles of 128 rows unevenly, blocks of any size with values that are not finite."""
import numpy as np
import pytest
import torch

import operator_refs as ref
import paged_kv_cache_39_gb300 as kv
from operator_refs import BF16, dev, normal
from step_refs import ancestors, as_int64, attend, block_table, i32, random_tree, starts
from test_gpu_attention_tree import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group", [3, 5, 6, 7, 12, 16, 48, 64])
@pytest.mark.parametrize("rows", [[64, 50], [21, 7, 30]])
@pytest.mark.parametrize("D", [64, 72, 128])
def test_groups_that_divide_a_tile_and_that_do_not(group, rows, D):
    run(rows, [70, 300, 5][:len(rows)], hq=2 * group, h=2, D=D, seed=group + D)


@pytest.mark.parametrize("group", [4, 6])
@pytest.mark.parametrize("tail", [0, 9])
def test_the_last_requests_rows_end_with_the_query(group, tail):
    """A tile's rows reach past the last row; those of the next request are other rows."""
    run([1, 33, 2, 40], [40, 40, 300, 9], hq=2 * group, h=2, D=128, seed=50 + group, tail=tail, max_rows=64)


@pytest.mark.parametrize("T", [5, 8, 20])
@pytest.mark.parametrize("rows", [3, 40])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_values_not_finite_in_any_block(T, rows, what):
    """Hidden ones change nothing, a seen one its channel in the rows that see it."""
    h, hq, D, ctx = 2, 8, 64, 53
    rng = np.random.default_rng(60)
    table, B = block_table([ctx + rows], T, rng)
    kc, vc = normal((1, B, T, h, D), 61), normal((1, B, T, h, D), 62)
    q = normal((rows, hq, D), 63)
    masks = ancestors(random_tree(rows, rng))
    args = (i32(table), i32([0, rows]), i32([ctx]))
    clean = kv.kv_attention_tree(q, kc, vc, *args, max_rows=rows, tree_mask=as_int64(masks))
    used = np.zeros(B * T, bool)
    used[[table[0, p // T] * T + p % T for p in range(ctx + rows)]] = True
    for cache in (kc, vc):
        cache[0].flatten(0, 1)[torch.from_numpy(np.nonzero(~used)[0]).to(dev())] = what
    at = ctx + 1
    vc[0, table[0, at // T], at % T, 1, 17] = what
    got = kv.kv_attention_tree(q, kc, vc, *args, max_rows=rows, tree_mask=as_int64(masks))
    want = clean.clone()
    sees = [i for i in range(rows) if masks[i] >> 1 & 1]
    want[sees, 4:, 17] = what
    assert len(sees) < rows
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(nan=0.0), want.nan_to_num(nan=0.0))


def test_cache_past_two_to_the_31st_element():
    """Blocks at both ends of a pool of 2^31 elements a layer and of the second layer, rows moved there."""
    T, h, D, L, ctx, rows = 16, 8, 128, 2, 40, 6
    B = 2 ** 31 // (T * h * D) + 5
    kc, vc = (torch.zeros((L, B, T, h, D), dtype=BF16, device=dev()) for _ in range(2))
    table = np.asarray([[1, B - 1, 2], [B - 2, B - 3, B // 2 + 1]], np.int32)
    for i, b in enumerate(table.flatten()):
        for layer in range(L):
            kc[layer, b] = normal((T, h, D), 70 + 4 * i + layer)
            vc[layer, b] = normal((T, h, D), 72 + 4 * i + layer)
    q = normal((2 * rows, 32, D), 69)
    err = kv.new_error_word(dev())
    at = torch.from_numpy(np.stack([[table[r, p // T].astype(np.int64) * T + p % T for p in range(ctx + rows)]
                                    for r in range(2)])).to(dev())
    for layer in range(L):
        got = kv.kv_attention_tree(q, kc, vc, i32(table), i32([0, rows, 2 * rows]), i32([ctx, ctx]), max_rows=rows,
                                   layer=layer, err=err)
        for r in range(2):
            seen = np.arange(ctx + rows) <= ctx + np.arange(rows)[:, None]
            o, bound = attend(q[r * rows:(r + 1) * rows], kc[layer].flatten(0, 1)[at[r]],
                              vc[layer].flatten(0, 1)[at[r]], seen, D ** -0.5)
            ref.check(got[r * rows:(r + 1) * rows], o, bound, f"layer {layer} request {r}")
    want = [c.flatten(1, 2)[:, at].clone() for c in (kc, vc)]
    for w in want:
        w[:, :, ctx + 1:ctx + 3] = w[:, :, [ctx + 2, ctx + 5]].clone()
    kv.kv_cache_keep_path(kc, vc, i32(table), i32([0, rows, 2 * rows]), i32([ctx, ctx]),
                          i32([0, 2, 5, -1, -1, -1] * 2), i32([2, 2]), err=err)
    for c, w in zip((kc, vc), want):
        assert torch.equal(c.flatten(1, 2)[:, at], w)
    assert err.item() == 0


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
def test_probabilities_past_two_to_the_31st_element(dtype):
    """Rows 2^31 / 3 elements apart: the last one begins past 2^31."""
    V, apart = 1000, 2 ** 31 // 3 + 8
    wide = torch.empty(3 * apart + V, dtype=dtype, device=dev())
    target = wide.as_strided((4, V), (apart, 1))
    p = torch.softmax(torch.arange(4 * V, device=dev()).view(4, V).float().sin() * 3, 1).to(dtype)
    target.copy_(p)
    tokens, uniform = i32([0, 3, 8, 14]), torch.tensor([0.37, 0.0, 0.0, 0.0], device=dev())
    args = (tokens, i32(starts([4])), uniform)
    want = kv.kv_verify_drafts(p, *args)
    got = kv.kv_verify_drafts(target, *args)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert want[2].tolist() == [3]      # a number of 0 keeps what has a probability
    last = p[3].double().cumsum(0)
    assert want[0][3].item() == int((last > 0.37 * last[-1]).nonzero()[0])
