"""kv_attention_tree against its formula in 64 bits."""
import numpy as np
import pytest
import torch

import operator_refs as ref
import paged_kv_cache_39_gb300 as kv
from operator_refs import BF16, dev, normal
from step_refs import ancestors, as_int64, attend, block_table, i32, random_tree, starts

pytestmark = pytest.mark.gpu


def places(table, B, T, lo, hi):
    """(position, slot) of the positions [lo, hi) that the table maps, and error bits."""
    pos = np.arange(lo, hi)
    bits = 0
    if len(pos) and pos[-1] // T >= len(table):
        bits |= kv.ERR_BITS["BAD_POSITION"]
    pos = pos[pos // T < len(table)]
    b = table[pos // T].astype(np.int64)
    if ((b < 0) | (b >= B)).any():
        bits |= kv.ERR_BITS["BAD_BLOCK"]
    ok = (b > 0) & (b < B)
    return pos[ok], b[ok] * T + pos[ok] % T, bits


def run(rows, ctx, T=16, hq=8, h=2, D=128, seed=0, masks="tree", start=None, table=None, scale=None,
        q_scale=1.0, layer=1, max_rows=None, spoil=None, tail=0, pool=0):
    rng = np.random.default_rng(seed)
    t, B = block_table([c + m for c, m in zip(ctx, rows)], T, rng, spare=3 + pool)
    table = t if table is None else table(t, B)
    kc, vc = normal((2, B, T, h, D), seed + 1), normal((2, B, T, h, D), seed + 2)
    n = sum(rows)
    q = normal((n + tail, hq + 3, D), seed + 3, q_scale)[:, 1:hq + 1]     # strided rows
    if masks == "tree":
        bits = [x for m in rows for x in ancestors(random_tree(m, rng))]
    elif masks == "random":   # rows that see nothing of the step, rows that see later ones
        bits = [int(x) for x in rng.integers(0, 2 ** 64, n, dtype=np.uint64) & rng.integers(0, 2 ** 64, n, dtype=np.uint64)]
    elif masks is None:
        bits = [(2 << i) - 1 for m in rows for i in range(m)]
    else:
        bits = masks
    if spoil is not None:
        spoil(kc, vc, table, T)
    begin = starts(rows)
    out = torch.full((n + tail, hq, D), 7.0, dtype=BF16, device=dev())
    err = kv.new_error_word(dev())
    got = kv.kv_attention_tree(q, kc, vc, i32(table), i32(begin), i32(ctx),
                               max_rows=max(max(rows), 1) if max_rows is None else max_rows,
                               tree_mask=None if masks is None else as_int64(bits + [2 ** 64 - 1] * tail),
                               span_start=None if start is None else i32(start), layer=layer,
                               scale=scale, out=out, err=err)
    assert got is out and (out[n:] == 7.0).all()
    want_err = 0
    scale = D ** -0.5 if scale is None else scale
    for r, (m, c) in enumerate(zip(rows, ctx)):
        s = 0 if start is None else int(start[r])
        if m and (s < 0 or c < s):
            want_err |= kv.ERR_BITS["BAD_POSITION"]
            assert not got[begin[r]:begin[r + 1]].any()
            continue
        pos, slot, e = places(table[r], B, T, s, c + m)
        if m:
            want_err |= e
        seen = np.asarray([[p < c or (bits[begin[r] + i] >> int(p - c)) & 1 == 1 for p in pos] for i in range(m)],
                          bool).reshape(m, len(pos))
        slot = torch.from_numpy(slot).to(dev())
        k, v = kc[layer].flatten(0, 1)[slot], vc[layer].flatten(0, 1)[slot]
        o, bound = attend(q[begin[r]:begin[r + 1]], k, v, seen, scale)
        ref.check(got[begin[r]:begin[r + 1]], o, bound, f"request {r} rows {m} ctx {c}")
    assert err.item() == want_err
    return got


@pytest.mark.parametrize("D", [64, 80, 128, 8])
@pytest.mark.parametrize("hq,h", [(1, 1), (4, 4), (8, 2), (6, 2), (8, 1), (24, 3), (35, 5), (33, 1), (64, 1)])
def test_head_groups(hq, h, D):
    run([1, 3, 9, 1, 2], [1, 0, 17, 100, 257], hq=hq, h=h, D=D, seed=hq + D)


@pytest.mark.parametrize("m", [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64])
@pytest.mark.parametrize("masks", ["tree", None, "random"])
def test_rows_and_masks(m, masks):
    run([m, 1, m, 64], [130, 5, 0, 300], seed=m, masks=masks, max_rows=64)


@pytest.mark.parametrize("T", [1, 3, 8, 12, 16, 20, 48, 128, 200, 528])
def test_block_sizes(T):
    run([2, 4, 5, 1, 9, 33], [1, T - 1, T, T + 1, 3 * T + 5, 700], T=T, seed=T)


@pytest.mark.parametrize("end", [126, 127, 128, 129, 255, 256, 257])
def test_keys_around_the_tiles_ends(end):
    run([1, 2, 5], [end - 1, end - 2, end - 3], seed=end)


@pytest.mark.parametrize("D", [64, 128])
def test_long_and_short_together(D):
    run([3, 1, 1, 16, 2, 64], [20000, 1, 0, 3, 5001, 64], hq=8, h=2, D=D, seed=7)


def test_one_long_request():
    run([5], [40007], seed=8)


def test_one_long_request_of_many_rows():
    run([64], [30011], hq=16, h=2, seed=8)


def test_many_requests():
    rng = np.random.default_rng(9)
    run(list(rng.integers(0, 9, 300)), list(rng.integers(0, 300, 300)), hq=4, h=1, D=64, seed=9)


def test_more_requests_than_a_block_of_threads_scans():
    rng = np.random.default_rng(10)
    run(list(rng.integers(0, 3, 1500)), list(rng.integers(0, 40, 1500)), hq=4, h=2, D=64, seed=10)


def test_empty_contexts_and_rows_that_see_nothing():
    got = run([4, 1, 3], [0, 0, 0], masks=[0, 1, 2, 15, 0, 0, 0, 7], seed=11)
    assert not got[0].any() and not got[4].any() and not got[5].any()


def test_bits_past_the_rows_mean_nothing():
    run([3, 2], [40, 17], masks=[2 ** 64 - 1] * 5, seed=12)


def test_spans_that_start_late_are_empty_or_invalid():
    run([2, 2, 3, 1, 2, 2, 2], [100, 300, 100, 50, 77, 40, 400], seed=13, start=[0, 37, 99, 50, -1, 41, 256])


def test_null_bad_and_missing_table_entries():
    def spoil(t, B):
        t[0, :3] = 0                  # recycled blocks
        t[1, 1] = B                   # outside the pool
        t[2, 0] = -5
        t[3, :] = 0                   # nothing left
        return t[:, :5].copy()        # positions 80.. have no entry
    got = run([2, 1, 3, 2, 4], [75, 63, 30, 58, 96], seed=14, table=spoil)
    assert not got[6].any() and not got[7].any()


def test_rows_behind_the_last_request_stay():
    run([3, 0, 2], [40, 12, 17], seed=15, tail=4)


def test_rows_out_of_order_or_too_many():
    T, h, D = 16, 1, 64
    kc, vc = normal((1, 9, T, h, D), 1), normal((1, 9, T, h, D), 2)
    q = normal((8, 2, D), 3)
    for qs, most, good in (([0, 3, 1, 2], 4, (0, 2)), ([0, 2, 4, 9], 4, (0, 1)), ([-1, 1, 2, 4], 4, (1, 2)),
                           ([0, 4, 5, 7], 3, (1, 2))):
        out = torch.full((8, 2, D), 7.0, dtype=BF16, device=dev())
        err = kv.new_error_word(dev())
        table = i32([[1, 2], [3, 4], [5, 6]])
        kv.kv_attention_tree(q, kc, vc, table, i32(qs), i32([9, 10, 11]), max_rows=most, out=out, err=err)
        assert err.item() == kv.ERR_BITS["BAD_QSL"]
        claimed = torch.zeros(8, dtype=torch.bool)
        for r in good:
            claimed[qs[r]:qs[r + 1]] = True
            alone = kv.kv_attention_tree(q[qs[r]:qs[r + 1]], kc, vc, table[r:r + 1], i32([0, qs[r + 1] - qs[r]]),
                                         i32([9 + r]), max_rows=most)
            if qs != [0, 3, 1, 2]:      # there two requests claim row 1
                assert torch.equal(out[qs[r]:qs[r + 1]], alone)
        assert (out[~claimed] == 7.0).all()


@pytest.mark.parametrize("scale,q_scale", [(0.5, 1.0), (None, 30.0), (1e-4, 1.0), (None, 1e-3)])
def test_scales(scale, q_scale):
    run([3, 9], [300, 40], seed=16, scale=scale, q_scale=q_scale)


def test_maximum_that_keeps_rising():
    """Logits that grow along the keys, so that every tile raises the reference."""
    def spoil(kc, vc, table, T):
        b = torch.from_numpy(table[0, :-1]).to(dev()).long()
        grow = torch.arange(len(b), device=dev()).to(BF16)[:, None, None, None] * 0.5
        kc[1, b] = (kc[1, b] * 0.1 + grow * 0.05).to(BF16)
    run([2], [1500], seed=17, spoil=spoil, q_scale=1.0)


@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("rows", [3, 40])
def test_values_not_finite_in_hidden_places(what, rows):
    """Behind the rows, in other rows' places and in blocks of others: nothing of it is seen."""
    T, h, D, ctx = 16, 2, 128, 53
    rng = np.random.default_rng(18)
    table, B = block_table([ctx + rows], T, rng)
    kc, vc = normal((1, B, T, h, D), 19), normal((1, B, T, h, D), 20)
    q = normal((rows, 8, D), 21)
    parents = random_tree(rows, rng)
    masks = ancestors(parents)
    leaf = next(j for j in range(rows - 1, 0, -1) if all(not masks[i] >> j & 1 for i in range(rows) if i != j))
    clean = kv.kv_attention_tree(q, kc, vc, i32(table), i32([0, rows]), i32([ctx]), max_rows=rows,
                                 tree_mask=as_int64(masks))
    used = np.zeros(B * T, bool)
    used[[table[0, p // T] * T + p % T for p in range(ctx + rows)]] = True
    hidden = torch.from_numpy(np.nonzero(~used)[0]).to(dev())
    for cache in (kc, vc):
        cache[0].flatten(0, 1)[hidden] = what
    p = ctx + leaf
    for cache in (kc, vc):
        cache[0, table[0, p // T], p % T] = what       # a leaf: seen by its own row alone
    got = kv.kv_attention_tree(q, kc, vc, i32(table), i32([0, rows]), i32([ctx]), max_rows=rows,
                               tree_mask=as_int64(masks))
    others = [i for i in range(rows) if i != leaf]
    assert torch.equal(got[others], clean[others])


@pytest.mark.parametrize("at", ["context", "row"])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_values_not_finite_in_seen_places(what, at):
    T, h, D, ctx, rows = 16, 2, 128, 200, 5
    table, B = block_table([ctx + rows], T, np.random.default_rng(22))
    kc, vc = normal((1, B, T, h, D), 23), normal((1, B, T, h, D), 24)
    q = normal((rows, 8, D), 25)
    args = (i32(table), i32([0, rows]), i32([ctx]))
    clean = kv.kv_attention_tree(q, kc, vc, *args, max_rows=rows)
    p = 77 if at == "context" else ctx + 2
    vc[0, table[0, p // T], p % T, 1, 40] = what
    got = kv.kv_attention_tree(q, kc, vc, *args, max_rows=rows)
    sees = list(range(rows)) if at == "context" else [2, 3, 4]
    for i in range(rows):
        bad = ~torch.isfinite(got[i].float())
        want = torch.zeros_like(bad)
        if i in sees:
            want[4:, 40] = True            # the query heads of KV head 1
        assert torch.equal(bad, want)
        assert torch.equal(got[i][~bad], clean[i][~want])


def test_rows_whose_logits_are_all_minus_infinity():
    T, h, D = 16, 1, 64
    kc, vc = normal((1, 6, T, h, D), 26), normal((1, 6, T, h, D), 27)
    kc[0, 1:3, :, 0, 0] = -float("inf")
    q = normal((2, 1, D), 28).abs() + 0.1
    kc[..., 1:] = kc[..., 1:].abs() * 0.01
    out = kv.kv_attention_tree(q, kc, vc, i32([[1, 2, 0]]), i32([0, 2]), i32([30]), max_rows=2)
    assert not out.any()


def test_decode_equals_the_row_of_a_chain():
    """One row a request over a cache, as the last row of a longer chain sees it."""
    T, h, hq, D, ctx = 16, 2, 8, 128, 90
    table, B = block_table([ctx + 9], T, np.random.default_rng(29))
    kc, vc = normal((1, B, T, h, D), 30), normal((1, B, T, h, D), 31)
    q = normal((9, hq, D), 32)
    chain = kv.kv_attention_tree(q, kc, vc, i32(table), i32([0, 9]), i32([ctx]), max_rows=9)
    for i in range(9):
        one = kv.kv_attention_tree(q[i:i + 1], kc, vc, i32(table), i32([0, 1]), i32([ctx + i]), max_rows=1)
        assert (one.float() - chain[i:i + 1].float()).abs().max() < 2.0 ** -6
