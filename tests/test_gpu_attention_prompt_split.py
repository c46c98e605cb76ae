"""kv_attention_prompt where few rows stand behind many keys, so that a cluster of CTAs shares
each tile's keys: against the formula in 64 bits."""
import numpy as np
import pytest
import torch

import operator_refs as ref
import paged_kv_cache_39_gb300 as kv
from operator_refs import BF16, dev, normal
from test_gpu_attention_prompt import expect, run, starts
from test_gpu_cache_q4 import i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,h,d", [(8, 2, 128), (4, 1, 64), (5, 1, 80), (6, 6, 128), (128, 1, 8)])
@pytest.mark.parametrize("new,total", [
    ([16], [640]), ([16], [641]), ([1], [5000]), ([100], [2000]), ([300], [2300]),
    ([33, 5, 0, 64], [1500, 700, 0, 900]),       # some with few keys, one with nothing
    ([7, 1, 3], [2500, 1, 3]), ([3, 40], [0, 4000]), ([20, 10], [1300, 4]),
])
def test_few_rows_behind_many_keys(new, total, hq, h, d):
    run(new, total, hq, h, d, seed=sum(total) + d, tail=3)


@pytest.mark.parametrize("keys", [769, 1024, 1281, 2049, 3000, 4200, 10000])
def test_every_share_of_the_keys(keys):
    """One to sixteen parts, of two tiles and more."""
    run([20], [keys], 4, 1, 128, seed=keys)
    run([70], [keys], 16, 4, 64, seed=keys + 1)


def test_more_sequences_than_run_at_once_unsplit():
    """From all SMs idle but one to no split at all."""
    for count in (1, 9, 10, 15, 19, 25, 38, 50, 76, 77):
        run([3] * count, [800 + 7 * i for i in range(count)], 4, 1, 64, seed=count)


def test_logits_that_grow_or_fall_along_the_keys():
    """Each part's weights outgrow the earlier ones', or vanish beside them."""
    n, m, d = 3000, 30, 128
    q = torch.ones((m, 2, d), device=dev()).to(BF16)
    v = normal((n, 1, d), 3)
    for slope in (0.02, -0.02, 1.0):
        k = (torch.arange(n, device=dev())[:, None, None] * slope * torch.ones((n, 1, d), device=dev())).to(BF16)
        got = kv.kv_attention_prompt(q, k, v, i32([0, m]), i32([0, n]))
        o, b = expect(q, k, v, starts([m]), starts([n]), d ** -0.5)
        ref.check(got, o, b)


def test_parts_with_infinite_logits_only():
    """Every logit of the first parts is -inf: they count for nothing."""
    n, m, d = 3000, 10, 64
    q = torch.ones((m, 1, d), device=dev()).to(BF16)
    k = torch.full((n, 1, d), -40.0, device=dev()).to(BF16)
    k[:2500, 0, 5] = -float("inf")
    v = normal((n, 1, d), 3)
    got = kv.kv_attention_prompt(q, k, v, i32([0, m]), i32([0, n]))
    for i in range(m):
        want = v[2500:n - m + i + 1].to(ref.F64).mean(0)
        size = v[2500:n - m + i + 1].to(ref.F64).abs().mean(0)
        # equal weights are exactly 1: the sum's roundings (2^-24 each) and the output's
        ref.check(got[i], want, want.abs() * 2.0 ** -8 + size * n * 2.0 ** -23)


def test_keys_out_of_sight_may_hold_anything():
    m, n = 100, 2000
    q, k, v = normal((m, 8, 128), 1), normal((n + 50, 2, 128), 2), normal((n + 50, 2, 128), 3)
    call = lambda k, v: kv.kv_attention_prompt(q, k, v, i32([0, m]), i32([0, n]))  # noqa: E731
    want = call(k, v).clone()
    for bad in (float("nan"), float("inf")):
        k2, v2 = k.clone(), v.clone()
        k2[n:], v2[n:] = bad, bad
        assert torch.equal(call(k2, v2), want)
        for at in (0, 50, 99):                       # a key that the query `at` and later ones see
            k2, v2 = k.clone(), v.clone()
            k2[n - m + at, 0, 3], v2[n - m + at, 1, 7] = bad, bad
            got = call(k2, v2)
            assert torch.equal(got[:at], want[:at])
            later = got[at:].float()
            assert not torch.isfinite(later[:, 4:, 7]).any()
            later[:, :4], later[:, 4:, 7] = 0, 0
            assert torch.isfinite(later).all()
        v2 = v.clone()
        v2[700, 1, 7] = bad                          # a value in a part that everybody sees whole
        got = call(k, v2).float()
        assert not torch.isfinite(got[:, 4:, 7]).any()
        got[:, 4:, 7] = 0
        assert torch.isfinite(got).all()


def test_repeats_bit_for_bit_in_graphs_on_two_streams():
    sets = [(normal((40, 32, 128), s), normal((5000, 8, 128), s + 1), normal((5000, 8, 128), s + 2)) for s in (1, 5)]
    qs, ks = i32([0, 25, 40]), i32([0, 4000, 5000])
    want = [kv.kv_attention_prompt(*x, qs, ks).clone() for x in sets]
    calls = [kv.kv_attention_prompt(*x, qs, ks, prepare=True) for x in sets]
    graphs = []
    torch.cuda.synchronize()
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c()
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for s, g, c in zip(streams, graphs, calls):
            with torch.cuda.stream(s):
                c.result.zero_()
                g.replay()
        torch.cuda.synchronize()
        for c, w in zip(calls, want):
            assert torch.equal(c.result, w)


def test_sequences_that_are_refused():
    q, k, v = normal((50, 4, 64), 1), normal((3000, 1, 64), 2), normal((3000, 1, 64), 3)
    good = kv.kv_attention_prompt(q, k, v, i32([0, 20, 50]), i32([0, 1500, 3000]))
    for qs, ks in (([0, 20, 51], [0, 1500, 3000]), ([0, 20, 50], [0, 1500, 3001]), ([0, 20, 50], [0, 1500, 15])):
        out = torch.full((50, 4, 64), 7.0, dtype=BF16, device=dev())
        err = kv.new_error_word(dev())
        kv.kv_attention_prompt(q, k, v, i32(qs), i32(ks), out=out, err=err)
        assert err.item() == kv.ERR_BITS["BAD_QSL"]
        assert torch.equal(out[:20], good[:20]) and (out[20:] == 7).all()
    assert np.isfinite(good.float().cpu().numpy()).all()


def test_rows_past_two_billion_elements():
    """Key rows and query rows whose elements are counted past 2^31."""
    free, _ = torch.cuda.mem_get_info()
    if free < 24 << 30:
        pytest.skip("needs 20 GB")
    m, n, h, d = 30, 1000, 8, 128
    far = 2 ** 31 // (h * d) + 5
    kv_rows = torch.empty((far + n, h, d), dtype=BF16, device=dev())
    kv_rows[far:] = normal((n, h, d), 1)
    q = normal((m, 2 * h, d), 2)
    got = kv.kv_attention_prompt(q, kv_rows, kv_rows, i32([0, m]), i32([far, far + n]))
    o, b = expect(q, kv_rows[far:], kv_rows[far:], starts([m]), starts([n]), d ** -0.5)
    ref.check(got, o, b)
    far = 2 ** 31 // (2 * h * d) + 3
    rows = torch.empty((far + m, 2 * h, d), dtype=BF16, device=dev())
    rows[far:] = q
    out = torch.empty_like(rows)
    kv.kv_attention_prompt(rows, kv_rows[-n:], kv_rows[-n:], i32([far, far + m]), i32([0, n]), out=out)
    ref.check(out[far:], o, b)


def test_the_longest_request_and_one_that_is_longer():
    n = 2 ** 24
    q = normal((5, 1, 8), 1)
    k = torch.zeros((n + 1, 1, 8), dtype=BF16, device=dev())
    v = torch.ones_like(k)
    err = kv.new_error_word(dev())
    got = kv.kv_attention_prompt(q, k, v, i32([0, 5]), i32([0, n]), err=err)
    assert (got == 1).all() and err.item() == 0   # sums of ones: exact in 32 bits up to 2^24
    out = torch.full_like(q, 7.0)
    kv.kv_attention_prompt(q, k, v, i32([0, 5]), i32([0, n + 1]), out=out, err=err)
    assert (out == 7).all() and err.item() == kv.ERR_BITS["BAD_QSL"]
