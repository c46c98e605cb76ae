"""kv_attention_prompt against its formula in 64 bits."""
import numpy as np
import pytest
import torch

import operator_refs as ref
import paged_kv_cache_39_gb300 as kv
from operator_refs import BF16, dev, normal
from test_gpu_cache_q4 import i32

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -8   # the weights are rounded to bf16


def starts(lengths):
    return np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)


def expect(q, k, v, qs, ks, scale):
    o = torch.zeros(q.shape, dtype=ref.F64, device=dev())
    b = torch.zeros_like(o)
    for r in range(len(qs) - 1):
        m, n = qs[r + 1] - qs[r], ks[r + 1] - ks[r]
        for a in range(0, m, 512):
            e = min(m, a + 512)
            seen = np.clip(np.arange(a, e) + n - m + 1, 0, n)
            o[qs[r] + a:qs[r] + e], b[qs[r] + a:qs[r] + e] = ref.attend(
                q[qs[r] + a:qs[r] + e], k[ks[r]:ks[r + 1]].to(ref.F64), v[ks[r]:ks[r + 1]].to(ref.F64),
                seen, scale, STEP)
    return o, b


def run(new, total, hq, h, d, seed=0, scale=None, q_scale=1.0, tail=0):
    qs, ks = starts(new), starts(total)
    n, nk = int(qs[-1]) + tail, int(ks[-1]) + tail
    qkv = normal((n, hq + 1, d), seed, q_scale)
    q = qkv[:, :hq]
    kvr = normal((nk, 2 * h, d), seed + 1)
    k, v = kvr[:, :h], kvr[:, h:]
    err = kv.new_error_word(dev())
    out = torch.full((n, hq, d), 7.0, dtype=BF16, device=dev())
    got = kv.kv_attention_prompt(q, k, v, i32(qs), i32(ks), scale=scale, out=out, err=err)
    o, b = expect(q, k, v, qs, ks, d ** -0.5 if scale is None else scale)
    m = int(qs[-1])
    ref.check(got[:m], o[:m], b[:m], f"{new} {total} hq={hq} h={h} d={d}")
    assert (got[m:] == 7).all()            # rows behind the last sequence
    assert err.item() == 0
    return got


@pytest.mark.parametrize("d", [8, 64, 72, 80, 128])
@pytest.mark.parametrize("hq,h", [(1, 1), (4, 4), (8, 2), (6, 2), (5, 1), (14, 2), (128, 1)])
def test_head_groups_and_dims(hq, h, d):
    run([1, 7, 130], [1, 7, 130], hq, h, d, seed=hq + d, tail=3)


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 511, 513, 1000])
def test_lengths_around_the_tiles(n):
    run([n], [n], 4, 1, 128, seed=n)
    run([n], [n], 2, 2, 64, seed=n + 1)


@pytest.mark.parametrize("new,total", [
    ([1], [1000]), ([5, 1, 200], [5, 300, 777]), ([128], [256]), ([100, 100], [101, 1500]),
    ([1] * 40, list(range(1, 41))), ([64, 3], [64 + 127, 3 + 128]),
])
def test_chunks_behind_earlier_tokens(new, total):
    run(new, total, 8, 2, 128, seed=len(new), tail=5)


def test_empty_sequences_and_queries_that_see_no_key():
    run([0, 3, 0, 0, 10, 0], [0, 3, 5, 0, 12, 0], 8, 2, 128)
    got = run([10, 300, 4], [4, 100, 0], 8, 2, 128, seed=1)
    assert not got[:6].any() and not got[10:210].any() and not got[310:].any()


def test_a_long_prompt_and_many_short_ones():
    run([3000], [3000], 4, 1, 128, seed=3)
    rng = np.random.default_rng(4)
    n = list(rng.integers(0, 60, 150))
    run(n, n, 8, 2, 64, seed=4)


def test_exactly_the_tensor_rows():
    """No row behind the last sequence, key rows that end at the buffer's end."""
    run([77, 50], [77, 60], 32, 8, 128, seed=9, tail=0)


@pytest.mark.parametrize("scale,q_scale", [(1.0, 1.0), (None, 20.0), (1e-4, 1.0), (None, 1e-3)])
def test_scales(scale, q_scale):
    run([200], [300], 4, 2, 128, seed=6, scale=scale, q_scale=q_scale)


def test_logits_that_grow_along_the_keys():
    """The running maximum rises at every tile: each tile's weights outgrow the earlier ones'."""
    n, d = 700, 128
    q = torch.ones((n, 2, d), device=dev()).to(BF16)
    k = (torch.arange(n, device=dev())[:, None, None] * 0.02 * torch.ones((n, 1, d), device=dev())).to(BF16)
    v = normal((n, 1, d), 3)
    qs = starts([n])
    got = kv.kv_attention_prompt(q, k, v, i32(qs))
    o, b = expect(q, k, v, qs, qs, d ** -0.5)
    ref.check(got, o, b)


def test_keys_out_of_sight_may_hold_anything():
    """NaN and infinity in key and value rows of other sequences, behind the last one, and
    in keys that only later queries see."""
    new, total = [60, 100, 33], [60, 300, 33]
    qs, ks = starts(new), starts(total)
    n, nk = int(qs[-1]), int(ks[-1]) + 100
    q, k, v = normal((n, 8, 128), 1), normal((nk, 2, 128), 2), normal((nk, 2, 128), 3)
    want = kv.kv_attention_prompt(q, k, v, i32(qs), i32(ks)).clone()
    for bad in (float("nan"), float("inf"), -float("inf")):
        k2, v2 = k.clone(), v.clone()
        k2[ks[3]:], v2[ks[3]:] = bad, bad            # behind the last sequence
        k2[ks[0]:ks[1]], v2[ks[0]:ks[1]] = bad, bad  # the first sequence's own rows
        got = kv.kv_attention_prompt(q, k2, v2, i32(qs), i32(ks))
        assert torch.equal(got[qs[1]:], want[qs[1]:])
        for at in (0, 5, 50, 99):                    # one key of sequence 1, counted from the first query's
            k2, v2 = k.clone(), v.clone()
            row = ks[1] + 200 + at
            k2[row, 0, 3], v2[row, 1, 7] = bad, bad
            got = kv.kv_attention_prompt(q, k2, v2, i32(qs), i32(ks))
            before = qs[1] + at
            assert torch.equal(got[:before], want[:before]) and torch.equal(got[qs[2]:], want[qs[2]:])
            later = got[before:qs[2]].float()
            assert not torch.isfinite(later[:, 4:, 7]).any()
            later[:, :4], later[:, 4:, 7] = 0, 0
            assert torch.isfinite(later).all()


def test_logits_of_minus_infinity_before_finite_ones():
    """Keys whose logits are -inf for a whole tile, then ordinary ones far below 0."""
    n, d = 300, 64
    q = torch.ones((n, 1, d), device=dev()).to(BF16)
    k = torch.full((n, 1, d), -40.0, device=dev()).to(BF16)
    k[:160, 0, 5] = -float("inf")
    v = normal((n, 1, d), 3)
    got = kv.kv_attention_prompt(q, k, v, i32([0, n]))
    for i in (160, 200, 299):   # equal logits: the mean of the values behind the infinite ones
        want = v[160:i + 1].to(ref.F64).mean(0)
        size = v[160:i + 1].to(ref.F64).abs().mean(0)
        # equal weights are exactly 1: the sum's roundings (2^-24 each) and the output's
        ref.check(got[i], want, want.abs() * 2.0 ** -8 + size * n * 2.0 ** -23)


def test_no_key_at_all():
    q, none = normal((70, 8, 128), 1), torch.empty((0, 2, 128), dtype=BF16, device=dev())
    out = torch.full_like(q, 7.0)
    err = kv.new_error_word(dev())
    kv.kv_attention_prompt(q, none, none, i32([0, 60, 65]), i32([0, 0, 0]), out=out, err=err)
    assert not out[:65].any() and (out[65:] == 7).all() and err.item() == 0
    assert kv.kv_attention_prompt(none[:, :2], none, none, i32([0])).shape == (0, 2, 128)


def test_more_requests_than_a_block_ranks():
    """Up to 384 requests are ordered by their keys, more are taken as they come."""
    rng = np.random.default_rng(11)
    for count in (383, 384, 385, 1200):
        new = rng.integers(0, 4, count)
        total = new + rng.integers(0, 40, count)
        run(list(new), list(total), 4, 2, 64, seed=count)


def test_sequences_that_are_refused():
    q, k, v = normal((50, 4, 64), 1), normal((50, 1, 64), 2), normal((50, 1, 64), 3)
    good = kv.kv_attention_prompt(q, k, v, i32([0, 20, 50]))
    for qs, ks, keep in (([0, 20, 51], [0, 20, 50], 20), ([0, 20, 50], [0, 20, 51], 20),
                         ([0, 20, 10], [0, 20, 50], 20), ([0, 20, 50], [0, 20, 15], 20),
                         ([-3, 20, 50], [0, 20, 50], None)):
        out = torch.full((50, 4, 64), 7.0, dtype=BF16, device=dev())
        err = kv.new_error_word(dev())
        kv.kv_attention_prompt(q, k, v, i32(qs), i32(ks), out=out, err=err)
        assert err.item() == kv.ERR_BITS["BAD_QSL"]
        if keep is not None:
            assert torch.equal(out[:keep], good[:keep]) and (out[keep:] == 7).all()
        else:
            assert (out[:20] == 7).all() and torch.equal(out[20:], good[20:])


def test_repeats_bit_for_bit_in_a_graph_and_on_two_streams():
    new = [300, 40, 129]
    qs = i32(starts(new))
    sets = [(normal((469, 32, 128), s), normal((469, 8, 128), s + 1), normal((469, 8, 128), s + 2)) for s in (1, 5)]
    want = [kv.kv_attention_prompt(*x, qs).clone() for x in sets]
    calls = [kv.kv_attention_prompt(*x, qs, prepare=True) for x in sets]
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


def test_binding_refusals():
    q, k = normal((8, 4, 64), 1), normal((9, 2, 64), 2)
    with pytest.raises(ValueError, match="k_start_loc"):
        kv.kv_attention_prompt(q, k, k, i32([0, 8]))
    with pytest.raises(ValueError, match="differ"):
        kv.kv_attention_prompt(q, k, k[:, :1], i32([0, 8]), i32([0, 9]))
    with pytest.raises(ValueError, match="out must be"):
        kv.kv_attention_prompt(q, k, k, i32([0, 8]), i32([0, 9]), out=q[:4])
    with pytest.raises(kv.KVError):
        kv.kv_attention_prompt(q[:, :3], k, k, i32([0, 8]), i32([0, 9]))
    with pytest.raises(kv.KVError):
        kv.kv_attention_prompt(q, k, k, i32([0, 8]), i32([0, 9]), out=q)
