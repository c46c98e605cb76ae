"""kv_attention_prompt with far more tile pairs than SMs, so that a CTA goes from one sequence's
pair to another's: against the formula in 64 bits."""
import numpy as np
import pytest
import torch

import paged_kv_cache_39_gb300 as kv
from operator_refs import BF16, dev, normal
from test_gpu_attention_prompt import run, starts
from test_gpu_cache_q4 import i32

pytestmark = pytest.mark.gpu


def lengths(count, seed, new_max, prior_max):
    rng = np.random.default_rng(seed)
    new = rng.integers(0, new_max, count)
    total = new + rng.integers(0, prior_max, count) * (rng.random(count) < 0.7)
    total[rng.random(count) < 0.05] //= 2          # some queries see no key
    total[rng.random(count) < 0.03] = 0
    return [int(x) for x in new], [int(x) for x in total]


@pytest.mark.parametrize("hq,h,d", [(16, 8, 128), (8, 8, 64), (24, 4, 80), (35, 5, 128)])
@pytest.mark.parametrize("count,new_max,prior_max", [(90, 400, 700), (400, 130, 300), (120, 3, 1500)])
def test_many_sequences(count, new_max, prior_max, hq, h, d):
    new, total = lengths(count, count + d, new_max, prior_max)
    run(new, total, hq, h, d, seed=count, tail=2)


def test_pairs_of_one_and_two_tiles_take_turns():
    new = [32, 33, 1, 64, 0, 65, 128, 31] * 20
    total = [32, 160, 129, 64, 50, 193, 128, 400] * 20
    run(new, total, 16, 4, 128, seed=1)
    run(new, total, 16, 4, 64, seed=2)


def test_a_long_prompt_beside_short_ones():
    run([2100] + [50] * 300, [2500] + [50] * 300, 8, 8, 64, seed=3)


def test_a_bad_value_stays_in_its_sequence():
    """NaN and infinity in a value of every third sequence: its later queries' channel and no
    other sequence, whichever CTA takes them after one another."""
    rng = np.random.default_rng(7)
    count = 300
    new = rng.integers(1, 90, count)
    total = new + rng.integers(0, 200, count)
    qs, ks = starts(new), starts(total)
    q, k, v = normal((int(qs[-1]), 16, 128), 1), normal((int(ks[-1]), 8, 128), 2), normal((int(ks[-1]), 8, 128), 3)
    want = kv.kv_attention_prompt(q, k, v, i32(qs), i32(ks)).clone()
    for bad in (float("nan"), float("inf")):
        v2, first = v.clone(), np.full(count, -1)
        for r in range(0, count, 3):
            first[r] = rng.integers(0, new[r])     # the first query that sees the key
            v2[ks[r + 1] - new[r] + first[r], 5, 77] = bad
        got = kv.kv_attention_prompt(q, k, v2, i32(qs), i32(ks))
        hit = torch.zeros(int(qs[-1]), dtype=torch.bool, device=dev())
        for r in range(0, count, 3):
            hit[qs[r] + first[r]:qs[r + 1]] = True
        assert torch.equal(got[~hit], want[~hit])
        assert not torch.isfinite(got[hit][:, 10:12, 77].float()).any()
        rest = got[hit].clone()
        rest[:, 10:12, 77] = want[hit][:, 10:12, 77]
        assert torch.equal(rest, want[hit])


def test_repeats_bit_for_bit_on_two_streams():
    new, total = lengths(250, 9, 200, 300)
    qs, ks = starts(new), starts(total)
    sets = [(normal((int(qs[-1]), 16, 128), s), normal((int(ks[-1]), 8, 128), s + 1),
             normal((int(ks[-1]), 8, 128), s + 2)) for s in (1, 5)]
    tq, tk = i32(qs), i32(ks)
    want = [kv.kv_attention_prompt(*x, tq, tk).clone() for x in sets]
    out = [torch.empty_like(w) for w in want]
    calls = [kv.kv_attention_prompt(*x, tq, tk, out=o, prepare=True) for x, o in zip(sets, out)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        calls[0]()
        calls[0]()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        with torch.cuda.stream(streams[0]):
            out[0].zero_()
            graph.replay()
        with torch.cuda.stream(streams[1]):
            out[1].zero_()
            calls[1]()
            calls[1]()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    assert want[0].dtype == BF16
