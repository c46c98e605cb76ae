"""Both attentions at the ends of what a positive, finite scale can be."""
import numpy as np
import pytest
import torch

import operator_refs as ref
import paged_kv_cache_39_gb300 as kv
from operator_refs import BF16, dev, normal
from test_gpu_attention_q4 import layout
from test_gpu_cache_q4 import i32, random_cache

pytestmark = pytest.mark.gpu
SCALES = [3.4e38, 2.0 ** 110, 1e-25, 2e-38, 1e-45]


def mean_check(got, v, what):
    """Equal weights: under 2^-11 of each weight, 32-bit sums, and the output's rounding."""
    want, size = v.to(ref.F64).mean(0), v.to(ref.F64).abs().mean(0)
    ref.check(got, want, want.abs() * 2.0 ** -8 + size * (2.0 ** -11 + len(v) * 2.0 ** -23), what)


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("hq,h,D", [(4, 1, 128), (8, 1, 64), (16, 1, 64)])
def test_attention_q4(scale, hq, h, D):
    """Logits of zero, or far below one: the mean of the values, in spans that end inside a unit."""
    n, T = 77, 16
    table, B = layout([n], T, 1)
    kc, vc = random_cache(1, B, T, h, D, 1), random_cache(1, B, T, h, D, 2)
    p = np.arange(3, n)
    v = ref.values(vc, T, D, 0, table[0, p // T].astype(np.int64) * T + p % T)[:, 0]
    tiny = normal((1, hq, D), 3).float() * 2.0 ** -95
    for q in [torch.zeros((1, hq, D), device=dev())] + ([tiny] if scale < 1 else []):
        got = kv.kv_attention_q4(q.to(BF16), kc, vc, i32(table), i32([3]), i32([n]), T, scale=scale)
        for head in range(hq):
            mean_check(got[0, head], v, f"scale {scale} head {head}")


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("m,n", [(5, 77), (5, 3000)])
def test_attention_prompt(scale, m, n):
    k, v = normal((n, 1, 128), 1), normal((n, 1, 128), 2)
    tiny = normal((m, 4, 128), 3).float() * 2.0 ** -95
    for q in [torch.zeros((m, 4, 128), device=dev())] + ([tiny] if scale < 1 else []):
        got = kv.kv_attention_prompt(q.to(BF16), k, v, i32([0, m]), i32([0, n]), scale=scale)
        for i in range(m):
            mean_check(got[i], v[:n - m + i + 1].expand(-1, 4, -1), f"scale {scale} row {i}")


@pytest.mark.parametrize("m,n", [(5, 77), (5, 3000), (300, 300)])
def test_prompt_rows_whose_logits_are_all_minus_infinity(m, n):
    """They get zeros, as rows that see no key; a finite logit makes an ordinary row."""
    q = torch.ones((m, 4, 64), dtype=BF16, device=dev())
    k, v = normal((n, 1, 64), 1), normal((n, 1, 64), 2)
    k[:, 0, 7] = -float("inf")
    assert not kv.kv_attention_prompt(q, k, v, i32([0, m]), i32([0, n])).any()
    at = n - m + 3
    k[at, 0, 7] = 0
    got = kv.kv_attention_prompt(q, k, v, i32([0, m]), i32([0, n]))
    assert not got[:3].any() and torch.equal(got[3:], v[at].expand_as(got[3:]))
