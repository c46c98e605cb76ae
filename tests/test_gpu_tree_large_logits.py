"""kv_attention_tree with logits of up to 2^30, where a step of 32 bits is 64: only the likeliest keys count."""
import numpy as np
import pytest
import torch

import operator_refs as ref
import paged_kv_cache_39_gb300 as kv
from operator_refs import BF16, F64, dev, normal
from step_refs import block_table, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [2.0 ** 8, 2.0 ** 16, 2.0 ** 20, 2.0 ** 22])
@pytest.mark.parametrize("low", [1, -255])             # logits above zero, logits below
@pytest.mark.parametrize("order", ["rising", "falling", "any"])
@pytest.mark.parametrize("rows,group,ctx,T", [(3, 4, 700, 16), (3, 4, 700, 20), (40, 5, 700, 16), (2, 2, 20000, 16)])
def test_the_likeliest_keys(rows, group, ctx, T, order, low, scale):
    """Logits are scale times a whole number of the key: weights are 1 for the largest and, below it, 2^-369
    and less.  What counts has equal logits, so equal weights: each is rounded to bf16 for its product
    with V and the sum takes it before that (2^-8), then the output's rounding; sums of n in 32 bits."""
    h, D, n = 2, 64, ctx + rows
    rng = np.random.default_rng(rows + ctx + low)
    table, B = block_table([n], T, rng)
    whole = rng.integers(low, low + 255, n)
    if order != "any":
        whole = np.sort(whole)[::1 if order == "rising" else -1]
    at = torch.from_numpy(table[0, np.arange(n) // T].astype(np.int64) * T + np.arange(n) % T).to(dev())
    kc, vc = torch.zeros((1, B, T, h, D), dtype=BF16, device=dev()), normal((1, B, T, h, D), 1)
    w = torch.from_numpy(whole.copy()).to(dev())
    kc[0].flatten(0, 1)[at, :, 5] = w[:, None].to(BF16)
    q = torch.zeros((rows, h * group, D), dtype=BF16, device=dev())
    q[..., 5] = 1
    got = kv.kv_attention_tree(q, kc, vc, i32(table), i32([0, rows]), i32([ctx]), max_rows=rows, scale=scale)
    v = vc[0].flatten(0, 1)[at].to(F64)
    for i in range(rows):
        seen = w[:ctx + i + 1]
        some = v[:ctx + i + 1][seen == seen.max()]
        want, size = some.mean(0).repeat_interleave(group, 0), some.abs().mean(0).repeat_interleave(group, 0)
        ref.check(got[i], want, want.abs() * 2.0 ** -8 + size * (2.0 ** -8 + n * 2.0 ** -22), f"row {i}")
