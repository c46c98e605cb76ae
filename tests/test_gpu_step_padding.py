"""A step's calls over a padded batch: requests without rows, whose other entries mean nothing."""
import pytest
import torch

import paged_kv_cache_39_gb300 as kv
from operator_refs import BF16, dev, normal
from step_refs import i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ctx", [-1, -2 ** 31, 2 ** 31 - 1])
@pytest.mark.parametrize("kept", [-1, 0, 64])
def test_requests_without_rows_change_and_report_nothing(ctx, kept):
    """The same outputs as without them, no error, and rows behind the last request as they were."""
    T, h, D, V, n = 16, 2, 64, 50, 5
    kc, vc = normal((2, 9, T, h, D), 1), normal((2, 9, T, h, D), 2)
    q, p = normal((n + 3, 8, D), 3), torch.softmax(torch.randn((n + 3, V), device=dev()), 1)
    parents, tokens, u = i32([-1, 0, 0, -1, 0, 9, 9, 9]), i32([1, 2, 3, 4, 5, -7, -7, -7]), torch.zeros(n + 3, device=dev())
    want = pad = None
    for padded in (False, True):
        starts, context = ([0, 0, 3, 3, 5, 5, 5], [ctx, 20, ctx, 33, ctx, ctx]) if padded else ([0, 3, 5], [20, 33])
        rows = [r for r in range(len(context)) if starts[r + 1] > starts[r]]
        table = torch.full((len(context), 3), -9, dtype=torch.int32, device=dev())
        table[rows] = i32([[1, 2, 3], [4, 5, 6]])
        qs, cl, err = i32(starts), i32(context), kv.new_error_word(dev())
        outs = [torch.full((n + 3,), -5, dtype=torch.int64, device=dev()) for _ in range(3)]
        kv.kv_tree_layout(parents, qs, cl, n + 3, *outs, err=err)
        out = torch.full((n + 3, 8, D), 7.0, dtype=BF16, device=dev())
        kv.kv_attention_tree(q, kc, vc, table, qs, cl, max_rows=3, tree_mask=outs[0], out=out, err=err)
        new = [torch.full((n + 3,), -5, dtype=torch.int32, device=dev()) for _ in range(2)]
        _, _, num = kv.kv_verify_drafts(p, tokens, qs, u, None, parents, *new, err=err)
        assert num.tolist() == ([0, 1, 0, 1, 0, 0] if padded else [1, 1])
        pad = torch.ones(len(context), dtype=torch.bool, device=dev())
        pad[rows] = False
        num[pad] = kept
        k2, v2 = kc.clone(), vc.clone()
        kv.kv_cache_keep_path(k2, v2, table, qs, cl, new[1], num, err=err)
        assert err.item() == 0
        got = (*outs, out, *new, k2, v2)
        assert all((x[n:] == (7 if x is out else -5)).all() for x in got[:6])
        want = want or got
        assert all(torch.equal(a, b) for a, b in zip(got, want))
