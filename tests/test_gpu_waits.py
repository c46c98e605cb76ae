"""Waits that nothing will satisfy: they end within their limit and the GPU works on."""
import pytest
import torch

import paged_kv_cache_39_gb300 as kv
from operator_refs import dev, normal
from test_gpu_cache_q4 import i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("limit_ms", [0, 1, 20])
def test_the_roles_wait_ends_by_its_timer(limit_ms):
    """The warp with the short limit ends a little after it, the others (limit 1 s) with it."""
    q, k, v = normal((100, 8, 128), 1), normal((100, 2, 128), 2), normal((100, 2, 128), 3)
    want = kv.kv_attention_prompt(q, k, v, i32([0, 100])).clone()
    err, waited = kv.new_error_word(dev()), torch.zeros(4, dtype=torch.int64, device=dev())
    stream = torch.cuda.current_stream().cuda_stream
    assert kv.load().kv_diag_role_wait(limit_ms * 1000000, waited.data_ptr(), err.data_ptr(), stream) == 0
    got = kv.kv_attention_prompt(q, k, v, i32([0, 100]))
    torch.cuda.synchronize()
    assert err.item() == kv.ERR_BITS["TIMEOUT"]
    waited = waited.tolist()
    assert waited[3] >= limit_ms * 1000000
    # five tries' own suspensions lie beside the limit: half of the 1 s bound is far above them
    assert max(waited) < limit_ms * 1000000 + 500000000
    assert torch.equal(got, want)


def _prompt(mode):
    """Sequences (new, total) whose tile pairs run in one wave, in many, or shared by clusters."""
    return {"one": ([300, 20], [300, 150]), "many": ([600] * 40, [600] * 40),
            "clusters": ([16, 3], [5000, 900])}[mode]


@pytest.mark.parametrize("limit_ns", [0, 1000000])
@pytest.mark.parametrize("role", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("mode,item", [("one", 0), ("many", 0), ("many", 1), ("many", 2), ("clusters", 0)])
def test_a_role_that_gives_up_ends_the_call(mode, item, role, limit_ns):
    """One role of every CTA waits for nothing and gives up: the call ends, says so, and the next
    ones are right."""
    new, total = _prompt(mode)
    qs, ks = i32([0] + list(torch.tensor(new).cumsum(0))), i32([0] + list(torch.tensor(total).cumsum(0)))
    m, n, hq, h, d = sum(new), sum(total), 32, 8, 128
    q, k, v = normal((m, hq, d), 1), normal((n, h, d), 2), normal((n, h, d), 3)
    want = kv.kv_attention_prompt(q, k, v, qs, ks).clone()
    err, out = kv.new_error_word(dev()), torch.zeros_like(q)
    args = (q.data_ptr(), hq * d, k.data_ptr(), h * d, v.data_ptr(), h * d, qs.data_ptr(), ks.data_ptr(),
            len(new), m, n, hq, h, d, d ** -0.5, out.data_ptr(), err.data_ptr())
    stream = torch.cuda.current_stream().cuda_stream
    for _ in range(3):
        err.zero_()
        assert kv.load().kv_diag_attention_prompt_stall(*args, role, item, limit_ns, stream) == 0
        after = kv.kv_attention_prompt(q, k, v, qs, ks)
        torch.cuda.synchronize()
        assert err.item() == kv.ERR_BITS["TIMEOUT"]
        assert torch.equal(after, want)
    # a work number that no CTA reaches: an ordinary call
    err.zero_()
    assert kv.load().kv_diag_attention_prompt_stall(*args, role, 1000, limit_ns, stream) == 0
    torch.cuda.synchronize()
    assert err.item() == 0 and torch.equal(out, want)
