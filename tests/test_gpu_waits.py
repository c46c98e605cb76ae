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
