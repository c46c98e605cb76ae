"""Host-visible refusals of the waits' self-tests: none of these calls reaches the GPU."""
import pytest

from test_operators_abi import A, N, PROMPT, lib  # noqa: F401


@pytest.mark.parametrize("limit,waited,err", [
    (-1, A[0], A[1]), (10 ** 9 + 1, A[0], A[1]), (1, N, A[1]), (1, A[0] + 4, A[1]), (1, A[0], N),
    (1, A[0], A[1] + 2),
])
def test_role_wait_refuses(lib, limit, waited, err):  # noqa: F811
    assert lib.kv_diag_role_wait(limit, waited, err, N) == -1


@pytest.mark.parametrize("want,change", [
    (-1, dict(role=-1)), (-1, dict(role=5)), (-1, dict(item=-1)), (-1, dict(limit=-1)),
    (-1, dict(limit=10 ** 9 + 1)), (-1, dict(err=N)), (-1, dict(scale=0.0)), (-2, dict(reqs=4097)),
    (-1, dict(query=N)), (0, dict(reqs=0)),
])
def test_prompt_stall_refuses(lib, want, change):  # noqa: F811
    args = {**PROMPT, "err": A[6]}
    args.pop("stream")
    args = {**args, "role": 0, "item": 0, "limit": 1000, "stream": N, **change}
    assert lib.kv_diag_attention_prompt_stall(*args.values()) == want
