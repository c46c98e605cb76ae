"""Host-visible refusals of the waits' self-tests: none of these calls reaches the GPU."""
import pytest

from test_operators_abi import A, N, lib  # noqa: F401


@pytest.mark.parametrize("limit,waited,err", [
    (-1, A[0], A[1]), (10 ** 9 + 1, A[0], A[1]), (1, N, A[1]), (1, A[0] + 4, A[1]), (1, A[0], N),
    (1, A[0], A[1] + 2),
])
def test_role_wait_refuses(lib, limit, waited, err):  # noqa: F811
    assert lib.kv_diag_role_wait(limit, waited, err, N) == -1
