"""Outputs that share bytes with an input are refused on the host; neighbours are not."""
import pytest

from test_operators_abi import A, ATTEND4, N, PROMPT, ROPE, lib  # noqa: F401

ROW = 32 * 128 * 2     # bytes of a query row


@pytest.mark.parametrize("out", ["q_out", "k_out"])
@pytest.mark.parametrize("name,size", [("qw", 256), ("kw", 256), ("positions", 32), ("cos_sin", 100 * 512),
                                       ("slots", 32)])
def test_norm_rope_refuses_shared_bytes(lib, out, name, size):  # noqa: F811
    call = lambda **x: lib.kv_qk_norm_rope_write(*{**ROPE, **x}.values())  # noqa: E731
    rows = 4 * (ROW if out == "q_out" else ROW // 4)
    assert call(**{out: ROPE[name]}) == -1
    assert call(**{out: ROPE[name] + size - 16}) == -1
    assert call(**{out: ROPE[name] - rows + 16}) == -1


@pytest.mark.parametrize("name", ["q_start", "k_start"])
def test_prompt_attention_refuses_shared_bytes(lib, name):  # noqa: F811
    for at in (0, -8 * ROW + 16):
        assert lib.kv_attention_prompt(*{**PROMPT, "out": PROMPT[name] + at}.values()) == -1


@pytest.mark.parametrize("name,size", [("kc", 8 * 8 * 16 * 72), ("vc", 8 * 8 * 16 * 72), ("table", 32),
                                       ("s0", 8), ("s1", 8), ("ws", 1 << 20)])
def test_attention_q4_refuses_shared_bytes(lib, name, size):  # noqa: F811
    for at in (0, -2 * ROW + 16, size - size % 16 - 16 if size > 16 else 0):
        assert lib.kv_attention_q4(*{**ATTEND4, "out": ATTEND4[name] + at}.values()) == -1
        if name != "ws":
            assert lib.kv_attention_q4(*{**ATTEND4, "ws": ATTEND4[name] + at}.values()) == -1
    assert lib.kv_attention_q4(*{**ATTEND4, "ws": ATTEND4["query"] + 64}.values()) == -1
