"""Host-visible refusals of the operators around the cache: none of these calls
reaches the GPU (pointers are plain numbers the library must not follow)."""
import os

import pytest

N = None
A = [0x10000000 * (i + 1) for i in range(16)]  # 16-byte aligned, far apart


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_39_gb300 import _lib
    from paged_kv_cache_39_gb300 import build as kbuild
    if not os.path.exists(_lib.LIB_PATH):
        kbuild.build()
    return _lib.load()


ROPE = dict(query=A[0], qs=32 * 128, key=A[1], ks=8 * 128, value=A[2], vs=8 * 128, qw=A[3], kw=A[4],
            positions=A[5], cos_sin=A[6], max_position=100, rotary=128, inter=0, eps=1e-6, n=4, hq=32,
            h=8, d=128, q_out=A[7], k_out=A[8], kc=A[9], vc=A[10], layer=0, layers=1, blocks=8, t=16,
            slots=A[11], err=N, stream=N)


@pytest.mark.parametrize("want,change", [
    (-1, dict(n=-1)), (-1, dict(hq=0)), (-1, dict(h=0)), (-1, dict(d=0)), (-1, dict(rotary=0)),
    (-1, dict(rotary=136)), (-1, dict(eps=-1.0)), (-1, dict(eps=float("nan"))),
    (-1, dict(layer=1)), (-1, dict(layer=-1)), (-1, dict(blocks=0)), (-1, dict(t=0)),
    (-2, dict(rotary=12)), (-2, dict(d=260, qs=32 * 260, ks=8 * 260, vs=8 * 260)),
    (-2, dict(d=12, qs=512, ks=128, vs=128, rotary=8)),
    (-1, dict(qs=32 * 128 - 8)), (-1, dict(ks=8)), (-1, dict(vs=8)),
    (-2, dict(qs=32 * 128 + 4)), (-2, dict(ks=8 * 128 + 1)), (-2, dict(vs=8 * 128 + 2)),
    (-1, dict(query=N)), (-1, dict(key=N)), (-1, dict(value=N)), (-1, dict(qw=N)), (-1, dict(kw=N)),
    (-1, dict(positions=N)), (-1, dict(cos_sin=N)), (-1, dict(q_out=N)), (-1, dict(slots=N)),
    (-1, dict(kc=N)), (-1, dict(vc=N)), (-1, dict(kc=N, vc=N, k_out=N)),
    (-1, dict(query=A[0] + 8)), (-1, dict(key=A[1] + 2)), (-1, dict(value=A[2] + 8)),
    (-1, dict(qw=A[3] + 4)), (-1, dict(positions=A[5] + 4)), (-1, dict(cos_sin=A[6] + 4)),
    (-1, dict(q_out=A[7] + 8)), (-1, dict(k_out=A[8] + 8)), (-1, dict(kc=A[9] + 8)),
    (-1, dict(slots=A[11] + 4)), (-1, dict(err=A[12] + 2)),
    (-1, dict(q_out=A[0] + 16)),                       # overlaps query, not the same rows
    (-1, dict(q_out=A[0], qs=48 * 128)),               # in place over rows that are not dense
    (-1, dict(q_out=A[1])), (-1, dict(k_out=A[0])), (-1, dict(k_out=A[2])), (-1, dict(k_out=A[7])),
    (0, dict(n=0)),
])
def test_norm_rope_refuses(lib, want, change):
    assert lib.kv_qk_norm_rope_write(*{**ROPE, **change}.values()) == want


PROMPT = dict(query=A[0], qs=32 * 128, key=A[1], ks=8 * 128, value=A[2], vs=8 * 128, q_start=A[3],
              k_start=A[4], reqs=2, nq=8, nk=16, hq=32, h=8, d=128, scale=0.1, out=A[5], err=N, stream=N)


@pytest.mark.parametrize("want,change", [
    (-1, dict(reqs=-1)), (-1, dict(nq=-1)), (-1, dict(nk=-1)), (-1, dict(hq=0)), (-1, dict(h=0)),
    (-1, dict(d=0)), (-1, dict(hq=30)), (-1, dict(scale=0.0)), (-1, dict(scale=-1.0)),
    (-1, dict(scale=float("inf"))), (-1, dict(scale=float("nan"))),
    (-2, dict(d=132, qs=32 * 136, ks=8 * 136, vs=8 * 136)),
    (-2, dict(d=136, qs=32 * 136, ks=8 * 136, vs=8 * 136)),
    (-2, dict(hq=129, h=1, qs=129 * 128)), (-2, dict(reqs=4097)),
    (-1, dict(qs=128)), (-1, dict(ks=128)), (-1, dict(vs=128)),
    (-2, dict(qs=32 * 128 + 4)), (-2, dict(ks=8 * 128 + 4)), (-2, dict(vs=8 * 128 + 4)),
    (-1, dict(query=N)), (-1, dict(key=N)), (-1, dict(value=N)), (-1, dict(out=N)),
    (-1, dict(q_start=N)), (-1, dict(k_start=N)), (-1, dict(query=A[0] + 8)),
    (-1, dict(key=A[1] + 8)), (-1, dict(value=A[2] + 8)), (-1, dict(out=A[5] + 8)),
    (-1, dict(q_start=A[3] + 2)), (-1, dict(err=A[6] + 1)),
    (-1, dict(out=A[0])), (-1, dict(out=A[1] + 16)), (-1, dict(out=A[2])),
    (0, dict(reqs=0)), (0, dict(nq=0)),
])
def test_prompt_attention_refuses(lib, want, change):
    assert lib.kv_attention_prompt(*{**PROMPT, **change}.values()) == want


WRITE4 = dict(key=A[0], ks=8 * 128, value=A[1], vs=8 * 128, kc=A[2], vc=A[3], slots=A[4], n=4, layer=0,
              layers=1, blocks=8, t=16, h=8, d=128, err=N, stream=N)


@pytest.mark.parametrize("want,change", [
    (-1, dict(n=-1)), (-1, dict(layer=1)), (-1, dict(layers=0)), (-1, dict(blocks=0)), (-1, dict(t=0)),
    (-1, dict(h=0)), (-1, dict(d=0)), (-2, dict(d=96)), (-2, dict(d=256)), (-2, dict(t=12)),
    (-2, dict(h=4097)), (-1, dict(ks=8)), (-1, dict(vs=8)), (-2, dict(ks=8 * 128 + 4)),
    (-1, dict(key=N)), (-1, dict(value=N)), (-1, dict(kc=N)), (-1, dict(vc=N)), (-1, dict(slots=N)),
    (-1, dict(key=A[0] + 8)), (-1, dict(kc=A[2] + 8)), (-1, dict(vc=A[3] + 4)), (-1, dict(slots=A[4] + 4)),
    (-1, dict(err=A[5] + 2)), (0, dict(n=0)),
])
def test_write_q4_refuses(lib, want, change):
    assert lib.kv_cache_write_q4(*{**WRITE4, **change}.values()) == want


GATHER4 = dict(kc=A[0], vc=A[1], layer=0, layers=1, blocks=8, t=16, h=8, d=128, table=A[2], stride=4,
               g0=A[3], g1=A[4], reqs=2, ko=A[5], vo=A[6], rows=10, err=N, stream=N)


@pytest.mark.parametrize("want,change", [
    (-1, dict(layer=-1)), (-1, dict(reqs=-1)), (-1, dict(rows=-1)), (-1, dict(stride=-1)),
    (-2, dict(reqs=4097)), (-2, dict(d=80)), (-2, dict(t=4)), (-1, dict(table=N)), (-1, dict(g0=N)),
    (-1, dict(g1=N)), (-1, dict(kc=N)), (-1, dict(vc=N)), (-1, dict(ko=N)), (-1, dict(vo=A[6] + 8)),
    (-1, dict(table=A[2] + 2)), (0, dict(reqs=0)),
])
def test_gather_q4_refuses(lib, want, change):
    assert lib.kv_cache_gather_q4(*{**GATHER4, **change}.values()) == want


ATTEND4 = dict(query=A[0], qs=32 * 128, kc=A[1], vc=A[2], layer=0, layers=1, blocks=8, t=16, hq=32, h=8,
               d=128, table=A[3], stride=4, s0=A[4], s1=A[5], reqs=2, scale=0.1, out=A[6], ws=A[7],
               ws_bytes=1 << 40, err=N, stream=N)


@pytest.mark.parametrize("want,change", [
    (-1, dict(layer=1)), (-1, dict(reqs=-1)), (-1, dict(stride=-1)), (-1, dict(hq=0)), (-1, dict(hq=31)),
    (-1, dict(scale=0.0)), (-1, dict(scale=float("nan"))), (-1, dict(ws_bytes=-1)), (-2, dict(reqs=4097)),
    (-2, dict(d=32)), (-2, dict(t=20)), (-1, dict(qs=8)), (-2, dict(qs=32 * 128 + 4)),
    (-1, dict(query=N)), (-1, dict(out=N)), (-1, dict(s0=N)), (-1, dict(s1=N)), (-1, dict(kc=N)),
    (-1, dict(vc=N)), (-1, dict(table=N)), (-1, dict(query=A[0] + 8)), (-1, dict(out=A[6] + 8)),
    (-1, dict(kc=A[1] + 8)), (-1, dict(s0=A[4] + 2)), (-1, dict(err=A[8] + 2)), (-1, dict(out=A[0])),
    (0, dict(reqs=0)),
])
def test_attention_q4_refuses(lib, want, change):
    assert lib.kv_attention_q4(*{**ATTEND4, **change}.values()) == want


def test_attention_q4_workspace_arguments(lib):
    assert lib.kv_attention_q4_workspace(-1, 32, 8, 128) == -1
    assert lib.kv_attention_q4_workspace(1, 31, 8, 128) == -1
    assert lib.kv_attention_q4_workspace(1, 32, 0, 128) == -1
    assert lib.kv_attention_q4_workspace(0, 32, 8, 128) >= 0
    need = lib.kv_attention_q4_workspace(4, 32, 8, 128)
    assert need >= 0
    if need > 0:
        assert lib.kv_attention_q4(*{**ATTEND4, "reqs": 4, "ws_bytes": need - 1}.values()) == -1
        assert lib.kv_attention_q4(*{**ATTEND4, "reqs": 4, "ws": N}.values()) == -1


def test_binding_refuses_cpu_tensors_and_bad_caches():
    import torch
    import paged_kv_cache_39_gb300 as kv
    x = torch.zeros((2, 8, 64), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kv.kv_attention_prompt(x, x, x, i)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kv.kv_qk_norm_rope_write(x, x, None, x[0, 0], x[0, 0], i.long(), torch.zeros(4, 64))
    with pytest.raises(ValueError, match="CUDA tensor"):
        kv.kv_cache_write_q4(x, x, x, x, i.long(), 16)
    with pytest.raises(ValueError, match="block_size"):
        kv.new_q4_cache(1, 4, 12, 8, 128, device="cpu")
    with pytest.raises(ValueError, match="head_dim"):
        kv.new_q4_cache(1, 4, 16, 8, 96, device="cpu")
    c = kv.new_q4_cache(2, 4, 16, 8, 128, device="cpu")
    assert tuple(c.shape) == (2, 4, 8, 16 * 72) and c.dtype == torch.uint8


@pytest.mark.parametrize("change", [dict(nq=2 ** 31 - 60000), dict(nk=2 ** 31 - 1)])
def test_prompt_attention_refuses_rows_past_its_indices(lib, change):
    assert lib.kv_attention_prompt(*{**PROMPT, **change}.values()) == -2
