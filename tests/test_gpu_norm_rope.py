"""kv_qk_norm_rope_write against its formula in 64 bits."""
import numpy as np
import pytest
import torch

import operator_refs as ref
import paged_kv_cache_39_gb300 as kv
from operator_refs import BF16, dev, normal

pytestmark = pytest.mark.gpu
POSITIONS = 512


def table(rotary):
    p = torch.arange(POSITIONS, dtype=torch.float64, device=dev())[:, None]
    a = p * 10000.0 ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device=dev()) / rotary)
    return torch.cat([a.cos(), a.sin()], 1).float()


def case(n, hq, h, d, rotary, seed=0, packed=True, blocks=64, t=16):
    rng = np.random.default_rng(seed)
    if packed:
        qkv = normal((n, hq + 2 * h, d), seed, 2.0)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + h], qkv[:, hq + h:]
    else:
        q, k, v = normal((n, hq, d), seed, 2.0), normal((n, h, d), seed + 1), normal((n, h, d), seed + 2)
    slots = rng.permutation(np.arange(t, blocks * t))[:n].astype(np.int64)
    return dict(q=q, k=k, v=v, qw=(1 + normal((d,), seed + 3, 0.3).float()).to(BF16),
                kw=(1 + normal((d,), seed + 4, 0.3).float()).to(BF16),
                pos=torch.from_numpy(rng.integers(0, POSITIONS, n)).to(dev()), cs=table(rotary),
                slots=torch.from_numpy(slots).to(dev()),
                kc=normal((2, blocks, t, h, d), seed + 5), vc=normal((2, blocks, t, h, d), seed + 6))


def want(c, rotary, inter, eps):
    rows = c["cs"][c["pos"].clamp(0, POSITIONS - 1)]
    return (ref.norm_rope(c["q"], c["qw"], rows, rotary, inter, eps),
            ref.norm_rope(c["k"], c["kw"], rows, rotary, inter, eps))


def call(c, eps=1e-6, inter=False, **kw):
    return kv.kv_qk_norm_rope_write(c["q"], c["k"], c["v"], c["qw"], c["kw"], c["pos"], c["cs"],
                                    k_cache=c["kc"], v_cache=c["vc"], slot_mapping=c["slots"], eps=eps,
                                    interleaved=inter, **kw)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("n,hq,h,d,rotary", [
    (1, 1, 1, 8, 8), (3, 2, 1, 16, 8), (5, 4, 4, 64, 64), (7, 16, 8, 64, 32), (33, 3, 1, 96, 96),
    (129, 32, 8, 128, 128), (64, 30, 5, 128, 32), (17, 8, 2, 256, 64), (2, 7, 7, 200, 200),
    (1, 64, 8, 128, 128), (700, 8, 1, 72, 24),
])
def test_rows_and_caches(n, hq, h, d, rotary, inter):
    c = case(n, hq, h, d, rotary, seed=n)
    kc0, vc0 = c["kc"].clone(), c["vc"].clone()
    err = kv.new_error_word(dev())
    q_out, k_out = call(c, inter=inter, layer=1, err=err)
    (wq, bq), (wk, bk) = want(c, rotary, inter, 1e-6)
    ref.check(q_out, wq, bq, "q")
    ref.check(k_out, wk, bk, "k")
    s = c["slots"]
    kc0[1].flatten(0, 1)[s] = k_out          # the cache holds the same bits as k_out, v the input's
    vc0[1].flatten(0, 1)[s] = c["v"]
    assert torch.equal(c["kc"], kc0) and torch.equal(c["vc"], vc0)
    assert err.item() == 0


@pytest.mark.parametrize("eps,scale", [(1e-6, 1e-3), (1e-2, 1.0), (0.0, 1.0), (1e-6, 1e4)])
def test_epsilon_and_magnitude(eps, scale):
    c = case(9, 8, 2, 128, 128, seed=5, packed=False)
    c["q"], c["k"] = (c["q"].float() * scale).to(BF16), (c["k"].float() * scale).to(BF16)
    q_out, k_out = call(c, eps=eps)
    (wq, bq), (wk, bk) = want(c, 128, False, eps)
    ref.check(q_out, wq, bq)
    ref.check(k_out, wk, bk)


def test_zero_rows_stay_zero():
    c = case(4, 8, 2, 64, 64)
    c["q"].zero_()
    c["k"].zero_()
    q_out, k_out = call(c)
    assert not q_out.any() and not k_out.any()


def test_slots_and_positions_that_are_refused():
    c = case(8, 4, 2, 128, 64, seed=2)
    c["slots"][0] = -1                      # PAD
    c["slots"][1] = 5                       # inside the null block
    c["slots"][2] = 64 * 16                 # past the pool
    c["pos"][3] = -1
    c["pos"][4] = POSITIONS
    kc0, vc0 = c["kc"].clone(), c["vc"].clone()
    err = kv.new_error_word(dev())
    q_out, k_out = call(c, err=err)
    assert err.item() == (kv.ERR_BITS["NULL_WRITE"] | kv.ERR_BITS["BAD_SLOT"] | kv.ERR_BITS["BAD_POSITION"])
    (wq, bq), (wk, bk) = want(c, 64, False, 1e-6)
    for t in range(8):
        if t in (3, 4):
            assert not q_out[t].any() and not k_out[t].any()
        else:
            ref.check(q_out[t], wq[t], bq[t])
            ref.check(k_out[t], wk[t], bk[t])
    keep = c["slots"][5:]
    kc0[0].flatten(0, 1)[keep] = k_out[5:]
    vc0[0].flatten(0, 1)[keep] = c["v"][5:]
    assert torch.equal(c["kc"], kc0) and torch.equal(c["vc"], vc0)


def test_without_caches_in_place_and_padded():
    c = case(10, 8, 2, 128, 128, seed=3, packed=False)
    (wq, bq), (wk, bk) = want(c, 128, False, 1e-6)
    q, k = c["q"].clone(), c["k"].clone()
    got = kv.kv_qk_norm_rope_write(q, k, None, c["qw"], c["kw"], c["pos"], c["cs"], q_out=q, k_out=k,
                                   num_tokens=7)
    assert got[0] is q and got[1] is k
    ref.check(q[:7], wq[:7], bq[:7])
    ref.check(k[:7], wk[:7], bk[:7])
    assert torch.equal(q[7:], c["q"][7:]) and torch.equal(k[7:], c["k"][7:])  # rows behind the last token


def test_other_rows_nan_and_infinity_stay_theirs():
    c = case(6, 4, 2, 64, 64, seed=4, packed=False)
    c["q"][2, 1, 5] = float("nan")
    c["k"][4, 0, 9] = float("inf")
    q_out, k_out = call(c)
    assert torch.isnan(q_out[2, 1]).all()
    assert torch.isnan(k_out[4, 0, 9].float()) or torch.isnan(k_out[4, 0]).any()
    q_out[2, 1], k_out[4, 0] = 0, 0
    assert torch.isfinite(q_out.float()).all() and torch.isfinite(k_out.float()).all()


def test_prepared_call_replayed_from_a_graph_on_another_stream():
    c = case(40, 32, 8, 128, 128, seed=6)
    run = call(c, prepare=True)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    c["q"].copy_(normal(c["q"].shape, 77))
    c["k"].copy_(normal(c["k"].shape, 78))
    c["kc"].zero_()
    g.replay()
    torch.cuda.synchronize()
    (wq, bq), (wk, bk) = want(c, 128, False, 1e-6)
    ref.check(run.result[0], wq, bq)
    ref.check(run.result[1], wk, bk)
    assert torch.equal(c["kc"][0].flatten(0, 1)[c["slots"]], run.result[1])


def test_binding_refusals():
    c = case(4, 8, 2, 128, 128)
    with pytest.raises(ValueError, match="needs k_cache"):
        kv.kv_qk_norm_rope_write(c["q"], c["k"], None, c["qw"], c["kw"], c["pos"], c["cs"], k_cache=c["kc"],
                                 v_cache=c["vc"], slot_mapping=c["slots"])
    with pytest.raises(ValueError, match="contiguous"):
        kv.kv_qk_norm_rope_write(c["q"].transpose(1, 2).contiguous().transpose(1, 2), c["k"], None, c["qw"],
                                 c["kw"], c["pos"], c["cs"])
    with pytest.raises(TypeError):
        kv.kv_qk_norm_rope_write(c["q"].half(), c["k"], None, c["qw"], c["kw"], c["pos"], c["cs"])
    with pytest.raises(ValueError, match="num_tokens"):
        call(c, num_tokens=5)
    q = c["q"].contiguous()
    with pytest.raises(kv.KVError):   # q_out one row into query: another head's rows
        kv.kv_qk_norm_rope_write(q[:3], c["k"][:3], None, c["qw"], c["kw"], c["pos"], c["cs"], q_out=q[1:])


def test_rows_past_two_billion_elements():
    """Token strides and slots whose elements are counted past 2^31."""
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 30 GB")
    n, hq, h, d, T = 3, 8, 8, 128, 16
    c = case(n, hq, h, d, d, seed=3, packed=False)
    (wq, bq), (wk, bk) = want(c, d, False, 1e-6)
    stride = 2 ** 30 + 8                               # the last token's row starts past 2^31
    far = {}
    for name in ("q", "k", "v"):
        buffer = torch.empty(2 * stride + h * d, dtype=BF16, device=dev())
        far[name] = buffer.as_strided((n, h, d), (stride, d, 1))
        far[name].copy_(c[name])
    blocks = 2 ** 31 // (T * h * d) + 2
    kc = torch.empty((1, blocks, T, h, d), dtype=BF16, device=dev())
    vc = torch.empty_like(kc)
    slots = torch.arange(n, device=dev()) + (blocks - 1) * T + 5
    q_out, k_out = kv.kv_qk_norm_rope_write(far["q"], far["k"], far["v"], c["qw"], c["kw"], c["pos"], c["cs"],
                                            k_cache=kc, v_cache=vc, slot_mapping=slots)
    ref.check(q_out, wq, bq, "q")
    ref.check(k_out, wk, bk, "k")
    assert torch.equal(kc[0, -1, 5:5 + n], k_out) and torch.equal(vc[0, -1, 5:5 + n], c["v"])
