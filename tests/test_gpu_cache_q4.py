"""The 4-bit cache: write and gather, bit for bit against a byte-by-byte host
implementation of the layout's formula."""
import numpy as np
import pytest
import torch

import operator_refs as ref
import paged_kv_cache_39_gb300 as kv
from operator_refs import BF16, dev, normal

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=dev())


def random_cache(L, B, T, H, D, seed):
    """Any bytes as codes, positive finite scales."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = torch.randint(0, 256, (L, B, H, T * (D // 2 + D // 16)), generator=g, device="cuda",
                      dtype=torch.uint8)
    s = torch.rand((L, B, H, T * D // 32), generator=g, device="cuda").mul(0.9).add(0.1).to(BF16)
    c[..., T * D // 2:] = s.view(torch.uint8)
    return c


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,H,n", [(8, 1, 1), (16, 8, 37), (48, 3, 130), (16, 5, 9)])
def test_write_bits(D, T, H, n):
    B, L = 24, 2
    kc, vc = random_cache(L, B, T, H, D, 1), random_cache(L, B, T, H, D, 2)
    wk, wv = kc.cpu().numpy().copy(), vc.cpu().numpy().copy()
    qkv = normal((n, 3 * H, D), 3, 3.0)
    k, v = qkv[:, :H], qkv[:, H:2 * H]
    slots = np.random.default_rng(4).permutation(np.arange(T, B * T))[:n]
    err = kv.new_error_word(dev())
    kv.kv_cache_write_q4(k, v, kc, vc, torch.from_numpy(slots).to(dev()), T, layer=1, err=err)
    ref.put_rows(wk, T, 1, slots, k)
    ref.put_rows(wv, T, 1, slots, v)
    assert np.array_equal(kc.cpu().numpy(), wk) and np.array_equal(vc.cpu().numpy(), wv)
    assert err.item() == 0


def test_write_ties_zeros_extremes():
    """Rows made of halves of their scale (every tie), of one value, of zeros, of the
    largest and the smallest bf16 values."""
    T, H, D, n = 16, 1, 128, 7
    x = torch.zeros((n, H, D), dtype=torch.float32)
    for i, top in enumerate((7.0, 3.5, 1.109375, 448.0)):     # scale = bf16(top / 7)
        s = float(torch.tensor(top / 7).to(BF16))
        x[i, 0] = torch.tensor([(j % 29 - 14) * 0.5 * s for j in range(D)])
        x[i, 0, ::32] = top
    x[4, 0, :64] = 3.3895e38
    x[4, 0, 64:] = 1.1754944e-38     # scale below the normal range
    x[5, 0] = 9.2e-41                # subnormal
    x = x.to(BF16).to(dev())
    kc, vc = random_cache(1, 4, T, H, D, 1), random_cache(1, 4, T, H, D, 2)
    wk, wv = kc.cpu().numpy().copy(), vc.cpu().numpy().copy()
    slots = np.arange(T, T + n)
    kv.kv_cache_write_q4(x, -x, kc, vc, torch.from_numpy(slots).to(dev()), T)
    ref.put_rows(wk, T, 0, slots, x)
    ref.put_rows(wv, T, 0, slots, -x)
    assert np.array_equal(kc.cpu().numpy(), wk) and np.array_equal(vc.cpu().numpy(), wv)


def test_write_not_finite_groups_read_as_nan():
    T, H, D = 8, 2, 64
    x = normal((3, H, D), 1)
    x[0, 0, 3] = float("nan")
    x[1, 1, 40] = float("inf")
    x[2, 0, 33] = -float("inf")
    kc, vc = kv.new_q4_cache(1, 4, T, H, D), kv.new_q4_cache(1, 4, T, H, D)
    kv.kv_cache_write_q4(x, x, kc, vc, torch.tensor([8, 9, 10], device=dev()), T)
    k, v = kv.kv_cache_gather_q4(kc, vc, i32([[1]]), i32([0]), i32([3]), T, D, out_rows=3)
    for out in (k, v):
        nan = torch.isnan(out.float()).view(3, H, 2, 32).all(-1)
        any_nan = torch.isnan(out.float()).view(3, H, 2, 32).any(-1)
        want = torch.zeros((3, H, 2), dtype=torch.bool, device=dev())
        want[0, 0, 0] = want[1, 1, 1] = want[2, 0, 1] = True
        assert torch.equal(nan, want) and torch.equal(any_nan, want)


def test_write_slots_refused_and_padded_rows():
    T, H, D, B = 16, 2, 128, 6
    kc, vc = random_cache(1, B, T, H, D, 1), random_cache(1, B, T, H, D, 2)
    wk, wv = kc.cpu().numpy().copy(), vc.cpu().numpy().copy()
    x = normal((6, H, D), 3)
    slots = np.array([-1, 3, B * T, 20, -7, 21])
    err = kv.new_error_word(dev())
    kv.kv_cache_write_q4(x, x, kc, vc, torch.from_numpy(slots).to(dev()), T, num_tokens=5, err=err)
    ref.put_rows(wk, T, 0, slots[:5], x[:5])
    ref.put_rows(wv, T, 0, slots[:5], x[:5])
    assert np.array_equal(kc.cpu().numpy(), wk) and np.array_equal(vc.cpu().numpy(), wv)
    assert err.item() == kv.ERR_BITS["NULL_WRITE"] | kv.ERR_BITS["BAD_SLOT"]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,H,R,stride", [(8, 1, 3, 7), (16, 8, 40, 9), (48, 3, 5, 4), (16, 130, 2, 3)])
def test_gather(D, T, H, R, stride):
    rng = np.random.default_rng(R)
    B, L = 64, 2
    kc, vc = random_cache(L, B, T, H, D, 5), random_cache(L, B, T, H, D, 6)
    table = rng.integers(-1, B + 2, (R, stride)).astype(np.int32)
    table[rng.random(table.shape) < 0.2] = 0
    start = rng.integers(0, stride * T, R)
    end = start + rng.integers(0, 2 * T, R)
    start[0], end[0] = 3, 3                       # empty
    if R > 2:
        start[1], end[1] = 5, 2                   # invalid
        start[2] = -1
    slots, bits = [], 0
    for r in range(R):
        if start[r] < 0 or end[r] < start[r]:
            bits |= kv.ERR_BITS["BAD_POSITION"]
            continue
        for p in range(start[r], end[r]):
            if p // T >= stride:
                bits |= kv.ERR_BITS["BAD_POSITION"]
                slots.append(-1)
                continue
            b = table[r, p // T]
            if b < 0 or b >= B:
                bits |= kv.ERR_BITS["BAD_BLOCK"]
            slots.append(b * T + p % T if 0 < b < B else -1)
    rows = len(slots) + 5
    k = torch.full((rows, H, D), 7.0, dtype=BF16, device=dev())
    v = torch.full((rows, H, D), 7.0, dtype=BF16, device=dev())
    err = kv.new_error_word(dev())
    kv.kv_cache_gather_q4(kc, vc, i32(table), i32(start), i32(end), T, D, layer=1, k_out=k, v_out=v, err=err)
    n = len(slots)
    for out, cache in ((k, kc), (v, vc)):
        # the product of a code and a bf16 scale has 12 bits, so 64 -> 32 -> 16 bits rounds once
        assert torch.equal(out[:n], ref.values(cache, T, D, 1, slots).float().to(BF16))
        assert (out[n:] == 7).all()               # rows behind the last span
    assert err.item() == bits
    short = max(n - 3, 0)
    k.fill_(7), v.fill_(7), err.zero_()
    kv.kv_cache_gather_q4(kc, vc, i32(table), i32(start), i32(end), T, D, layer=1, k_out=k, v_out=v,
                          out_rows=short, err=err)
    assert (k[short:] == 7).all() and torch.equal(v[:short], ref.values(vc, T, D, 1, slots[:short]).float().to(BF16))
    assert (err.item() & kv.ERR_BITS["OUT_OF_SPACE"] != 0) == (n > short)


def test_copy_blocks_of_a_4bit_cache():
    for bulk in (False, True):
        kc, vc = random_cache(3, 10, 16, 4, 128, 1), random_cache(3, 10, 16, 4, 128, 2)
        k0, v0 = kc.clone(), vc.clone()
        kv.kv_copy_blocks(kc, vc, i32([1, 3]), i32([8, 9]), bulk=bulk)
        k0[:, [8, 9]], v0[:, [8, 9]] = k0[:, [1, 3]], v0[:, [1, 3]]
        assert torch.equal(kc, k0) and torch.equal(vc, v0)


def test_records_past_four_gigabytes():
    """The last block of a cache of more than 2^32 bytes, written and read back."""
    T, H, D = 16, 8, 128
    B = (1 << 32) // (H * T * 72) + 1000
    free, _ = torch.cuda.mem_get_info()
    if free < 3 * B * H * T * 72:
        pytest.skip("needs 14 GB")
    kc = torch.empty((1, B, H, T * 72), dtype=torch.uint8, device=dev())
    vc = torch.empty_like(kc)
    x = normal((T, H, D), 1)
    slots = torch.arange((B - 1) * T, B * T, device=dev())
    kv.kv_cache_write_q4(x, -x, kc, vc, slots, T)
    k, v = kv.kv_cache_gather_q4(kc, vc, i32([[B - 1]]), i32([0]), i32([T]), T, D, out_rows=T)
    codes, scale, _ = ref.quantise(x)
    want = torch.from_numpy((codes.reshape(T, H, 4, 32) - 8) * scale[..., None]).reshape(T, H, D)
    assert torch.equal(k.cpu(), want.float().to(BF16)) and torch.equal(v.cpu(), (-want).float().to(BF16))
    o = kv.kv_attention_q4(x[:1], kc, vc, i32([[B - 1]]), i32([0]), i32([T]), T)
    wo, bound = ref.attend(x[:1], want.to(dev()), -want.to(dev()), [T], D ** -0.5, 2.0 ** -8,
                           unit=ref.units(vc, T, D, 0, slots.cpu()))
    ref.check(o, wo, bound)
