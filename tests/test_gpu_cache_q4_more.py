"""The 4-bit cache: refusals of the block copy, and scales and codes of every bf16 magnitude."""
import numpy as np
import pytest
import torch

import operator_refs as ref
import paged_kv_cache_39_gb300 as kv
from operator_refs import BF16, dev
from test_gpu_cache_q4 import i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("record", [33, 32, 64, 300, 288 * 3 + 16])
@pytest.mark.parametrize("bulk", [False, True])
def test_block_copy_refuses_bytes_that_are_no_4_bit_cache(record, bulk):
    c = torch.zeros((2, 4, 2, record), dtype=torch.uint8, device=dev())
    with pytest.raises(ValueError, match="4-bit"):
        kv.kv_copy_blocks(c, c.clone(), i32([1]), i32([2]), bulk=bulk)


def write(x, T=32):
    """(got, want) caches of rows x [n, 1, D] bf16 written one to a slot, as key and as value."""
    n, _, D = x.shape
    B = -(-n // T) + 1
    kc, vc = (kv.new_q4_cache(1, B, T, 1, D, device=dev()) for _ in range(2))
    slots = np.arange(T, T + n)
    kv.kv_cache_write_q4(x, x, kc, vc, torch.from_numpy(slots).to(dev()), T)
    codes, _, bits = ref.quantise(x)
    g = D // 32
    ch = np.arange(D)
    at = 2 * g * (ch % 32 // 4) + 2 * (ch // 32) + ch % 4 // 2
    rows = np.zeros((n, D // 2), np.uint8)
    rows[:, at[::2]] = codes[:, 0, ::2] | codes[:, 0, 1::2] << 4
    want = np.zeros((B, T * (D // 2 + D // 16)), np.uint8)
    for r, s in enumerate(slots):
        want[s // T, s % T * D // 2:(s % T + 1) * D // 2] = rows[r]
        lo = T * D // 2 + s % T * D // 16
        want[s // T, lo:lo + D // 16] = bits[r, 0].astype(np.int16).view(np.uint8)
    return [c[0, :, 0].cpu().numpy() for c in (kc, vc)], want


@pytest.mark.parametrize("D", [64, 128])
def test_the_scale_of_every_magnitude(D):
    """Each finite bf16 magnitude as a group's largest: scale and codes, bit for bit."""
    m = torch.arange(0x7f80, dtype=torch.int32).to(torch.int16).view(BF16).view(-1, D // 32)
    x = torch.zeros((m.shape[0], 1, D // 32, 32), dtype=BF16)
    x[:, 0, :, 5] = -m
    x[:, 0, :, 9] = (m.float() * 0.37).to(BF16)
    got, want = write(x.flatten(2).to(dev()))
    assert all(np.array_equal(c, want) for c in got)


def test_the_codes_of_every_pair_of_mantissas():
    """Every mantissa as a group's largest with every value down to 2^-6 of it: codes bit for bit."""
    top = torch.arange(0x3f80, 0x4000, dtype=torch.int32)                  # 1 to 2
    x = torch.arange(0x3f80 - 6 * 128, 0x4000, dtype=torch.int32)
    x = torch.cat([x, torch.full((-len(x) % 31,), 0)]).view(-1, 31)        # 31 values to a group
    both = torch.cat([top[:, None, None].expand(-1, len(x), 1),
                      torch.minimum(x[None].expand(len(top), -1, -1), top[:, None, None])], -1)
    sign = torch.from_numpy(np.random.default_rng(1).integers(0, 2, tuple(both.shape))).int() * 0x8000
    rows = (both + sign).to(torch.int32).bitwise_and(0xffff)
    rows = torch.where(rows >= 0x8000, rows - 0x10000, rows).to(torch.int16).view(BF16)
    rows = rows.reshape(-1, 32)
    rows = rows[:len(rows) // 2 * 2].reshape(-1, 1, 64).contiguous()
    got, want = write(rows.to(dev()))
    assert all(np.array_equal(c, want) for c in got)
