"""Plain 64-bit implementations of the operators around the paged cache, written
from their formulas, with the error bounds the tests use.

Roundings counted by the bounds (half a step each): bf16 2^-8, fp16 2^-11, fp32
2^-24, relative to the value that is rounded.
"""
import numpy as np
import torch

F64 = torch.float64
BF16 = torch.bfloat16


def dev():
    return torch.device("cuda:0")


def normal(shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(BF16)


# ---------------------------------------------------------------------------
# norm and rotation


def norm_rope(x, w, rows, rotary, interleaved, eps):
    """(y, bound of |got - y|) of head rows x [N, H, D]; rows [N, rotary] of cos, sin."""
    d = x.shape[-1]
    x, w, rows = x.to(F64), w.to(F64), rows.to(F64)
    y = x * w / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    c, s = rows[:, None, :rotary // 2], rows[:, None, rotary // 2:]
    i = torch.arange(rotary // 2, device=x.device)
    a_at, b_at = (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)
    a, b = y[..., a_at].clone(), y[..., b_at].clone()
    size = y.abs().clone()  # what the last sums add up, in magnitude
    y[..., a_at], y[..., b_at] = a * c - b * s, b * c + a * s
    size[..., a_at] = size[..., b_at] = a.abs() + b.abs()
    # the mean sums d squares, the root, two products, the rotation: under d + 16
    # roundings of 32 bits on `size`; then one to bf16
    return y, y.abs() * 2.0 ** -8 + size * ((d + 16) * 2.0 ** -24)


# ---------------------------------------------------------------------------
# 4-bit rows (numpy, channel by channel of the layout's formula)


def quantise(x):
    """(codes [.., D], scale [.., D/32] as float64, bf16 bits of the scale) of bf16 rows."""
    v = x.to(F64).cpu().numpy().reshape(*x.shape[:-1], -1, 32)
    top = np.abs(v).max(-1)
    with np.errstate(all="ignore"):
        s = torch.from_numpy((top / 7).astype(np.float32)).to(BF16)
        s = torch.where(s < 2.0 ** -126, torch.zeros_like(s), s)
        s = torch.where(torch.from_numpy(~np.isfinite(v).all(-1)), torch.full_like(s, float("nan")), s)
        sf = s.to(F64).numpy()
        q = np.where(sf[..., None] > 0, np.rint(v / np.where(sf > 0, sf, 1)[..., None]), 0)
    assert np.abs(q).max(initial=0) <= 7
    return (q.astype(np.int64) + 8).reshape(x.shape), sf, s.view(torch.int16).numpy()


def put_rows(cache, block_size, layer, slots, x):
    """Write bf16 rows x [N, H, D] at `slots` of a host cache (uint8 numpy), byte by byte."""
    n, h, d = x.shape
    g = d // 32
    codes, _, bits = quantise(x)
    for t, s in enumerate(slots):
        b, off = divmod(int(s), block_size)
        if s < 0 or b == 0 or b >= cache.shape[1]:
            continue
        for head in range(h):
            rec = cache[layer, b, head]
            for ch in range(0, d, 2):
                at = off * d // 2 + 2 * g * (ch % 32 // 4) + 2 * (ch // 32) + ch % 4 // 2
                rec[at] = codes[t, head, ch] | codes[t, head, ch + 1] << 4
            for j in range(g):
                at = block_size * d // 2 + off * d // 16 + 2 * j
                rec[at:at + 2] = np.frombuffer(np.int16(bits[t, head, j]).tobytes(), np.uint8)


def values(cache, block_size, head_dim, layer, slots):
    """Rows [n, H, D] (float64, on the GPU) that a 4-bit cache holds at `slots`; slot < 0 gives zeros."""
    cache = torch.as_tensor(cache, device=dev())
    slots = torch.as_tensor(np.asarray(slots), device=dev()).long()
    d, g, h = head_dim, head_dim // 32, cache.shape[2]
    ch = torch.arange(d, device=dev())
    at = 2 * g * (ch % 32 // 4) + 2 * (ch // 32) + ch % 4 // 2
    s = slots.clamp_min(0)
    b, off = (s // block_size)[:, None, None], (s % block_size)[:, None, None]
    head = torch.arange(h, device=dev())[None, :, None]
    byte = cache[layer][b, head, off * (d // 2) + at].int()
    code = torch.where(ch % 2 == 1, byte >> 4, byte & 15) - 8
    scale = cache.view(torch.int16)[layer][b, head, block_size * d // 4 + off * g + ch // 32]
    v = code.to(F64) * scale.view(BF16).to(F64)
    v[slots < 0] = 0
    return v


def units(cache, block_size, head_dim, layer, slots):
    """The largest scale of each row [n, H] that a 4-bit cache holds at `slots`."""
    slots = torch.as_tensor(np.asarray(slots), device=dev()).long()
    g, h = head_dim // 32, cache.shape[2]
    b, off = (slots // block_size)[:, None, None], (slots % block_size)[:, None, None]
    at = block_size * head_dim // 4 + off * g + torch.arange(g, device=dev())
    scale = cache.view(torch.int16)[layer][b, torch.arange(h, device=dev())[None, :, None], at]
    return scale.view(BF16).to(F64).amax(-1)


# ---------------------------------------------------------------------------
# attention


def attend(q, k, v, seen, scale, weight_step, unit=None):
    """(o, bound) of query rows q [m, Hq, D] over k, v [n, H, D] (float64); query i sees the
    first seen[i] keys.  weight_step: half a step of the type the weights are rounded to.
    unit [n, H]: where weight times value scale is held in fp16, the largest scale of a row."""
    m, hq, d = q.shape
    n, h = k.shape[0], k.shape[1]
    if m == 0 or n == 0:
        z = torch.zeros((m, hq, d), dtype=F64, device=q.device)
        return z, z.clone()
    q = q.to(F64).view(m, h, hq // h, d)
    x = torch.einsum("mhgd,nhd->hgmn", q, k) * scale
    size = torch.einsum("mhgd,nhd->hgmn", q.abs(), k.abs()) * scale
    hidden = torch.arange(n, device=q.device) >= torch.as_tensor(seen, device=q.device)[:, None]
    x = x.masked_fill(hidden, -float("inf"))
    top = x.amax(-1, keepdim=True)
    w = torch.where(hidden, torch.zeros_like(x), torch.exp(x - torch.where(top.isfinite(), top, torch.zeros_like(top))))
    total = w.sum(-1, keepdim=True)
    w = torch.where(total > 0, w / total, torch.zeros_like(w))
    o = torch.einsum("hgmn,nhd->mhgd", w, v)
    a = torch.einsum("hgmn,nhd->mhgd", w, v.abs())
    # a logit sums d products, is scaled and has the maximum taken off: d + 4 roundings
    # of 32 bits (2^-23: the matrix unit may cut off instead of rounding); exp2 within
    # 2^-21; both move a weight, and the sum of the weights, by that relative amount
    seen_size = torch.where(hidden, torch.zeros_like(size), size).amax(-1)
    slack = 2 * ((d + 4) * 2.0 ** -23 * seen_size + 2.0 ** -20) + n * 2.0 ** -23
    slack = slack.permute(2, 0, 1)[..., None]
    bound = o.abs() * 2.0 ** -8 + a * (weight_step + slack)
    # a weight under 2^-126 of the largest one leaves the 32-bit range: each of n keys may
    # lose a contribution of at most 2^-126 of the largest |v|
    bound = bound + n * 2.0 ** -126 * v.abs().max()
    if unit is not None:
        # weight * scale is held in fp16 with the row's largest such product at 1 or above, so
        # one below 2^-14 is off by at most 2^-25 of it, times a code of at most 8: 2^-22 a key
        top = torch.einsum("hgmn,nh->hgmn", w, unit).amax(-1).permute(2, 0, 1)[..., None]
        bound = bound + n * 2.0 ** -22 * top
    return o.reshape(m, hq, d), bound.reshape(m, hq, d)


def check(got, want, bound, what=""):
    d = (got.to(F64) - want).abs()
    assert torch.isfinite(got.to(F64)).all(), f"{what}: not finite"
    bad = d > bound
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst "
                           f"{float((d / bound.clamp_min(1e-300)).max()):.3g} times the bound")
