"""The operators around the cache in a run, as a serving loop uses them: a layer's
prompt, chunks behind it and single tokens, over the bf16 and the 4-bit cache."""
import numpy as np
import pytest
import torch

import operator_refs as ref
import paged_kv_cache_39_gb300 as kv
from operator_refs import BF16, dev, normal
from test_gpu_cache_q4 import i32

pytestmark = pytest.mark.gpu
T, HQ, H, D, ROT = 16, 8, 2, 128, 128
STEP = 2.0 ** -8


def rotation():
    p = torch.arange(600, dtype=torch.float64, device=dev())[:, None]
    a = p * 10000.0 ** (-torch.arange(0, ROT, 2, dtype=torch.float64, device=dev()) / ROT)
    return torch.cat([a.cos(), a.sin()], 1).float()


@pytest.mark.parametrize("bits", [16, 4])
def test_prompt_chunk_and_tokens(bits):
    """Two requests: a prompt, a second chunk, then three single tokens.  Every step's output is
    compared with attention in 64 bits over the rows the cache stands for."""
    cs, qw, kw = rotation(), normal((D,), 1, 0.3) + 1, normal((D,), 2, 0.3) + 1
    table = np.random.default_rng(0).permutation(np.arange(1, 65)).reshape(2, 32).astype(np.int32)
    tab, B = i32(table), 70
    if bits == 16:
        kc = torch.zeros((1, B, T, H, D), dtype=BF16, device=dev())
        vc = torch.zeros_like(kc)
    else:
        kc, vc = kv.new_q4_cache(1, B, T, H, D), kv.new_q4_cache(1, B, T, H, D)
    ctx = np.zeros(2, np.int64)
    err = kv.new_error_word(dev())
    for step, new in enumerate(([150, 37], [64, 201], [1, 1], [1, 1], [1, 1])):
        n = sum(new)
        qkv = normal((n, HQ + 2 * H, D), 10 + step)
        q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + H], qkv[:, HQ + H:]
        pos = np.concatenate([np.arange(c, c + m) for c, m in zip(ctx, new)])
        qsl = i32([0, new[0], n])
        pos_d = torch.from_numpy(pos).to(dev())
        slots = kv.kv_slot_mapping_paged(qsl, pos_d, tab, T, B, err=err)
        args = (q, k, v, qw, kw, pos_d, cs)
        if bits == 16:
            qr, kr = kv.kv_qk_norm_rope_write(*args, k_cache=kc, v_cache=vc, slot_mapping=slots, err=err)
        else:
            qr, kr = kv.kv_qk_norm_rope_write(*args, err=err)
            kv.kv_cache_write_q4(kr, v, kc, vc, slots, T, err=err)
        ctx += new
        total = int(ctx.sum())
        end = i32(ctx)
        ksl = i32([0, ctx[0], total])
        if bits == 16:
            kg, vg = kv.kv_cache_gather(kc, vc, tab, i32([0, 0]), end, out_rows=total, err=err)
            out = kv.kv_attention_prompt(qr, kg, vg, qsl, ksl, err=err)
            kx, vx = kg.to(ref.F64), vg.to(ref.F64)
        else:
            at = np.concatenate([table[r, np.arange(c) // T].astype(np.int64) * T + np.arange(c) % T
                                 for r, c in enumerate(ctx)])
            kx, vx = ref.values(kc, T, D, 0, at), ref.values(vc, T, D, 0, at)
            if new == [1, 1]:
                out = kv.kv_attention_q4(qr, kc, vc, tab, i32([0, 0]), end, T, err=err)
            else:
                kg, vg = kv.kv_cache_gather_q4(kc, vc, tab, i32([0, 0]), end, T, D, out_rows=total, err=err)
                out = kv.kv_attention_prompt(qr, kg, vg, qsl, ksl, err=err)
                kx, vx = kg.to(ref.F64), vg.to(ref.F64)
        at = 0
        for r in range(2):
            lo, hi = (0, int(ctx[0])) if r == 0 else (int(ctx[0]), total)
            m = new[r]
            o, b = ref.attend(qr[at:at + m], kx[lo:hi], vx[lo:hi], np.arange(m) + hi - lo - m + 1,
                              D ** -0.5, STEP)
            ref.check(out[at:at + m], o, b, f"step {step} request {r}")
            at += m
        # what the cache stands for is what went in: bit for bit, or within half a 4-bit step
        rows = slice(int(ctx[0]) - new[0], int(ctx[0]))
        want = kr[:new[0]].to(ref.F64)
        if bits == 16:
            assert torch.equal(kx[rows], want)
        else:
            top = want.view(new[0], H, D // 32, 32).abs().amax(-1, keepdim=True)
            d = (kx[rows] - want).abs().view(new[0], H, D // 32, 32)
            # half a step, the scale's bf16 rounding (on 7 codes) and the gather's bf16 rounding
            assert (d <= top * (0.5 / 7 * (1 + 2.0 ** -8) + 2.0 ** -8 + 2.0 ** -8)).all()
    assert err.item() == 0
