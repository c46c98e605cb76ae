"""The operators of a step with drafted rows in a run, as a serving loop uses them."""
import numpy as np
import pytest
import torch

import operator_refs as ref
import paged_kv_cache_39_gb300 as kv
from operator_refs import BF16, F64, dev, normal
from step_refs import ancestors, as_int64, attend, block_table, i32, random_tree, starts

pytestmark = pytest.mark.gpu
T, HQ, H, D, V = 16, 8, 2, 128, 401


def rotation():
    p = torch.arange(600, dtype=F64, device=dev())[:, None]
    a = p * 10000.0 ** (-torch.arange(0, D, 2, dtype=F64, device=dev()) / D)
    return torch.cat([a.cos(), a.sin()], 1).float()


def test_steps_follow_one_another():
    """Three steps of a two-layer cache: layout, norm + rotation + write to the slots, attention of
    the trees, verification, kept rows moved.  After each step the cache holds exactly the rows of
    the kept tokens, and the next step's attention reads them."""
    rng = np.random.default_rng(0)
    cs, w = rotation(), torch.ones(D, dtype=BF16, device=dev())
    ctx = [37, 150, 1]
    R = len(ctx)
    table, B = block_table([c + 3 * 64 + 64 for c in ctx], T, rng)
    tab = i32(table)
    kc, vc = normal((2, B, T, H, D), 1), normal((2, B, T, H, D), 2)
    err = kv.new_error_word(dev())

    def rows_of(cache, layer, r, n):
        p = np.arange(n)
        slots = torch.from_numpy(table[r, p // T].astype(np.int64) * T + p % T).to(dev())
        return cache[layer].flatten(0, 1)[slots]

    held = [[(rows_of(kc, y, r, ctx[r]), rows_of(vc, y, r, ctx[r])) for y in range(2)] for r in range(R)]
    context = i32(ctx)
    for step, rows in enumerate(([9, 64, 1], [17, 2, 33], [1, 1, 1])):
        n, begin = sum(rows), starts(rows)
        parents = [x for m in rows for x in random_tree(m, rng)]
        masks = [x for r, m in enumerate(rows) for x in ancestors(parents[begin[r]:begin[r + 1]])]
        qsl, par = i32(begin), i32(parents)
        mask, pos, place = kv.kv_tree_layout(par, qsl, context, err=err)
        assert torch.equal(mask, as_int64(masks))
        slots = kv.kv_slot_mapping_paged(qsl, place, tab, T, B, err=err)
        new = []
        for layer in range(2):
            qkv = normal((n, HQ + 2 * H, D), 100 * step + layer)
            q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + H], qkv[:, HQ + H:]
            qr, kr = kv.kv_qk_norm_rope_write(q, k, v, w, w, pos, cs, k_cache=kc, v_cache=vc, slot_mapping=slots,
                                              layer=layer, err=err)
            out = kv.kv_attention_tree(qr, kc, vc, tab, qsl, context, max_rows=max(rows), tree_mask=mask,
                                       layer=layer, err=err)
            new.append((kr, v))
            for r, m in enumerate(rows):
                s = slice(begin[r], begin[r + 1])
                kx, vx = (torch.cat([a, b[s]]) for a, b in zip(held[r][layer], (kr, v)))
                c = len(kx) - m
                seen = np.asarray([[p < c or masks[begin[r] + i] >> (p - c) & 1 == 1 for p in range(c + m)] for i in range(m)])
                o, bound = attend(qr[s], kx, vx, seen, D ** -0.5)
                ref.check(out[s], o, bound, f"step {step} layer {layer} request {r}")
        probs = torch.softmax(2 * torch.randn((2, n, V), generator=torch.Generator(device="cuda").manual_seed(step),
                                              device=dev()), -1)
        tokens = i32(rng.integers(0, V, n))
        target = 0.5 * probs[0] + 0.5 * torch.nn.functional.one_hot(tokens.long().roll(-1), V)
        uniform = torch.rand(n, generator=torch.Generator(device="cuda").manual_seed(50 + step), device=dev())
        got, path, kept = kv.kv_verify_drafts(target, tokens, qsl, uniform, None, par, err=err)
        kv.kv_cache_keep_path(kc, vc, tab, qsl, context, path, kept, err=err)
        context = context + kept + 1
        for r in range(R):
            way = [x for x in path[begin[r]:begin[r + 1]].tolist() if x >= 0]
            assert len(way) == int(kept[r]) + 1 and all(parents[begin[r] + b] == a for a, b in zip(way, way[1:]))
            held[r] = [tuple(torch.cat([a, b[begin[r]:begin[r + 1]][way]]) for a, b in zip(held[r][y], new[y]))
                       for y in range(2)]
            for y in range(2):
                assert torch.equal(rows_of(kc, y, r, int(context[r])), held[r][y][0])
                assert torch.equal(rows_of(vc, y, r, int(context[r])), held[r][y][1])
    assert err.item() == 0


def step_buffers(seed, rows=(5, 12, 1, 8), ctx=(300, 40, 17, 1000)):
    rng = np.random.default_rng(seed)
    n = sum(rows)
    table, B = block_table([c + m for c, m in zip(ctx, rows)], T, rng)
    b = dict(kc=normal((2, B, T, H, D), seed), vc=normal((2, B, T, H, D), seed + 1), table=i32(table),
             qsl=i32(starts(rows)), ctx=i32(ctx), par=i32([x for m in rows for x in random_tree(m, rng)]),
             q=normal((n, HQ, D), seed + 2), tokens=i32(rng.integers(0, V, n)), u=torch.rand(n, device=dev()),
             p=torch.softmax(torch.randn((n, V), device=dev()), 1), d=torch.softmax(torch.randn((n, V), device=dev()), 1))
    return b


def prepared(b):
    mask, pos, place = kv.kv_tree_layout(b["par"], b["qsl"], b["ctx"])
    layout = kv.kv_tree_layout(b["par"], b["qsl"], b["ctx"], tree_mask=mask, positions=pos, cache_positions=place,
                               prepare=True)
    att = kv.kv_attention_tree(b["q"], b["kc"], b["vc"], b["table"], b["qsl"], b["ctx"], max_rows=12, tree_mask=mask,
                               layer=1, prepare=True)
    ver = kv.kv_verify_drafts(b["p"], b["tokens"], b["qsl"], b["u"], b["d"], b["par"], prepare=True)
    keep = kv.kv_cache_keep_path(b["kc"], b["vc"], b["table"], b["qsl"], b["ctx"], *ver.result[1:], prepare=True)
    return layout, att, ver, keep


def results(b):
    """The step's outputs by direct calls, on copies of the caches."""
    kc, vc = b["kc"].clone(), b["vc"].clone()
    mask, pos, place = kv.kv_tree_layout(b["par"], b["qsl"], b["ctx"])
    out = kv.kv_attention_tree(b["q"], kc, vc, b["table"], b["qsl"], b["ctx"], max_rows=12, tree_mask=mask, layer=1)
    ver = kv.kv_verify_drafts(b["p"], b["tokens"], b["qsl"], b["u"], b["d"], b["par"])
    kv.kv_cache_keep_path(kc, vc, b["table"], b["qsl"], b["ctx"], *ver[1:])
    return mask, pos, place, out, *ver, kc, vc


def outputs(b, calls):
    return (*calls[0].result, calls[1].result, *calls[2].result, b["kc"], b["vc"])


def same(got, want):
    assert all(torch.equal(g.view(torch.int16) if g.dtype == BF16 else g, w.view(torch.int16) if w.dtype == BF16 else w)
               for g, w in zip(got, want))


def test_prepared_calls_and_captured_graphs():
    """The step as prepared calls, then captured; replayed over new contents of the same buffers."""
    b, other = step_buffers(1), step_buffers(2)
    want = results(b)
    calls = prepared(b)
    for c in calls:
        c()
    same(outputs(b, calls), want)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        for c in calls:
            c()
    for name in b:
        if name not in ("table", "qsl", "ctx") and b[name].shape == other[name].shape:
            b[name].copy_(other[name])
    want = results(b)
    graph.replay()
    torch.cuda.synchronize()
    same(outputs(b, calls), want)


def test_two_streams_at_once():
    """Two steps on streams of their own, prepared calls with a workspace each, many times over."""
    bs = [step_buffers(3, (1, 2, 1), (3000, 20, 511)), step_buffers(4)]
    want = [results(b)[3] for b in bs]
    calls = [prepared(b)[1] for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    for _ in range(50):
        for c, s in zip(calls, streams):
            with torch.cuda.stream(s):
                c()
    torch.cuda.synchronize()
    for c, w in zip(calls, want):
        same([c.result], [w])


def test_two_captured_graphs_replayed_in_turn():
    bs = [step_buffers(5, (1, 2, 1), (3000, 20, 511)), step_buffers(6)]
    want = [results(b)[3] for b in bs]
    calls, graphs = [prepared(b)[1] for b in bs], []
    for c in calls:
        c()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c()
        graphs.append(g)
    for c in calls:
        c.result.zero_()
    for g in graphs + graphs[::-1]:
        g.replay()
    torch.cuda.synchronize()
    for c, w in zip(calls, want):
        same([c.result], [w])


def test_the_same_call_gives_the_same_bits():
    b = step_buffers(7, (3, 1, 30, 2), (5000, 900, 64, 12000))
    args = (b["q"], b["kc"], b["vc"], b["table"], b["qsl"], b["ctx"])
    first = kv.kv_attention_tree(*args, max_rows=30)
    for _ in range(20):
        same([kv.kv_attention_tree(*args, max_rows=30)], [first])


def test_max_rows_beyond_the_requests_rows():
    """The bound is an upper one: a larger one changes nothing but the rounding of sums."""
    b = step_buffers(8)
    args = (b["q"], b["kc"], b["vc"], b["table"], b["qsl"], b["ctx"])
    a, c = (kv.kv_attention_tree(*args, max_rows=x).float() for x in (12, 64))
    assert (a - c).abs().max() < 2.0 ** -6
