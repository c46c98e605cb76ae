"""Host-visible refusals of the operators of a step with drafted rows: none of these calls reaches
the GPU (pointers are plain numbers the library must not follow)."""
import pytest

from test_operators_abi import A, N, lib  # noqa: F401

LAYOUT = dict(parents=A[0], qs=A[1], ctx=A[2], reqs=2, rows=8, mask=A[3], pos=A[4], place=A[5], err=N, stream=N)


@pytest.mark.parametrize("want,change", [
    (-1, dict(reqs=-1)), (-1, dict(rows=-1)), (-2, dict(reqs=4097)), (-2, dict(rows=64 * 4096 + 1)),
    (-1, dict(qs=N)), (-1, dict(ctx=N)), (-1, dict(mask=N)), (-1, dict(pos=N)), (-1, dict(place=N)),
    (-1, dict(parents=A[0] + 2)), (-1, dict(qs=A[1] + 2)), (-1, dict(ctx=A[2] + 1)), (-1, dict(mask=A[3] + 4)),
    (-1, dict(pos=A[4] + 4)), (-1, dict(place=A[5] + 4)), (-1, dict(err=A[6] + 2)),
    (-1, dict(mask=A[0])), (-1, dict(pos=A[1])), (-1, dict(place=A[2])), (-1, dict(pos=A[3])),
    (-1, dict(place=A[3] + 56)), (-1, dict(place=A[4] - 56)), (-1, dict(mask=A[0] + 24)),
    (0, dict(reqs=0)), (0, dict(rows=0)),
])
def test_layout_refuses(lib, want, change):  # noqa: F811
    assert lib.kv_tree_layout(*{**LAYOUT, **change}.values()) == want


TREE = dict(query=A[0], qstride=32 * 128, kc=A[1], vc=A[2], layer=0, layers=1, blocks=8, t=16, hq=32, h=8, d=128,
            table=A[3], stride=4, qs=A[4], start=A[5], ctx=A[6], mask=A[7], reqs=2, rows=8, most=8, scale=0.1,
            out=A[8], ws=A[9], ws_bytes=1 << 27, err=N, stream=N)
ROW = 32 * 128 * 2


@pytest.mark.parametrize("want,change", [
    (-1, dict(layer=1)), (-1, dict(layer=-1)), (-1, dict(layers=0)), (-1, dict(blocks=0)), (-1, dict(t=0)),
    (-1, dict(hq=0)), (-1, dict(h=0)), (-1, dict(d=0)), (-1, dict(hq=30)), (-1, dict(stride=-1)),
    (-1, dict(reqs=-1)), (-1, dict(rows=-1)), (-1, dict(most=0)), (-1, dict(most=65)),
    (-1, dict(scale=0.0)), (-1, dict(scale=-1.0)), (-1, dict(scale=float("inf"))), (-1, dict(scale=float("nan"))),
    (-1, dict(ws_bytes=-1)), (-2, dict(reqs=4097)), (-2, dict(rows=64 * 4096 + 1)), (-2, dict(d=132, qstride=32 * 136)),
    (-2, dict(d=136, qstride=32 * 136)), (-2, dict(hq=65, h=1, qstride=65 * 128)),
    (-2, dict(hq=4104, h=1026, qstride=4104 * 128)),
    (-1, dict(qstride=128)), (-2, dict(qstride=32 * 128 + 4)),
    (-1, dict(query=N)), (-1, dict(kc=N)), (-1, dict(vc=N)), (-1, dict(table=N)), (-1, dict(qs=N)), (-1, dict(ctx=N)),
    (-1, dict(out=N)), (-1, dict(query=A[0] + 8)), (-1, dict(kc=A[1] + 8)), (-1, dict(vc=A[2] + 8)),
    (-1, dict(table=A[3] + 2)), (-1, dict(qs=A[4] + 2)), (-1, dict(start=A[5] + 2)), (-1, dict(ctx=A[6] + 2)),
    (-1, dict(mask=A[7] + 4)), (-1, dict(out=A[8] + 8)), (-1, dict(err=A[10] + 2)),
    (-1, dict(out=A[0])), (-1, dict(out=A[1] + 16)), (-1, dict(out=A[2])), (-1, dict(out=A[3])), (-1, dict(out=A[4])),
    (-1, dict(out=A[5])), (-1, dict(out=A[6])), (-1, dict(out=A[7])), (-1, dict(out=A[7] - 8 * ROW + 16)),
    (0, dict(reqs=0)), (0, dict(rows=0)),
])
def test_attention_refuses(lib, want, change):  # noqa: F811
    assert lib.kv_attention_tree(*{**TREE, **change}.values()) == want


def test_attention_workspace(lib):  # noqa: F811
    for want, args in ((-1, (-1, 8, 32, 8, 128)), (-1, (2, 0, 32, 8, 128)), (-1, (2, 65, 32, 8, 128)),
                       (-1, (2, 8, 30, 8, 128)), (-1, (2, 8, 32, 0, 128)), (-1, (2, 8, 32, 8, 0)),
                       (-2, (4097, 8, 32, 8, 128)), (-2, (2, 8, 65, 1, 128)), (-2, (2, 8, 32, 8, 12)),
                       (-2, (2, 8, 32, 8, 136))):
        assert lib.kv_attention_tree_workspace(*args) == want
    assert lib.kv_attention_tree_workspace(0, 1, 32, 8, 128) >= 0
    need = lib.kv_attention_tree_workspace(2, 8, 32, 8, 128)
    assert 0 <= need <= 1 << 27
    if need > 0:
        for change in (dict(ws_bytes=need - 1), dict(ws=N), dict(ws=A[9] + 8), dict(ws=A[0]), dict(ws=A[1]),
                       dict(ws=A[7]), dict(ws=A[8] - need + 16), dict(out=A[9] + need - need % 16 - 16)):
            assert lib.kv_attention_tree(*{**TREE, **change}.values()) == -1


VERIFY = dict(target=A[0], ts=100, draft=A[1], ds=100, kind=0, vocab=100, tokens=A[2], parents=A[3], qs=A[4], u=A[5],
              reqs=2, rows=8, out=A[6], path=A[7], kept=A[8], err=N, stream=N)


@pytest.mark.parametrize("want,change", [
    (-1, dict(reqs=-1)), (-1, dict(rows=-1)), (-2, dict(reqs=4097)), (-2, dict(rows=64 * 4096 + 1)),
    (-1, dict(vocab=0)), (-2, dict(vocab=2 ** 20 + 1, ts=2 ** 21, ds=2 ** 21)), (-1, dict(kind=2)), (-1, dict(kind=-1)),
    (-1, dict(ts=99)), (-1, dict(ds=99)), (-1, dict(target=N)), (-1, dict(tokens=N)), (-1, dict(qs=N)),
    (-1, dict(u=N)), (-1, dict(out=N)), (-1, dict(path=N)), (-1, dict(kept=N)), (-1, dict(target=A[0] + 2)),
    (-1, dict(target=A[0] + 1, kind=1)), (-1, dict(draft=A[1] + 2)), (-1, dict(tokens=A[2] + 2)),
    (-1, dict(parents=A[3] + 2)), (-1, dict(qs=A[4] + 2)), (-1, dict(u=A[5] + 2)), (-1, dict(out=A[6] + 2)),
    (-1, dict(path=A[7] + 2)), (-1, dict(kept=A[8] + 2)), (-1, dict(err=A[9] + 2)),
    (-1, dict(out=A[0])), (-1, dict(out=A[1] + 3100)), (-1, dict(path=A[2])), (-1, dict(path=A[3] + 28)),
    (-1, dict(kept=A[4])), (-1, dict(kept=A[5])), (-1, dict(path=A[6])), (-1, dict(kept=A[7] + 4)),
    (-1, dict(kept=A[6])), (0, dict(reqs=0)),
])
def test_verify_refuses(lib, want, change):  # noqa: F811
    assert lib.kv_verify_drafts(*{**VERIFY, **change}.values()) == want


KEEP = dict(kc=A[0], vc=A[1], layers=2, blocks=8, t=16, h=8, d=128, table=A[2], stride=4, qs=A[3], ctx=A[4], path=A[5],
            kept=A[6], reqs=2, rows=8, err=N, stream=N)
CACHE = 2 * 8 * 16 * 8 * 128 * 2


@pytest.mark.parametrize("want,change", [
    (-1, dict(reqs=-1)), (-1, dict(rows=-1)), (-2, dict(reqs=4097)), (-2, dict(rows=64 * 4096 + 1)),
    (-1, dict(layers=0)), (-1, dict(blocks=0)), (-1, dict(t=0)), (-1, dict(h=0)), (-1, dict(d=0)),
    (-1, dict(stride=-1)), (-2, dict(h=1, d=12)), (-1, dict(kc=N)), (-1, dict(vc=N)), (-1, dict(table=N)),
    (-1, dict(qs=N)), (-1, dict(ctx=N)), (-1, dict(path=N)), (-1, dict(kept=N)), (-1, dict(kc=A[0] + 8)),
    (-1, dict(vc=A[1] + 8)), (-1, dict(table=A[2] + 2)), (-1, dict(qs=A[3] + 2)), (-1, dict(ctx=A[4] + 2)),
    (-1, dict(path=A[5] + 2)), (-1, dict(kept=A[6] + 2)), (-1, dict(err=A[7] + 2)), (-1, dict(vc=A[0])),
    (-1, dict(vc=A[0] + CACHE - 16)), (-1, dict(table=A[0] + 64)), (-1, dict(path=A[1] + CACHE - 4)),
    (-1, dict(kept=A[0])), (-1, dict(ctx=A[1])), (-1, dict(qs=A[1] - 8)), (-1, dict(err=A[0] + 4)),
    (0, dict(reqs=0)), (0, dict(rows=0)),
])
def test_keep_refuses(lib, want, change):  # noqa: F811
    assert lib.kv_cache_keep_path(*{**KEEP, **change}.values()) == want


def test_binding_refuses():
    import torch
    import paged_kv_cache_39_gb300 as kv
    i, f = torch.zeros(4, dtype=torch.int32), torch.zeros((4, 8))
    b = torch.zeros((4, 8, 64), dtype=torch.bfloat16)
    for call in (lambda: kv.kv_tree_layout(i, i, i), lambda: kv.kv_verify_drafts(f, i, i, f[:, 0]),
                 lambda: kv.kv_attention_tree(b, b, b, i, i, i, 4), lambda: kv.kv_cache_keep_path(b, b, i, i, i, i, i)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    assert kv.MAX_TREE_ROWS == 64
    assert {kv.ERR_BITS[x] for x in ("BAD_TREE", "BAD_TOKEN", "BAD_PROBS")} == {256, 512, 1024}
