"""kv_verify_drafts against its rule in exact arithmetic."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import paged_kv_cache_39_gb300 as kv
from operator_refs import BF16, dev
from step_refs import i32, random_tree, starts, verify

pytestmark = pytest.mark.gpu
MANTISSA = {torch.float32: 24, BF16: 8}


def probabilities(n, V, dtype, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    return torch.softmax(spread * torch.randn((n, V), generator=g, dtype=torch.float64), 1).to(dtype)


def fractions(t):
    return [[Fraction(x) for x in row] for row in t.double().tolist()]


def expect(target, draft, tokens, parents, uniform, rows):
    begin = starts(rows)
    out, path, kept = [], [], []
    for r, m in enumerate(rows):
        if m == 0:
            kept.append(0)
            continue
        s = slice(begin[r], begin[r + 1])
        o, p = verify(fractions(target[s]), None if draft is None else fractions(draft[s]), tokens[s].tolist(),
                      parents[s], [Fraction(x) for x in uniform[s].double().tolist()])
        out += o + [-1] * (m - len(o))
        path += p + [-1] * (m - len(p))
        kept.append(len(p) - 1)
    return out, path, kept


def run(rows, V, dtype, drafted, seed, chain=False, stride=0, offset=0, spread=2.0, repeats=False, bits=0,
        change=None):
    """Tokens drawn from the draft, so that some are kept and some are not."""
    rng = np.random.default_rng(seed)
    n = sum(rows)
    target = probabilities(n, V, dtype, seed, spread)
    draft = probabilities(n, V, dtype, seed, spread) * 0.5 + probabilities(n, V, dtype, seed + 1, spread) * 0.5
    draft = draft.to(dtype)
    parents = [x for m in rows for x in (list(range(-1, m - 1)) if chain else random_tree(m, rng))]
    begin = np.repeat(starts(rows)[:-1], rows)
    tokens = torch.zeros(n, dtype=torch.int32)
    for t in range(n):
        p = draft[begin[t] + max(parents[t], 0)].double()
        tokens[t] = int(torch.multinomial(p, 1, generator=torch.Generator().manual_seed(seed + t)))
    if repeats:      # siblings with the same token
        tokens = tokens % 3
    uniform = torch.rand(n, generator=torch.Generator().manual_seed(seed + 7))
    if change is not None:
        change(target, draft, tokens, parents, uniform)
    want = expect(target, draft if drafted else None, tokens, parents, uniform, rows)

    def place(t):    # rows `stride` elements further apart, the first one `offset` elements in
        wide = torch.full((n * (V + stride) + offset + 8,), float("nan"), dtype=dtype, device=dev())
        view = wide[offset:offset + n * (V + stride)].view(n, V + stride)[:, :V]
        view.copy_(t)
        return view

    err = kv.new_error_word(dev())
    got = kv.kv_verify_drafts(place(target), tokens.to(dev()), i32(starts(rows)), uniform.to(dev()),
                              place(draft) if drafted else None, None if chain else i32(parents), err=err)
    for g, w, name in zip(got, want, ("tokens", "path", "kept")):
        assert g.tolist() == w, name
    assert err.item() == bits
    return got


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("chain", [True, False])
@pytest.mark.parametrize("V", [1, 2, 3, 7, 33, 250, 1001])
def test_small(V, chain, drafted, dtype):
    run([1, 2, 5, 0, 9, 17, 3, 1, 12], V, dtype, drafted, seed=V, chain=chain)


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("drafted", [True, False])
def test_larger_vocabularies(drafted, dtype):
    run([9, 4], 20011, dtype, drafted, seed=5, spread=3.0)
    run([6], 32000, dtype, drafted, seed=6, chain=True, spread=3.0)


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("stride,offset", [(0, 1), (1, 0), (3, 3), (5, 2), (8, 4), (16, 8)])
def test_strides_and_alignment(stride, offset, dtype):
    run([5, 3, 8], 517, dtype, True, seed=stride * 10 + offset, stride=stride, offset=offset)


def test_target_and_draft_of_different_alignment():
    n, V = 6, 301
    target, draft = probabilities(n, V, torch.float32, 1), probabilities(n, V, torch.float32, 2)
    tokens = torch.argmax(draft, 1).to(torch.int32).roll(1)
    uniform = torch.rand(n, generator=torch.Generator().manual_seed(3))
    want = expect(target, draft, tokens, list(range(-1, n - 1)), uniform, [n])
    wide = torch.zeros((n, V + 2), device=dev())
    wide[:, 1:-1] = draft
    got = kv.kv_verify_drafts(target.to(dev()), tokens.to(dev()), i32([0, n]), uniform.to(dev()), wide[:, 1:-1])
    assert [g.tolist() for g in got] == [want[0], want[1], want[2]]


@pytest.mark.parametrize("drafted", [True, False])
def test_wide_trees_with_many_refusals(drafted):
    """A star: up to 63 refusals at one row."""
    def star(target, draft, tokens, parents, uniform):
        for i in range(len(parents)):
            parents[i] = -1 if i in (0, 64) else 0
        uniform[1:64] = 0.999
        uniform[65:] = 0.97
    run([64, 40], 91, torch.float32, drafted, seed=8, change=star)


@pytest.mark.parametrize("drafted", [True, False])
def test_siblings_with_the_same_token(drafted):
    run([30, 12, 64], 50, torch.float32, drafted, seed=9, repeats=True)


def test_draft_equal_to_the_target_keeps_everything():
    def same(target, draft, tokens, parents, uniform):
        draft.copy_(target)
    rows = [8, 1, 5]
    got = run(rows, 100, torch.float32, True, seed=10, chain=True, change=same)
    assert got[2].tolist() == [m - 1 for m in rows]


def test_nothing_left_of_the_target():
    """p <= q everywhere and the token is refused: p again."""
    def below(target, draft, tokens, parents, uniform):
        draft.copy_(target)
        tokens[1] = 0
        draft[0, 0] = min(1.0, float(target[0, 0]) * 2)
        uniform[1] = 0.9
    got = run([2], 40, torch.float32, True, seed=11, chain=True, change=below)
    assert got[2].tolist() == [0]


def test_all_of_the_target_on_refused_tokens():
    def chosen(target, draft, tokens, parents, uniform):
        target[0] = 0
        target[0, 3], target[0, 5] = 0.25, 0.25     # refused, though nothing else has a weight
        tokens[1], tokens[2] = 3, 5
        parents[1] = parents[2] = 0
        uniform[1], uniform[2] = 0.9, 0.9
    run([3], 20, torch.float32, False, seed=12, change=chosen)


def test_rows_of_zeros():
    def zeros(target, draft, tokens, parents, uniform):
        target.zero_()
    got = run([3, 1], 20, torch.float32, True, seed=13, change=zeros, bits=kv.ERR_BITS["BAD_PROBS"])
    assert got[0].tolist() == [-1] * 4


def test_numbers_at_the_ends():
    def ends(target, draft, tokens, parents, uniform):
        uniform[0], uniform[4] = 0.0, 1 - 2.0 ** -24
        target[0, :9] = 0            # the first token with a weight
    run([4, 5], 77, torch.float32, True, seed=14, change=ends)
    # outside [0, 1): the nearest inside
    p = torch.full((1, 4), 0.25, device=dev())
    for u, want in ((-1.0, 0), (float("nan"), 0), (1.0, 3), (7.0, 3), (0.5, 2), (0.49999997, 1)):
        got = kv.kv_verify_drafts(p, i32([0]), i32([0, 1]), torch.tensor([u], device=dev()))
        assert got[0].tolist() == [want]


def test_probabilities_that_are_none():
    """Below 0 and NaN count as 0, above 1 as 1."""
    p = torch.tensor([[float("nan"), -0.5, 0.0, 2.0, float("inf"), -float("inf")]], device=dev())
    for u, want in ((0.0, 3), (0.49, 3), (0.51, 4), (0.99, 4)):
        got = kv.kv_verify_drafts(p, i32([0]), i32([0, 1]), torch.tensor([u], device=dev()))
        assert got[0].tolist() == [want]


def test_tokens_and_parents_out_of_range():
    def spoil(target, draft, tokens, parents, uniform):
        tokens[1], tokens[2] = -1, 40
        parents[4], parents[5] = 4, -3
        parents[6] = 5          # below a row that is not there
        tokens[0] = 10 ** 6     # row 0's is not read
    run([8], 40, torch.float32, True, seed=15, change=spoil, bits=kv.ERR_BITS["BAD_TOKEN"] | kv.ERR_BITS["BAD_TREE"])


def test_small_weights_count():
    """Ten thousand weights of 2^-30 against one of 2^-10: sums of 32 bits would lose them."""
    V = 10001
    p = torch.full((1, V), 2.0 ** -30, device=dev())
    p[0, 0] = 2.0 ** -10
    total = Fraction(1, 2 ** 10) + 10000 * Fraction(1, 2 ** 30)
    for k in (1, 2, 777, 5000, 9999):
        border = (Fraction(1, 2 ** 10) + k * Fraction(1, 2 ** 30)) / total      # between tokens k and k + 1
        u = np.float32(float(border))
        want = next(i for i in range(V) if Fraction(1, 2 ** 10) + i * Fraction(1, 2 ** 30) > Fraction(float(u)) * total)
        got = kv.kv_verify_drafts(p, i32([0]), i32([0, 1]), torch.tensor([u], device=dev()))
        assert got[0].tolist() == [want]


def test_many_requests_and_rows_behind_them():
    rng = np.random.default_rng(16)
    rows = [int(x) for x in rng.integers(0, 5, 333)]
    run(rows, 60, BF16, True, seed=17)
    n = 5
    p = probabilities(n, 30, torch.float32, 18).to(dev())
    outs = [torch.full((n,), -9, dtype=torch.int32, device=dev()) for _ in range(2)]
    kv.kv_verify_drafts(p, i32([1] * n), i32([0, 2]), torch.rand(n, device=dev()), out_tokens=outs[0], path=outs[1])
    assert all((o[2:] == -9).all() and (o[:1] >= 0).all() for o in outs)


def test_rows_out_of_order_out_of_range_or_too_many():
    n = 70
    p = probabilities(n, 30, torch.float32, 19).to(dev())
    for qs, kept in (([0, 3, 2, 4], 1), ([-1, 3, 4, 5], 0), ([0, 2, 4, 71], 2), ([0, 65, 66, 67], 0)):
        outs = [torch.full((n,), -9, dtype=torch.int32, device=dev()) for _ in range(2)]
        num = torch.full((3,), 5, dtype=torch.int32, device=dev())
        err = kv.new_error_word(dev())
        kv.kv_verify_drafts(p, i32([1] * n), i32(qs), torch.rand(n, device=dev()), out_tokens=outs[0], path=outs[1],
                            num_kept=num, err=err)
        assert err.item() == kv.ERR_BITS["BAD_QSL"]
        good = [r for r in range(3) if 0 <= qs[r] <= qs[r + 1] <= n and qs[r + 1] - qs[r] <= 64]
        touched = torch.zeros(n, dtype=torch.bool)
        for r in good:
            touched[qs[r]:qs[r + 1]] = True
        for o in outs:
            assert (o.cpu()[~touched] == -9).all() and (o.cpu()[touched] != -9).all()
        assert all(num[r].item() == 0 for r in range(3) if r not in good)


def test_distribution_is_the_targets():
    """40,000 requests with drafts: the first emitted token of each is distributed as the target's
    first row.  Counts are within 5 standard deviations (fixed numbers, so this does not vary)."""
    V, R = 12, 4000
    p = probabilities(1, V, torch.float32, 20, 1.0)
    q = probabilities(1, V, torch.float32, 21, 1.0)
    for parents in ([-1, 0, 1], [-1, 0, 0]):
        g = torch.Generator(device="cuda").manual_seed(22)
        counts = torch.zeros(V, dtype=torch.long)
        for _ in range(10):
            tokens = torch.multinomial(q[0].to(dev()), 3 * R, replacement=True, generator=g).to(torch.int32)
            uniform = torch.rand(3 * R, generator=g, device=dev())
            out, _, _ = kv.kv_verify_drafts(p.to(dev()).expand(3 * R, V).contiguous(), tokens,
                                            i32(np.arange(R + 1) * 3), uniform,
                                            q.to(dev()).expand(3 * R, V).contiguous(), i32(parents * R))
            counts += torch.bincount(out[::3].cpu().long(), minlength=V)
        n = 10 * R
        e = p[0].double()
        assert ((counts.double() - n * e).abs() <= 5 * (n * e * (1 - e)).sqrt()).all()


@pytest.mark.parametrize("V", [7, 600])
@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_nothing_left_before_rows_that_hang_elsewhere(dtype, V):
    """p <= q everywhere, the refused row has rows below it and none beside it: p again."""
    def larger(target, draft, tokens, parents, uniform):
        parents[:] = [-1, 0, 1, 2, -1, 0, 1, 1]
        draft[0], draft[4] = target[0] * 2, target[4] * 4     # exact in either type
        uniform[1] = uniform[5] = 0.875
        uniform[0], uniform[4] = 0.6, 0.3
    got = run([4, 4], V, dtype, True, seed=11, spread=0.5, change=larger)
    assert got[2].tolist() == [0, 0] and got[0][0].item() >= 0 and got[0][4].item() >= 0
