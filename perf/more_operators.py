"""Cases of speculative decoding over the paged KV cache: what is measured, the operators'
plain forms in elementary torch, and their definition in 64 bits.

A step of a request is a tree of rows: row 0 is its last token, every other row a drafted
token with a parent row before it (a chain: each row's parent is the row before).  The
four paths are the step's parts in their order:
  layout  from the rows' parents: the rows that each row sees, its position for the
          rotation (context + depth) and its place in the cache (context + index)
  tree    attention of the rows over the bf16 paged cache: the whole context and, of the
          step's own rows, those of the row's mask (one row a request: a decode step)
  verify  from the target's and the draft's probabilities and given random numbers: the
          drafted tokens that are kept, and one more token
  keep    the kept rows' K and V moved to consecutive positions, in every layer

Verification.  At a row with target probabilities p and draft probabilities q its children
are tried in order.  With s_0 = p, Z_0 = 1: child c with token x and number u is kept when
u q(x) Z_j < s_j(x), else s_(j+1) = max(s_j - Z_j q, 0) and Z_(j+1) = sum s_(j+1).  Without
draft probabilities q is 1 at x, and Z_(j+1) = Z_j - s_j(x).  A kept child is the next row; when no child
is left, the last token is the first i with sum_(k <= i) s(k) > u_0 sum s, u_0 being row
0's number (s = p again where the sum is 0).
"""
import math
import random

import numpy as np
import torch

own = False

BF16 = torch.bfloat16
MOST = 64          # rows of a step


# ---------------------------------------------------------------------------
# Cases


def listed():
    return [
        # the trees of one request: latency
        dict(name="layout_one", op="layout", requests=1, m_lo=8, m_hi=8, shape=1),
        # a batch with trees of every size
        dict(name="layout_batch", op="layout", requests=256, m_lo=1, m_hi=64, shape=2),
        # one request with a small tree behind a short context: latency
        dict(name="tree_one", op="tree", requests=1, m_lo=8, m_hi=8, ctx_lo=1001, ctx_hi=1001, q_heads=32,
             kv_heads=8, head_dim=128, block_size=16, masked=True, shape=3),
        # the decode batch, one token each, no draft: 256 requests with contexts of 512 to 4096
        dict(name="tree_decode", op="tree", requests=256, m_lo=1, m_hi=1, ctx_lo=511, ctx_hi=4095, q_heads=32,
             kv_heads=8, head_dim=128, block_size=16, masked=False, shape=4),
        # 64 requests with trees of 2 to 25 rows
        dict(name="tree_batch", op="tree", requests=64, m_lo=2, m_hi=25, ctx_lo=512, ctx_hi=4096, q_heads=32,
             kv_heads=8, head_dim=128, block_size=16, masked=True, shape=5),
        # eight contexts of 131072 tokens, trees of 16
        dict(name="tree_long", op="tree", requests=8, m_lo=16, m_hi=16, ctx_lo=131072, ctx_hi=131072, q_heads=32,
             kv_heads=8, head_dim=128, block_size=16, masked=True, shape=6),
        # the largest trees, small heads, larger blocks
        dict(name="tree_wide", op="tree", requests=16, m_lo=57, m_hi=64, ctx_lo=1000, ctx_hi=8192, q_heads=40,
             kv_heads=5, head_dim=64, block_size=32, masked=True, shape=7),
        # one request's chain of 5 drafts: latency
        dict(name="verify_one", op="verify", requests=1, m_lo=6, m_hi=6, vocab=32000, chain=True, drafted=True,
             dtype="float32", shape=8),
        # the decode batch with chains of up to 5 drafts
        dict(name="verify_chain", op="verify", requests=256, m_lo=2, m_hi=6, vocab=131072, chain=True, drafted=True,
             dtype="float32", shape=9),
        # trees with several children a row, bf16 probabilities, an odd vocabulary
        dict(name="verify_tree", op="verify", requests=64, m_lo=5, m_hi=25, vocab=100003, chain=False, drafted=True,
             dtype="bfloat16", shape=10),
        # one request's kept rows, few layers: latency
        dict(name="keep_one", op="keep", requests=1, m_lo=12, m_hi=12, ctx_lo=70, ctx_hi=70, layers=4, kv_heads=8,
             head_dim=128, block_size=16, shape=11),
        # half the decode batch over 32 layers.  Only the blocks at a context's end take part: the contexts
        # are cut to those
        dict(name="keep_batch", op="keep", requests=128, m_lo=2, m_hi=25, ctx_lo=1, ctx_hi=16, layers=32, kv_heads=8,
             head_dim=128, block_size=16, shape=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["layout", "tree", "tree", "verify", "keep"])
    shape = rng.randrange(1 << 30)
    m_hi = _log(rng, 1, MOST)
    m_lo = rng.choice([1, m_hi, max(1, m_hi // 4)])
    if op == "layout":
        return dict(op=op, requests=_log(rng, 1, 256), m_lo=m_lo, m_hi=m_hi, shape=shape)
    heads = dict(kv_heads=rng.choice([1, 2, 4, 5, 8]), head_dim=rng.choice([64, 80, 128, 128]),
                 block_size=rng.choice([8, 16, 16, 20, 32, 48]))
    if op == "tree":
        # tokens of all contexts together, at most eight of 131072 with trees of 16 (or the like)
        total = min(_log(rng, 64, 1 << 20), (1 << 24) // m_hi)
        requests = max(min(_log(rng, 1, 256), total // 8), -(-total // 131072))
        top = total // requests
        return dict(op=op, requests=requests, m_lo=m_lo, m_hi=m_hi, ctx_lo=top // rng.choice([1, 2, 8]), ctx_hi=top,
                    q_heads=heads["kv_heads"] * rng.choice([1, 2, 3, 4, 6, 8] if top * requests * m_hi < 1 << 22
                                                           else [1, 2, 3, 4]),
                    masked=rng.random() < 0.7, shape=shape, **heads)
    if op == "verify":
        vocab = _log(rng, 100, 131072)
        rows = (1 << 27) // vocab
        requests = min(_log(rng, 1, 256), max(1, rows // m_hi))
        return dict(op=op, requests=requests, m_lo=m_lo, m_hi=m_hi, vocab=vocab, chain=rng.random() < 0.4,
                    drafted=rng.random() < 0.7, dtype=rng.choice(["float32", "bfloat16"]), shape=shape)
    ctx = _log(rng, 1, 100)
    return dict(op=op, requests=_log(rng, 1, 128), m_lo=min(m_lo, 25), m_hi=min(m_hi, 25), ctx_lo=ctx // 2,
                ctx_hi=ctx, layers=_log(rng, 1, 16), shape=shape, **heads)


def _sizes(case):
    """(rows, context) of every request and the rows' parents in their request (-1: row 0)."""
    rng = random.Random(case["shape"])
    n = case["requests"]
    rows = [rng.randint(case["m_lo"], case["m_hi"]) for _ in range(n)]
    ctx = [rng.randint(case.get("ctx_lo", 100), case.get("ctx_hi", 4096)) for _ in range(n)]
    if case.get("chain") or not case.get("masked", True):
        return rows, ctx, [list(range(-1, m - 1)) for m in rows]
    # a row hangs on one of the four before it: trees of some width and some depth
    return rows, ctx, [[-1] + [rng.randint(max(0, i - 4), i - 1) for i in range(1, m)] for m in rows]


def _ancestors(parents):
    """Bit j of entry i: row j is row i or above it."""
    mask = []
    for i, p in enumerate(parents):
        mask.append(1 << i | (mask[p] if p >= 0 else 0))
    return mask


def work(case):
    rows, ctx, parents = _sizes(case)
    n, r = sum(rows), case["requests"]
    if case["op"] == "layout":
        return {"bytes": n * (4 + 24) + 8 * r + 4, "flops": n}
    if case["op"] == "tree":
        d, h, hq = case["head_dim"], case["kv_heads"], case["q_heads"]
        pairs = sum(m * c + sum(bin(x).count("1") for x in _ancestors(p)) for m, c, p in zip(rows, ctx, parents))
        keys = n + sum(ctx)
        return {"bytes": 4 * keys * h * d + 4 * n * hq * d + 4 * keys // case["block_size"] + 8 * n + 8 * r,
                "flops": 4 * d * hq * pairs}
    if case["op"] == "verify":
        # one whole row of the target's probabilities a request and, where a draft was refused, one of the
        # draft's: with these inputs about half of the requests that have drafts and draft probabilities
        size = 4 if case["dtype"] == "float32" else 2
        half = 0.5 * sum(m > 1 for m in rows) if case["drafted"] else 0
        return {"bytes": int(size * case["vocab"] * (r + half)) + n * (4 + 4 + 4 + 4 + 4 + 2 * size) + 8 * r,
                "flops": int(2 * case["vocab"] * (r + half))}
    moved = sum(i != j for _, path in _paths(case) for i, j in enumerate(path))
    row = case["kv_heads"] * case["head_dim"] * 2
    return {"bytes": moved * 4 * row * case["layers"] + 4 * n + 12 * r, "flops": 0}


def _paths(case):
    """(rows, kept rows) of every request: the way down to a row of its tree."""
    rng = random.Random(case["shape"] + 1)
    out = []
    for m, _, parents in zip(*_sizes(case)):
        path, at = [], rng.randrange(m)
        while at >= 0:
            path.insert(0, at)
            at = parents[at]
        out.append((m, path))
    return out


# ---------------------------------------------------------------------------
# Inputs


def _table(lengths, block_size, np_rng):
    """A block table of permuted blocks (block 0 is never given out), and the pool's size."""
    counts = np.asarray([-(-n // block_size) for n in lengths])
    pool = int(counts.sum()) + 1 + len(lengths) // 4
    order = np_rng.permutation(np.arange(1, pool))[:counts.sum()]
    table = np.zeros((len(lengths), counts.max()), np.int32)
    table[np.arange(counts.max()) < counts[:, None]] = order
    return table, pool


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    np_rng = np.random.default_rng(seed)
    rows, ctx, parents = _sizes(case)
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(dev)  # noqa: E731

    def normal(shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=BF16)

    starts = np.concatenate([[0], np.cumsum(rows)])
    flat = np.concatenate(parents)
    s = dict(case=case, q_start=i32(starts), context=i32(ctx), parents=i32(flat))
    # where the plain forms look, too: request and index of every row
    req = np.repeat(np.arange(len(rows)), rows)
    s["req"] = torch.from_numpy(req).to(dev)
    s["index"] = torch.from_numpy(np.arange(sum(rows)) - starts[req]).to(dev)
    if case["op"] == "layout":
        # contexts of this seed's own
        s["context"] = i32(np_rng.integers(0, 32768, len(rows)))
    elif case["op"] == "verify":
        v, n = case["vocab"], sum(rows)
        t = getattr(torch, case["dtype"])
        logits = 4 * torch.randn((n, v), generator=gen, device=dev)
        s["target"] = torch.softmax(logits, 1).to(t)
        # the draft follows the target at a distance
        draft = torch.softmax(logits + torch.randn((n, v), generator=gen, device=dev), 1).to(t)
        # every row's token is drawn from its parent's draft probabilities, row 0's is any
        race = torch.rand((n, v), generator=gen, device=dev).log_().neg_()
        above = torch.from_numpy(np.maximum(flat, 0) + starts[req]).to(dev)
        s["tokens"] = (draft[above].float() / race).argmax(1).to(torch.int32)
        s["draft"] = draft if case["drafted"] else None
        s["uniform"] = torch.rand(n, generator=gen, device=dev)
        del logits, race
    else:
        h, d, t = case["kv_heads"], case["head_dim"], case["block_size"]
        table, pool = _table([a + b for a, b in zip(rows, ctx)], t, np_rng)
        s["table"] = i32(table)
        s["k_cache"] = normal((case.get("layers", 1), pool, t, h, d))
        s["v_cache"] = normal((case.get("layers", 1), pool, t, h, d))
        if case["op"] == "tree":
            s["query"] = normal((sum(rows), case["q_heads"], d))
            masks = np.asarray([x for p in parents for x in _ancestors(p)], np.uint64).view(np.int64)
            s["mask"] = torch.from_numpy(masks).to(dev) if case["masked"] else None
        else:
            paths = _paths(case)
            s["kept"] = i32([len(p) - 1 for _, p in paths])
            s["path"] = i32([j for m, p in paths for j in p + [-1] * (m - len(p))])
    if own:
        _handle(s)
    return s


def _handle(s):
    """The prepared call a serving loop keeps for its persistent buffers."""
    import paged_kv_cache_39_gb300 as kv
    c = s["case"]
    if c["op"] == "layout":
        s["call"] = kv.kv_tree_layout(s["parents"], s["q_start"], s["context"], prepare=True)
    elif c["op"] == "tree":
        s["call"] = kv.kv_attention_tree(s["query"], s["k_cache"], s["v_cache"], s["table"], s["q_start"],
                                         s["context"], max_rows=c["m_hi"], tree_mask=s["mask"], prepare=True)
    elif c["op"] == "verify":
        s["call"] = kv.kv_verify_drafts(s["target"], s["tokens"], s["q_start"], s["uniform"], s["draft"],
                                        None if c["chain"] else s["parents"], prepare=True)
    else:
        s["call"] = kv.kv_cache_keep_path(s["k_cache"], s["v_cache"], s["table"], s["q_start"], s["context"],
                                          s["path"], s["kept"], prepare=True)


# ---------------------------------------------------------------------------
# One pass


def run(s):
    op = s["case"]["op"]
    if own:
        out = s["call"]()
        return (s["k_cache"], s["v_cache"]) if op == "keep" else out
    if op == "verify":
        return _verify_chain(s) if s["case"]["chain"] else _verify_tree(s)
    return {"layout": _layout, "tree": _tree, "keep": _keep}[op](s)


def _by_request(s, x, fill):
    """Rows [N, ...] as [requests, most rows of one, ...]."""
    out = torch.full((s["case"]["requests"], s["case"]["m_hi"], *x.shape[1:]), fill, dtype=x.dtype, device=x.device)
    out[s["req"], s["index"]] = x
    return out


def _layout(s):
    ctx = s["context"].long()[s["req"]]
    parent = _by_request(s, s["parents"].long(), -1)
    n = parent.shape[1]
    above = (parent[:, :, None] == torch.arange(n, device=parent.device)).float()
    above = above + torch.eye(n, device=parent.device)
    above = (above @ above > 0).float()       # 2 rows up, 4, 8, 16, 32, 64
    above = (above @ above > 0).float()
    above = (above @ above > 0).float()
    above = (above @ above > 0).float()
    above = (above @ above > 0).float()
    above = (above @ above > 0).long()[s["req"], s["index"]]
    mask = (above << torch.arange(n, device=parent.device)).sum(1)
    return mask, ctx + above.sum(1) - 1, ctx + s["index"]


def _softmax(x):
    p = torch.exp(x - x.amax(-1, keepdim=True))
    return p / p.sum(-1, keepdim=True)


def _tree(s):
    c = s["case"]
    h, d, m = c["kv_heads"], c["head_dim"], c["m_hi"]
    at = s["table"].long()
    n = at.shape[1] * c["block_size"]

    def rows(cache):
        return cache[0][at].float().flatten(1, 2).transpose(1, 2)             # [r, h, n, d]

    q = _by_request(s, s["query"].float(), 0.0).unflatten(2, (h, -1))         # [r, m, h, group, d]
    q = q.permute(0, 2, 3, 1, 4).flatten(2, 3)                                # [r, h, group m, d]
    x = (q @ rows(s["k_cache"]).transpose(-1, -2) * d ** -0.5).unflatten(2, (-1, m))
    ahead = torch.arange(n, device=x.device) - s["context"].long()[:, None]   # a key's row of the step
    if s["mask"] is None:
        seen = ahead[:, None] <= torch.arange(m, device=x.device)[:, None]
    else:
        seen = (_by_request(s, s["mask"], 0)[:, :, None] >> ahead[:, None].clamp(0, 63)) & 1 == 1
        seen = (seen | (ahead < 0)[:, None]) & (ahead < m)[:, None]
    x = x.masked_fill_(~seen[:, None, None], -math.inf)
    o = _softmax(x).flatten(2, 3) @ rows(s["v_cache"])
    return o.unflatten(2, (-1, m)).permute(0, 3, 1, 2, 4).flatten(2, 3)[s["req"], s["index"]].to(BF16)


def _pick(weights, u):
    """The first index whose running sum passes u times the whole; sums in 64 bits."""
    run = weights.cumsum(1)
    return (run > u[:, None].double() * run[:, -1:]).int().argmax(1)


def _one_hot(tokens, like):
    return (tokens[:, None] == torch.arange(like.shape[1], device=like.device)).to(like.dtype)


def _answer(s, path, kept, last):
    """Outputs of a way `path` [requests, rows] down the tree and the token behind it."""
    i, kept_of = s["index"], kept[s["req"]]
    path = torch.where(i <= kept_of, path[s["req"], i], -1)
    base = s["q_start"].long()[:-1][s["req"]]
    step = path.roll(-1)                     # the row that follows on the way
    token = s["tokens"][(base + step).clamp(0, len(i) - 1)]
    token = torch.where(i < kept_of, token, torch.where(i == kept_of, last[s["req"]].int(), -1))
    return token.int(), path.int(), kept.int()


def _verify_chain(s):
    target, draft = s["target"], s["draft"]
    first = s["q_start"].long()[:-1]
    count = s["q_start"].long()[1:] - first
    n = target.shape[0]
    row = torch.arange(n, device=target.device)
    above = (row - 1).clamp_min(0)
    x = s["tokens"].long()
    p = target[above, x].double()
    q = 1.0 if draft is None else draft[above, x].double()
    ok = _by_request(s, (s["uniform"].double() * q < p).int(), 0)
    ok[:, 0] = 1
    kept = ok.cumprod(1).sum(1) - 1          # rows past the end count as refused
    at = first + kept
    weights = target[at].double()
    refused = (kept < count - 1)[:, None]
    q = _one_hot(x[(at + 1).clamp_max(n - 1)], weights) if draft is None else draft[at].double()
    left = torch.where(refused, (weights - q).clamp_min(0), weights)
    weights = torch.where(left.sum(1, keepdim=True) > 0, left, weights)
    path = torch.arange(s["case"]["m_hi"], device=x.device).expand(len(first), -1)
    return _answer(s, path, kept, _pick(weights, s["uniform"][first]))


def _verify_tree(s):
    """Rows in their order: a row counts when its parent is the row that the request stands at."""
    target, draft = s["target"], s["draft"]
    dev, r, m = target.device, s["case"]["requests"], s["case"]["m_hi"]
    first = s["q_start"].long()[:-1]
    last = s["q_start"].long()[1:] - 1
    parent = _by_request(s, s["parents"].long(), -2)
    at = torch.zeros(r, dtype=torch.long, device=dev)
    kept = torch.zeros_like(at)
    path = torch.zeros((r, m), dtype=torch.long, device=dev)
    each = torch.arange(r, device=dev)
    left = target[first].double()
    z = torch.ones(r, dtype=torch.float64, device=dev)
    for t in range(1, m):
        row = torch.minimum(first + t, last)
        tried = parent[:, t] == at
        x = s["tokens"][row].long()
        q = _one_hot(x, left) if draft is None else draft[first + at].double()
        s_x = left[each, x]
        ok = tried & (s["uniform"][row].double() * q[each, x] * z < s_x)
        no = tried & ~ok
        less = (left - z[:, None] * q).clamp_min(0)
        z = torch.where(no, (z - s_x).clamp_min(0) if draft is None else less.sum(1), torch.where(ok, 1.0, z))
        left = torch.where(no[:, None], less, torch.where(ok[:, None], target[row].double(), left))
        at = torch.where(ok, t, at)
        kept = kept + ok
        path[each, kept] = at
    whole = target[first + at].double()
    weights = torch.where(left.sum(1, keepdim=True) > 0, left, whole)
    return _answer(s, path, kept, _pick(weights, s["uniform"][first]))


def _keep(s):
    c = s["case"]
    t, ctx, i = c["block_size"], s["context"].long()[s["req"]], s["index"]
    moved = (i > 0) & (i <= s["kept"].long()[s["req"]])
    table = s["table"].long()

    def slots(row):
        return table[s["req"], (ctx + row) // t] * t + (ctx + row) % t

    src, dst = slots(torch.where(moved, s["path"].long(), i)), slots(i)
    for cache in (s["k_cache"], s["v_cache"]):
        rows = cache.flatten(1, 2)
        rows[:, dst] = rows[:, src]
    return s["k_cache"], s["v_cache"]


# ---------------------------------------------------------------------------
# The definition in 64 bits


def exact(case, seed):
    was = globals()["own"]
    globals()["own"] = False
    try:
        s = prepare(case, seed)
    finally:
        globals()["own"] = was
    f64 = torch.float64
    rows, _, parents = _sizes(case)
    begin = np.concatenate([[0], np.cumsum(rows)]).tolist()
    ctx = s["context"].tolist()
    if case["op"] == "layout":
        masks = [x for p in parents for x in _ancestors(p)]
        depth = [bin(x).count("1") - 1 for x in masks]
        context = np.repeat(ctx, rows)
        place = context + np.concatenate([np.arange(m) for m in rows])
        return (torch.from_numpy(np.asarray(masks, np.uint64).view(np.int64)), torch.from_numpy(context + depth),
                torch.from_numpy(place))
    if case["op"] == "tree":
        h, hq, d, t = case["kv_heads"], case["q_heads"], case["head_dim"], case["block_size"]
        out = torch.empty(s["query"].shape, dtype=f64, device="cuda")
        for r, (m, p) in enumerate(zip(rows, parents)):
            n = ctx[r] + m
            seen = torch.ones((m, n), dtype=torch.bool)
            seen[:, ctx[r]:] = torch.tensor([[x >> j & 1 for j in range(m)] for x in _ancestors(p)]) == 1
            seen = seen.cuda()
            blocks = s["table"][r, :-(-n // t)].long()
            k, v = (c[0, blocks].flatten(0, 1)[:n] for c in (s["k_cache"], s["v_cache"]))
            q = s["query"][begin[r]:begin[r + 1]].to(f64).unflatten(1, (h, hq // h))
            for g in range(h):
                x = q[:, g].transpose(0, 1) @ k[:, g].to(f64).T / math.sqrt(d)
                w = x.exp() * seen               # |logit| is a few: no maximum needed
                o = (w @ v[:, g].to(f64)) / w.sum(-1, keepdim=True)
                out[begin[r]:begin[r + 1], g * (hq // h):(g + 1) * (hq // h)] = o.transpose(0, 1)
        return out
    if case["op"] == "verify":
        tokens, uniform = s["tokens"].tolist(), s["uniform"].double().tolist()
        out_tokens, out_path, out_kept = [], [], []
        for r, m in enumerate(rows):
            at, way = 0, [0]
            while True:
                p = s["target"][begin[r] + at].to(f64)
                rest, whole, nxt = p, 1.0, None
                for c in (c for c in range(at + 1, m) if parents[r][c] == at):
                    x = tokens[begin[r] + c]
                    if s["draft"] is None:
                        q = torch.zeros_like(p)
                        q[x] = 1
                    else:
                        q = s["draft"][begin[r] + at].to(f64)
                    if uniform[begin[r] + c] * float(q[x]) * whole < float(rest[x]):
                        nxt = c
                        break
                    was_x = float(rest[x])
                    rest = torch.clamp(rest - whole * q, min=0)
                    whole = max(whole - was_x, 0.0) if s["draft"] is None else float(rest.sum())
                if nxt is None:
                    break
                at = nxt
                way.append(at)
            if float(rest.sum()) == 0:
                rest = p
            up = torch.cumsum(rest, 0)
            final = int(torch.searchsorted(up, uniform[begin[r]] * up[-1], right=True))
            got = [tokens[begin[r] + c] for c in way[1:]] + [final]
            out_tokens += got + [-1] * (m - len(got))
            out_path += way + [-1] * (m - len(way))
            out_kept.append(len(way) - 1)
        return tuple(torch.tensor(x, dtype=torch.int32) for x in (out_tokens, out_path, out_kept))
    t = case["block_size"]
    caches = [s["k_cache"].clone(), s["v_cache"].clone()]
    table = s["table"].tolist()
    for r, (_, path) in enumerate(_paths(case)):
        for i, j in enumerate(path):             # in order: a source is never a place filled before
            a, b = ctx[r] + j, ctx[r] + i
            if a != b:
                for x in caches:
                    x[:, table[r][b // t], b % t] = x[:, table[r][a // t], a % t]
    return tuple(caches)
