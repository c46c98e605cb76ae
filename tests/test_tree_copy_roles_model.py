"""The tree attention's other form as a model on the CPU: blocks that are no multiple of 8 tokens, where four
warps each describe the units, copy their 32 rows of K, V and Q in groups, check their rows of V and
tell the issuer.  The issuer, the softmax warps and the checks are those of the form with tiled copies.

Checked besides: a group's rows are told of only when they have arrived, the history of the units in flight is
that of the unit told of, and the rows noted for a segment (their words are taken in turn) are cleared
before they are written, all there when the segment's output reads them, and not cleared before that.

What the models take from the kernel (rings, counts of arrivals, units in flight) is compared with its source."""
import pathlib
import random
import re

import pytest

from test_tree_roles_model import NOTES, Bar, Model, segments_of

COPIERS = 4
BAD_RING = 16
SOURCE = pathlib.Path(__file__).resolve().parent.parent / "paged_kv_cache_39_gb300" / "csrc" / "kv_attention_tree.cu"


class CopyModel(Model):
    """`lag`: units in flight beside the newest."""

    def __init__(self, rng, segments, tiles, slots, q_bufs, quarters, lag, stall=None):
        super().__init__(rng, segments, tiles, slots, q_bufs, quarters, stall)
        self.lag = lag
        self.telling, self.bad_ring = True, BAD_RING
        self.full = [Bar(COPIERS) for _ in range(slots)]
        self.note_full, self.note_free = [Bar(COPIERS) for _ in range(NOTES)], [Bar() for _ in range(NOTES)]
        self.note_parts = [[None] * COPIERS for _ in range(NOTES)]
        self.rows = [[None] * COPIERS for _ in range(slots)]       # by warp: what its rows of a slot hold
        self.q_parts = [[None] * COPIERS for _ in range(2)]
        self.bad = self.words_of_noted_rows()
        self.last_segment = self.units[-1]["seg"]

    def words_of_noted_rows(self):
        return [dict(seg=g, noted=set(), read=set()) for g in range(self.bad_ring)]

    # no barrier of Q: it comes with its segment's first unit, which is told of by its K and V
    def wait(self, bar, phase):
        if any(bar is b for b in self.q_full):
            return True
        return (yield from super().wait(bar, phase))

    def v_there(self, u, edges):
        return (yield from self.wait(self.full[(2 * u + 1) % self.slots], (2 * u + 1) // self.slots))

    def copier(self, w):
        units, lag = self.units, self.lag
        groups = []                      # of this warp, by unit: True once landed
        state = dict(told=0)
        hist = [None] * (lag + 2)

        def landed_but(newest):
            """All groups but the newest ones have arrived."""
            while not all(groups[:max(0, len(groups) - newest)]):
                yield

        def tell(back):
            u = state["told"]
            assert hist[back] == u, "the history of another unit"
            at_k, at_v = 2 * u % self.slots, (2 * u + 1) % self.slots
            assert groups[u], "told of before it is there"
            assert self.rows[at_k][w] == ("raw", u, False) and self.rows[at_v][w] == ("raw", u, True)
            if units[u]["edge"]:
                yield
                note = self.bad[units[u]["seg"] % self.bad_ring]
                assert note["seg"] == units[u]["seg"], "rows noted where another segment's are"
                note["noted"].add((u, w))
            for slot, v in ((at_k, False), (at_v, True)):
                self.rows[slot][w] = ("ready", u, v)
                if all(x == ("ready", u, v) for x in self.rows[slot]):
                    self.ring[slot] = ("ready", u, v)
            yield
            self.full[at_k].arrive()
            self.full[at_v].arrive()
            state["told"] += 1

        def wait_telling(bar, phase, so_far):
            while self.telling and state["told"] < so_far and (bar.phase & 1) == (phase & 1):
                back = so_far - 1 - state["told"]
                assert back <= lag
                yield from landed_but(back)
                yield from tell(back + 1)
            return (yield from self.wait(bar, phase))

        ok = True
        for u, x in enumerate(units):
            if (yield from self.gives_up(("copier", w), u)):
                ok = False
                break
            hist = [u] + hist[:-1]
            if u >= NOTES and not (yield from self.wait(self.note_free[u % NOTES], u // NOTES - 1)):
                ok = False
                break
            parts = self.note_parts[u % NOTES]
            self.notes[u % NOTES] = parts[w] = None
            yield
            parts[w] = u
            if w == 0 and x["first"]:
                self.seg_notes[x["seg"] % NOTES] = x["seg"]
                old = self.bad[(x["seg"] + 7) % self.bad_ring]
                if old["seg"] != x["seg"] + 7:
                    assert old["seg"] == x["seg"] + 7 - self.bad_ring
                    assert len(old["read"]) == self.readers(old["seg"]), "cleared before it is read"
                assert old["seg"] != x["seg"] + 7 or not old["noted"]
                self.bad[(x["seg"] + 7) % self.bad_ring] = dict(seg=x["seg"] + 7, noted=set(), read=set())
            if all(p == u for p in parts):
                self.notes[u % NOTES] = u
            self.note_full[u % NOTES].arrive()
            yield
            g, b = x["seg"], x["seg"] % self.q_bufs
            if x["first"] and g >= self.q_bufs:
                if not (yield from wait_telling(self.q_free[b], g // self.q_bufs - 1, u)):
                    ok = False
                    break
            gone = False
            for v in (False, True):
                slot, turn = (2 * u + v) % self.slots, (2 * u + v) // self.slots
                if turn and not (yield from self.wait(self.empty[slot], turn - 1)):
                    gone = True
                    break
            if gone:
                ok = False
                break
            groups.append(False)
            if x["first"]:
                self.q[b] = self.q_parts[b][w] = None
            for v in (False, True):
                slot = (2 * u + v) % self.slots
                self.rows[slot][w], self.ring[slot] = ("loading", u, v), None

            def landed(u=u, x=x, b=b):
                if x["first"]:
                    self.q_parts[b][w] = x["seg"]
                    if all(p == x["seg"] for p in self.q_parts[b]):
                        self.q[b] = x["seg"]
                for v in (False, True):
                    assert self.rows[(2 * u + v) % self.slots][w] == ("loading", u, v)
                    self.rows[(2 * u + v) % self.slots][w] = ("raw", u, v)
                groups[u] = True
            self.copies.append(landed)
            yield
            if u - state["told"] >= lag:
                yield from landed_but(lag)
                yield from tell(u - state["told"])
        yield from landed_but(0)
        while ok and state["told"] < len(units):
            yield from tell(len(units) - 1 - state["told"])
        yield from self.meet_all()

    def readers(self, seg):
        two = any(x["two"] for x in self.units if x["seg"] == seg)
        return self.quarters * (2 if self.tiles == 1 else 4 if two else 2)

    def took_out(self, seg, who):
        """A softmax warp's output: it reads what was noted."""
        note = self.bad[seg % self.bad_ring]
        assert note["seg"] == seg, "noted rows that were cleared"
        want = {(u, w) for u, x in enumerate(self.units) if x["seg"] == seg and x["edge"] for w in range(COPIERS)}
        assert note["noted"] == want, "noted rows that are not there yet"
        note["read"].add(who)

    def softmax(self, t, half, quarter):
        out, mine = self.out, (t, half, quarter)
        seen = set()
        for step in super().softmax(t, half, quarter):
            for seg in range(self.last_segment + 1):
                if seg not in seen and (half, quarter) in out.get((seg, t), ()):
                    seen.add(seg)
                    self.took_out(seg, mine)
            yield step
        for seg in range(self.last_segment + 1):
            if seg not in seen and (half, quarter) in out.get((seg, t), ()):
                self.took_out(seg, mine)

    def every_role(self):
        return [self.copier(w) for w in range(COPIERS)] + [self.issuer()]

    def run(self):
        """As Model.run, with these roles."""
        rng = self.rng
        self.rises = [rng.random() < 0.3 for _ in self.units]
        roles = self.every_role()
        roles += [self.softmax(t, h, q) for t in range(self.tiles) for h in range(2) for q in range(self.quarters)]
        self.roles = len(roles)
        weight = [rng.choice([0.05, 0.3, 1, 1, 3]) for _ in roles] + [rng.choice([0.05, 0.3, 1, 3]) for _ in range(2)]
        live = set(range(len(roles)))
        steps = 0
        while live:
            steps += 1
            assert steps < 400000, "does not end"
            k = rng.choices(range(len(weight)), weight)[0]
            if k == len(roles):
                if self.copies:
                    self.copies.pop(rng.randrange(len(self.copies)))()
            elif k == len(roles) + 1:
                for _ in range(rng.randint(1, 4)):
                    if self.queue:
                        self.queue.pop(0)()
            elif k in live:
                try:
                    next(roles[k])
                except StopIteration:
                    live.remove(k)
        assert not self.copies and not self.queue, "in flight when the CTA ends"


FORMS = [(1, 5, 2, 1), (1, 6, 2, 1), (1, 12, 2, 3), (2, 5, 1, 1), (2, 10, 2, 3)]  # tiles, slots, Q buffers, lag


def many_segments(rng, tiles):
    """Also: more segments of one unit than there are words for noted rows."""
    if rng.random() < 0.7:
        return segments_of(rng, tiles)
    return [(1, tiles == 2 and rng.random() < 0.5, {0} if rng.random() < 0.8 else set()) for _ in range(rng.randint(17, 40))]


@pytest.mark.parametrize("tiles,slots,q_bufs,lag", FORMS)
@pytest.mark.parametrize("seed", range(24))
def test_every_schedule_ends_and_reads_what_is_there(tiles, slots, q_bufs, lag, seed):
    rng = random.Random(3000 * seed + 10 * slots + tiles)
    m = CopyModel(rng, many_segments(rng, tiles), tiles, slots, q_bufs, rng.choice([1, 2]), lag)
    m.run()
    assert not m.abort
    warps = {(h, q) for h in range(2) for q in range(m.quarters)}
    for x in m.units:
        for t in range(tiles):
            if t == 0 or x["two"]:
                assert m.out[x["seg"], t] == warps


@pytest.mark.parametrize("tiles,slots,q_bufs,lag", FORMS)
@pytest.mark.parametrize("seed", range(24))
def test_ends_where_a_role_gives_up(tiles, slots, q_bufs, lag, seed):
    rng = random.Random(9000 * seed + 10 * slots + tiles)
    segments = many_segments(rng, tiles)
    roles = [("copier", w) for w in range(COPIERS)] + ["issuer"] + [("softmax", t, h, 0) for t in range(tiles) for h in range(2)]
    m = CopyModel(rng, segments, tiles, slots, q_bufs, 1, lag,
                  stall=(rng.choice(roles), rng.randrange(sum(n for n, *_ in segments))))
    m.run()


def failures(segments, form, change, text):
    tiles, slots, q_bufs, lag = form
    out = 0
    for seed in range(5):
        m = CopyModel(random.Random(seed), segments, tiles, slots, q_bufs, 1, lag)
        m.__dict__.update(change)
        m.bad = m.words_of_noted_rows()
        try:
            m.run()
        except AssertionError as e:
            assert text in str(e)
            out += 1
    return out


@pytest.mark.parametrize("segments,form,change,text", [
    ([(2, True, {1})] * 3, (2, 5, 1, 1), dict(telling=False), "does not end"),
    ([(1, False, {0})] * 30, (1, 12, 2, 3), dict(bad_ring=8), "cleared before it is read"),
])
def test_the_model_sees_a_planted_mistake(segments, form, change, text):
    """A wait for Q's place that keeps units in flight to itself; words for half as many segments."""
    assert failures(segments, form, {}, text) == 0
    assert failures(segments, form, change, text) > 0


def constant(name, text):
    return int(re.search(rf"constexpr int (?:\w+ = [^;]*, )?{name} = (\d+)", text)[1])


def test_the_models_are_the_kernels():
    text = SOURCE.read_text()
    assert constant("kNotes", text) == NOTES and constant("kBadRing", text) == BAD_RING
    assert constant("kCopiers", text) == COPIERS and constant("kReaders", text) == 4
    m = Model(random.Random(0), [(1, False, set())], 1, 5, 2, 1)
    c = CopyModel(random.Random(0), [(1, False, set())], 1, 5, 2, 1, 1)
    assert m.note_free[0].count == 1 + 4 and c.note_free[0].count == 1
    for line in ("if (b < empty) count = kTma ? 1 : kCopiers;",
                 "if (b >= note_full && b < note_free) count = kTma ? 1 : kCopiers;",
                 "if (b >= note_free && b < s_full) count = 1 + (kTma ? kReaders : 0);",
                 "if (b >= p_full && b < o_full) count = a.warps;",
                 "if (b >= o_free && b < q_free) count = kHalves * a.warps;",
                 "if (b >= pairs) count = 2;",
                 "constexpr int kLag = DP == 128 ? 1 : 3;",
                 "bad[(segment + 7) & (kBadRing - 1)] = 0;"):
        assert line in text, line
    # rings and buffers of every size of call
    smem, head = constant("kSmemMax", text), 3 << 10
    assert "constexpr int kHead = 3 << 10;" in text
    forms = set()
    for dp in (64, 128):
        for rows in range(1, 513):
            tiles = 2 if rows > 128 else 1
            q = -(-(-(-min(rows, 128) // 8) * 8 * dp * 2 * tiles) // 1024) * 1024
            slot = 128 * dp * 2
            bufs = 2 if head + 2 * q + (10 if dp == 64 else 5) * slot <= smem else 1
            forms.add((tiles, min(12, (smem - head - bufs * q) // slot), bufs, 1 if dp == 128 else 3))
    assert forms == set(FORMS)
