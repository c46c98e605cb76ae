"""The roles of a tree attention CTA as a model on the CPU: the warp that describes units, the
copies of K and V, Q's load, the check of values, the issuer and the softmax warps, with their
barriers, run under random schedules.  Checked: no barrier takes an arrival of another turn, a
wait is never passed by another phase than its own, nothing is read before it is there or
overwritten while it is still needed, every schedule ends, and nothing is in flight when the CTA
ends, also where a role gave up on the way.

A barrier is passed by the parity of its phase, as the hardware does it.  Copies complete in any
order, matrix instructions and their arrivals in issue order."""
import random

import pytest

NOTES = 8


class Bar:
    def __init__(self, count=1):
        self.count = self.pending = count
        self.bytes = self.phase = 0

    def _turn(self):
        if self.pending == 0 and self.bytes == 0:
            self.phase, self.pending = self.phase + 1, self.count

    def arrive(self, expect=0):
        assert self.pending > 0, "an arrival of another turn"
        self.pending, self.bytes = self.pending - 1, self.bytes + expect
        self._turn()

    def landed(self):
        assert self.bytes > 0
        self.bytes -= 1
        self._turn()


class Model:
    """segments: (units, second tile, units whose values are checked) of one CTA in turn."""

    def __init__(self, rng, segments, tiles, slots, q_bufs, quarters, stall=None):
        self.rng, self.tiles, self.slots, self.q_bufs, self.stall = rng, tiles, slots, q_bufs, stall
        self.units = []
        for g, (n, two, edges) in enumerate(segments):
            for i in range(n):
                self.units.append(dict(seg=g, first=i == 0, last=i == n - 1, two=two, edge=i in edges))
        self.full, self.empty = [Bar() for _ in range(slots)], [Bar() for _ in range(slots)]
        self.note_full, self.note_free = [Bar() for _ in range(NOTES)], [Bar(5) for _ in range(NOTES)]
        self.s_full, self.p_full = [Bar(), Bar()], [Bar(quarters) for _ in range(4)]
        self.o_full, self.o_free = [Bar(), Bar()], [Bar(2 * quarters) for _ in range(2)]
        self.q_free, self.q_full = [Bar(), Bar()], [Bar(), Bar()]
        self.edge, self.checked = [Bar() for _ in range(NOTES)], [Bar() for _ in range(NOTES)]
        self.pairs = {(t, q): Bar(2) for t in range(tiles) for q in range(quarters)}
        self.drain = Bar()
        self.quarters = quarters
        self.notes, self.seg_notes = [None] * NOTES, [None] * NOTES
        self.ring, self.q = [None] * slots, [None, None]
        self.s, self.p = [None, None], [set(), set()]     # unit whose logits; (unit, half, quarter) of weights
        self.o, self.o_read = [None, None], [set(), set()]  # (segment, last unit added); warps that took it out
        self.added = -1                                    # one tile: the last unit whose P V is done
        self.copies, self.queue = [], []
        self.out, self.abort, self.ended = {}, False, 0
        self.tops, self.words, self.issued = {}, {}, [0, 0]

    # every wait gives up where another role has; `phase` is the one meant
    def wait(self, bar, phase):
        while (bar.phase & 1) == (phase & 1):
            if self.abort and self.rng.random() < 0.5:
                return False
            yield
        assert bar.phase == phase + 1, f"passed by phase {bar.phase - 1} instead of {phase}"
        return True

    def gives_up(self, role, u):
        if self.stall != (role, u):
            return False
        for _ in range(self.rng.choice([0, 3, 30, 300])):
            if self.abort:
                break
            yield
        self.abort = True
        return True

    def settle(self, bar, phase):
        while (bar.phase & 1) == (phase & 1):
            yield

    def meet_all(self):
        self.ended += 1
        while self.ended < self.roles:
            yield

    def read(self, u, seg=False):
        ok = yield from self.wait(self.note_full[u % NOTES], u // NOTES)
        if not ok:
            return None
        yield
        assert self.notes[u % NOTES] == u
        x = self.units[u]
        if seg:
            assert self.seg_notes[x["seg"] % NOTES] == x["seg"]
        return x

    def describer(self):
        for u, x in enumerate(self.units):
            if (yield from self.gives_up("describer", u)):
                break
            if u >= NOTES and not (yield from self.wait(self.note_free[u % NOTES], u // NOTES - 1)):
                break
            self.notes[u % NOTES] = None
            yield
            self.notes[u % NOTES] = u
            if x["first"]:
                self.seg_notes[x["seg"] % NOTES] = x["seg"]
            self.note_full[u % NOTES].arrive()
            yield
        yield from self.meet_all()

    def copier(self, is_v):
        issued = edges = 0
        for u in range(len(self.units)):
            if (yield from self.gives_up("v" if is_v else "k", u)):
                break
            x = yield from self.read(u)
            if x is None:
                break
            self.note_free[u % NOTES].arrive()
            yield
            at = 2 * u + is_v
            slot, turn = at % self.slots, at // self.slots
            if turn and not (yield from self.wait(self.empty[slot], turn - 1)):
                break
            check = is_v and x["edge"]
            bar = self.edge[edges % NOTES] if check else self.full[slot]
            bar.arrive(1)
            if check:
                self.full[slot].arrive()
                edges += 1
            self.ring[slot] = ("loading", u, is_v)

            def landed(slot=slot, u=u, check=check, bar=bar):
                assert self.ring[slot] == ("loading", u, is_v)
                self.ring[slot] = ("raw" if check else "ready", u, is_v)
                bar.landed()
            self.copies.append(landed)
            issued += 1
            yield
        self.issued[is_v] = issued
        yield from self.meet_all()
        if self.abort:
            for u in range(max(0, issued - (self.slots + 1) // 2), issued):
                at = 2 * u + is_v
                # a slot whose next turn has begun was read, and its barrier may be a phase further
                n = at + self.slots
                if n // 2 >= self.issued[n & 1]:
                    yield from self.settle(self.full[at % self.slots], at // self.slots)
            for e in range(max(0, edges - 6), edges):
                yield from self.settle(self.edge[e % NOTES], e // NOTES)

    def q_loader(self):
        loaded = 0
        for u in range(len(self.units)):
            if (yield from self.gives_up("q", u)):
                break
            x = yield from self.read(u, seg=True)
            if x is None:
                break
            self.note_free[u % NOTES].arrive()
            yield
            if x["first"]:
                g, b = x["seg"], x["seg"] % self.q_bufs
                if g >= self.q_bufs and not (yield from self.wait(self.q_free[b], g // self.q_bufs - 1)):
                    break
                self.q[b] = None
                self.q_full[b].arrive(1)
                loaded = g + 1

                def landed(g=g, b=b):
                    self.q[b] = g
                    self.q_full[b].landed()
                self.copies.append(landed)
            yield
        for g in range(max(0, loaded - self.q_bufs), loaded):
            yield from self.settle(self.q_full[g % self.q_bufs], g // self.q_bufs)
        yield from self.meet_all()

    def value_check(self):
        edges = 0
        for u in range(len(self.units)):
            if (yield from self.gives_up("values", u)):
                break
            x = yield from self.read(u)
            if x is None:
                break
            self.note_free[u % NOTES].arrive()
            yield
            if x["edge"]:
                if not (yield from self.wait(self.edge[edges % NOTES], edges // NOTES)):
                    break
                slot = (2 * u + 1) % self.slots
                yield
                assert self.ring[slot] == ("raw", u, True)
                self.ring[slot] = ("ready", u, True)
                self.checked[edges % NOTES].arrive()
                edges += 1
        yield from self.meet_all()

    # ---- matrix instructions, executed in order by the unit
    def scores(self, u, sb, tile, slot):
        def run():
            x = self.units[u]
            assert self.ring[slot] == ("ready", u, False)
            assert self.q[x["seg"] % self.q_bufs] == x["seg"]
            assert not self.p[sb], "weights that P V has not read yet"
            self.s[sb] = u
        self.queue.append(run)

    def values(self, u, sb, ob, slot, half):
        def run():
            x = self.units[u]
            assert self.ring[slot] == ("ready", u, True)
            mine = {(u, half, q) for q in range(self.quarters)}
            assert mine <= self.p[sb]
            self.p[sb] -= mine
            if x["first"] and half == 0:
                if self.o[ob] is not None:
                    assert len(self.o_read[ob]) == 2 * self.quarters, "sums that were not taken out"
                self.o[ob], self.o_read[ob] = (x["seg"], None), set()
            assert self.o[ob][0] == x["seg"]
            if half == 1:
                self.o[ob] = (x["seg"], u)
                self.added = u
        self.queue.append(run)

    def commit(self, bar):
        self.queue.append(bar.arrive)

    def free_slot(self, slot):
        def run():
            self.ring[slot] = None
            self.empty[slot].arrive()
        self.queue.append(run)

    def free_q(self, b):
        self.commit(self.q_free[b])

    def issuer(self):
        yield from (self.issuer_one() if self.tiles == 1 else self.issuer_two())
        self.commit(self.drain)
        yield from self.settle(self.drain, 0)
        yield from self.meet_all()

    def v_there(self, u, edges):
        slot, turn = (2 * u + 1) % self.slots, (2 * u + 1) // self.slots
        if self.units[u]["edge"]:
            return (yield from self.wait(self.checked[edges[0] % NOTES], edges[0] // NOTES))
        return (yield from self.wait(self.full[slot], turn))

    def issuer_one(self):
        edges = [0]

        def products(u):
            x = self.units[u]
            g, slot = x["seg"], (2 * u + 1) % self.slots
            if x["first"] and g >= 2 and not (yield from self.wait(self.o_free[g & 1], (g >> 1) - 1)):
                return False
            if not (yield from self.v_there(u, edges)):
                return False
            edges[0] += x["edge"]
            for half in (0, 1):
                if not (yield from self.wait(self.p_full[2 * (u & 1) + half], u >> 1)):
                    return False
                self.values(u, u & 1, g & 1, slot, half)
                yield
            self.commit(self.o_full[0])
            self.free_slot(slot)
            self.note_free[u % NOTES].arrive()
            yield
            return True

        for u, x in enumerate(self.units):
            if (yield from self.gives_up("issuer", u)):
                return
            if (yield from self.read(u)) is None:
                return
            if x["first"] and u > 0 and not (yield from products(u - 1)):
                return
            at = 2 * u
            if not (yield from self.wait(self.full[at % self.slots], at // self.slots)):
                return
            b = x["seg"] % self.q_bufs
            if x["first"] and not (yield from self.wait(self.q_full[b], x["seg"] // self.q_bufs)):
                return
            self.scores(u, u & 1, 0, at % self.slots)
            self.commit(self.s_full[u & 1])
            self.free_slot(at % self.slots)
            if x["last"]:
                self.free_q(b)
            yield
            if not x["first"] and not (yield from products(u - 1)):
                return
        yield from products(len(self.units) - 1)

    def issuer_two(self):
        edges, segments = [0], 0

        def k_there(u):
            return (yield from self.wait(self.full[2 * u % self.slots], 2 * u // self.slots))

        def tile_scores(u, t):
            if t == 0 or self.units[u]["two"]:
                self.scores(u, t, t, 2 * u % self.slots)
            self.commit(self.s_full[t])

        def scores_done(u):
            x = self.units[u]
            self.free_slot(2 * u % self.slots)
            if x["last"]:
                self.free_q(x["seg"] % self.q_bufs)

        def first_scores(u):
            x = self.units[u]
            if not (yield from k_there(u)):
                return False
            if not (yield from self.wait(self.q_full[x["seg"] % self.q_bufs], x["seg"] // self.q_bufs)):
                return False
            for t in (0, 1):
                tile_scores(u, t)
                yield
            scores_done(u)
            return True

        if (yield from self.read(0)) is None or not (yield from first_scores(0)):
            return
        for u, x in enumerate(self.units):
            if (yield from self.gives_up("issuer", u)):
                return
            if not (yield from self.v_there(u, edges)):
                return
            edges[0] += x["edge"]
            more = u + 1 < len(self.units)
            if more and (yield from self.read(u + 1)) is None:
                return
            if not x["last"] and not (yield from k_there(u + 1)):
                return
            slot = (2 * u + 1) % self.slots
            for t in (0, 1):
                if x["first"] and segments and not (yield from self.wait(self.o_free[t], segments - 1)):
                    return
                for half in (0, 1):
                    if not (yield from self.wait(self.p_full[2 * t + half], u)):
                        return
                    if t == 0 or x["two"]:
                        self.values(u, t, t, slot, half)
                    yield
                if x["last"]:
                    self.commit(self.o_full[t])
                else:
                    tile_scores(u + 1, t)
                yield
            self.free_slot(slot)
            self.note_free[u % NOTES].arrive()
            yield
            if not x["last"]:
                scores_done(u + 1)
            else:
                segments += 1
                if more and not (yield from first_scores(u + 1)):
                    return

    def softmax(self, t, half, quarter):
        meets, segments = [0], 0
        pair = self.pairs[t, quarter]

        def meet():
            pair.arrive()
            yield
            ok = yield from self.wait(pair, meets[0])
            meets[0] += 1
            return ok

        def join(tag):
            """Both halves' values in both: first one writes, the other answers."""
            key = (t, quarter)
            if half == 0:
                self.tops[key] = (tag, 0)
            if not (yield from meet()):
                return False
            if half == 1:
                assert self.tops[key] == (tag, 0)
                self.tops[key] = (tag, 1)
            if not (yield from meet()):
                return False
            if half == 0:
                assert self.tops[key] == (tag, 1)
            return True

        for u, x in enumerate(self.units):
            if (yield from self.gives_up(("softmax", t, half, quarter), u)):
                break
            sb = u & 1 if self.tiles == 1 else t
            if not (yield from self.wait(self.s_full[sb], u >> 1 if self.tiles == 1 else u)):
                break
            yield
            assert self.notes[u % NOTES] == u
            if x["first"]:
                assert self.seg_notes[x["seg"] % NOTES] == x["seg"]
            if t == 1 and not x["two"]:
                self.p_full[2 * sb + half].arrive()
                yield
                if x["last"]:
                    if not (yield from self.wait(self.o_full[t], segments)):
                        break
                    segments += 1
                    self.o_free[t].arrive()
                continue
            ob = x["seg"] & 1 if self.tiles == 1 else t
            assert self.s[sb] == u
            yield
            if self.tiles == 1 and u > 0 and x["last"]:
                if not (yield from self.wait(self.o_full[0], u - 1)):
                    break
            rise = x["first"]
            if not rise:
                self.words[t, quarter, u & 1, half] = u
                if not (yield from meet()):
                    break
                assert self.words[t, quarter, u & 1, half ^ 1] == u
                rise = self.rises[u]
            if rise:
                if not (yield from join(("top", u))):
                    break
                if not x["first"]:
                    if self.tiles == 1 and not x["last"]:
                        if not (yield from self.wait(self.o_full[0], u - 1)):
                            break
                    assert self.o[ob] == (x["seg"], u - 1), "sums rescaled while they change"
                    yield
                    assert self.o[ob] == (x["seg"], u - 1)
            assert self.s[sb] == u
            self.p[sb].add((u, half, quarter))
            self.p_full[2 * sb + half].arrive()
            yield
            if not x["last"]:
                continue
            if not (yield from join(("sum", u))):
                break
            if not (yield from self.wait(self.o_full[0 if self.tiles == 1 else t], u if self.tiles == 1 else segments)):
                break
            segments += 1
            yield
            assert self.o[ob] == (x["seg"], u)
            yield
            assert self.o[ob] == (x["seg"], u)
            self.o_read[ob].add((half, quarter))
            self.out.setdefault((x["seg"], t), set()).add((half, quarter))
            self.o_free[ob].arrive()
        yield from self.meet_all()

    def run(self):
        rng = self.rng
        self.rises = [rng.random() < 0.3 for _ in self.units]
        roles = [self.describer(), self.copier(False), self.copier(True), self.q_loader(), self.value_check(), self.issuer()]
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
        return steps


def segments_of(rng, tiles):
    out = []
    for _ in range(rng.randint(1, 6)):
        n = rng.choice([1, 1, 2, 3, rng.randint(1, 14)])
        edges = {i for i in range(n) if rng.random() < (0.8 if i == n - 1 else 0.2)}
        out.append((n, tiles == 2 and rng.random() < 0.5, edges))
    return out


@pytest.mark.parametrize("tiles,slots,q_bufs", [(1, 5, 2), (1, 6, 2), (1, 12, 2), (2, 5, 1), (2, 10, 2)])
@pytest.mark.parametrize("seed", range(40))
def test_every_schedule_ends_and_reads_what_is_there(tiles, slots, q_bufs, seed):
    rng = random.Random(1000 * seed + 10 * slots + tiles)
    m = Model(rng, segments_of(rng, tiles), tiles, slots, q_bufs, rng.choice([1, 2]))
    m.run()
    assert not m.abort
    warps = {(h, q) for h in range(2) for q in range(m.quarters)}
    for x in m.units:
        for t in range(tiles):
            if t == 0 or x["two"]:
                assert m.out[x["seg"], t] == warps


@pytest.mark.parametrize("tiles,slots,q_bufs", [(1, 6, 2), (1, 12, 2), (2, 5, 1), (2, 10, 2)])
@pytest.mark.parametrize("seed", range(60))
def test_ends_where_a_role_gives_up(tiles, slots, q_bufs, seed):
    rng = random.Random(7000 * seed + 10 * slots + tiles)
    segments = segments_of(rng, tiles)
    roles = ["describer", "k", "v", "q", "values", "issuer"] + \
        [("softmax", t, h, 0) for t in range(tiles) for h in range(2)]
    m = Model(rng, segments, tiles, slots, q_bufs, 1, stall=(rng.choice(roles), rng.randrange(sum(n for n, *_ in segments))))
    m.run()


def test_the_model_sees_a_look_that_comes_too_late():
    """A phase that is looked at behind this unit's own arrival may be over: what the wait ahead of the
    output is there for."""
    class Late(Model):
        def softmax(self, t, half, quarter):
            for u in range(len(self.units)):
                sb = u & 1
                if not (yield from self.wait(self.s_full[sb], u >> 1)):
                    break
                self.p[sb].add((u, half, quarter))
                self.p_full[2 * sb + half].arrive()
                yield
                if u + 1 == len(self.units):
                    if not (yield from self.wait(self.o_full[0], u - 1)):
                        break
            yield from self.meet_all()

    caught = 0
    for seed in range(30):
        m = Late(random.Random(seed), [(3, False, set())], 1, 6, 2, 1)
        try:
            m.run()
        except AssertionError:
            caught += 1
    assert caught
