"""The barriers of the attention of prompts and chunks, in a model of their protocol (csrc/kv_prompt.cu).

A barrier's phases are told apart by their parity alone, so a role may neither be two phases behind one
nor wait for one that may come round again.  Here the kernel's roles, each of their warps an actor of its
own, run in random orders at random speeds, with copies that arrive in any order and products that are done in
theirs.  Every wait that passes must be for the phase that it means, and whatever is read (slots of the ring,
queries, scores, p, o, what is known of a tile, values taken out) must be what the reader
takes it for, and not be overwritten before.  The model follows the kernel by hand, its sizes are read from the source.
"""
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "model_free_suffix_gb300", "csrc", "kv_prompt.cu")
TEXT = open(SOURCE).read()


def _int(name):
    return int(re.search(r"\b%s = (\d+)" % name, TEXT).group(1))


def _by_dim(name, dim):
    wide, narrow = re.search(r"\b%s = D == 128 \? (\d+) : (\d+)" % name, TEXT).groups()
    return int(wide if dim == 128 else narrow)


LOADERS, META, SEGMENTS = _int("LOADERS"), _int("META"), _int("BAD_SEGMENTS")
QUARTERS, SOFTMAX = 4, 8     # warps of a row tile, of both


class Wrong(Exception):
    pass


def require(what, *why):
    if not what:
        raise Wrong(why)


class Bar:
    def __init__(self, count):
        self.count = self.left = count
        self.phase = 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1


def wait(bar, k, who):
    """Until phase k is complete, as told by its parity."""
    while bar.phase & 1 == k & 1:
        require(bar.phase == k, who, "waits for phase", k, "and is at", bar.phase)
        yield
    require(bar.phase == k + 1, who, "took phase", bar.phase - 1, "for", k)


class Model:
    """segments: (tiles, two row tiles?) of a CTA; kinds: of each tile, "cached", "tma", "late" (values by a copy
    that is checked later) or "plain".  form: the kernel's, or one that is known to be wrong."""

    def __init__(self, seed, dim, form=""):
        rnd = self.rnd = random.Random(seed)
        self.stages, self.buffers, self.form = _by_dim("STAGES", dim), _by_dim("BUFFERS", dim), form
        longest = rnd.choice([1, 2, 3, 9])
        self.segments = [(rnd.randint(1, longest), rnd.random() < 0.6) for _ in range(rnd.randint(1, 14))]
        shares = rnd.choice([(1, 0, 0, 0), (0, 1, 1, 0), (0, 0, 1, 0), (2, 1, 2, 0), (1, 0, 0, 1)])
        self.kinds = [rnd.choices(["cached", "tma", "late", "plain"], shares, k=n) for n, _ in self.segments]
        S, B = self.stages, self.buffers
        self.full, self.empty = [Bar(LOADERS) for _ in range(S)], [Bar(1) for _ in range(S)]
        self.raw = [Bar(1) for _ in range(1 if form == "one barrier for checked values" else S)]
        self.q_full, self.q_empty = Bar(LOADERS), Bar(1)
        self.s_full = [[Bar(1) for _ in range(B)] for _ in range(2)]
        if form == "scores' barriers by buffer":
            self.s_full[1] = self.s_full[0]
        self.p_half, self.p_full = [Bar(QUARTERS) for _ in range(B)], [Bar(QUARTERS) for _ in range(B)]
        self.pv_half, self.pv_done = ([[Bar(1) for _ in range(B)] for _ in range(2)] for _ in range(2))
        self.o_empty, self.over = [Bar(QUARTERS) for _ in range(2)], [Bar(SOFTMAX) for _ in range(SEGMENTS)]
        # what lies where
        self.slot, self.slot_busy = [dict() for _ in range(S)], [False] * S
        self.queries, self.scores = {}, [None] * B
        self.p, self.o, self.o_read = {}, [None, None], [QUARTERS, QUARTERS]
        self.meta, self.meta_read = {}, {}
        self.bad, self.bad_read = {}, {}
        self.pipe, self.copies = [], []

    # -- the ring
    def fill(self, slot, item, part):
        held = self.slot[slot]
        if held.get("item") != item:
            require(not self.slot_busy[slot], "slot overwritten", slot, held, item)
            self.slot[slot] = held = {"item": item}
            self.slot_busy[slot] = True
        held[part] = True

    def use(self, slot, item, last):
        held = self.slot[slot]
        require(held.get("item") == item and ("all" in held or all(w in held for w in range(LOADERS))), "slot", slot, held, item)
        if last:
            self.slot_busy[slot] = False

    def loader(self, me):
        S, one_raw = self.stages, len(self.raw) == 1
        item = g = 0
        late, uses = None, [0] * S

        def put(kind, item):
            slot = item % S
            if kind in ("cached", "plain"):
                self.fill(slot, item, me)
                self.full[slot].arrive()
            elif me == 0:      # (its arrival counts once the bytes are there)
                self.copies.append(lambda: (self.fill(slot, item, "all"), self.full[slot].arrive()))
            else:
                self.full[slot].arrive()

        def settle():
            nonlocal late
            if late is None:
                return
            slot, item, segment = late
            late = None
            which = 0 if one_raw else slot
            yield from wait(self.raw[which], uses[which], "loader, checked values")
            uses[which] += 1
            require(self.slot[slot].get("item") == item, "checked values overwritten", slot)
            self.bad[segment % SEGMENTS][1].add(me)
            self.full[slot].arrive()

        for segment, (tiles, two) in enumerate(self.segments):
            if segment >= SEGMENTS:
                yield from wait(self.over[segment % SEGMENTS], segment // SEGMENTS - 1, "loader, segment over")
            for j in range(tiles):
                kind = self.kinds[segment][j]
                if me == 0:
                    if j == 0:
                        require(segment < SEGMENTS or self.bad_read[segment - SEGMENTS] == SOFTMAX, "values taken out overwritten")
                        self.bad[segment % SEGMENTS] = (segment, set())
                        self.bad_read.setdefault(segment, 0)
                    before = self.meta.get(g % META)
                    require(before is None or self.meta_read[before[0]] == QUARTERS * (1 + before[1]), "what is known of a tile overwritten")
                    self.meta[g % META] = (g, two)
                    self.meta_read[g] = 0
                g += 1
                if item >= S:
                    yield from wait(self.empty[item % S], item // S - 1, "loader, keys' slot")
                put("tma" if kind == "late" else kind, item)
                item += 1
                yield
                yield from settle()
                if j == 0:
                    if segment > 0:
                        yield from wait(self.q_empty, segment - 1, "loader, queries")
                    if self.queries.get("segment") != segment:
                        self.queries = {"segment": segment}
                    self.queries[me] = True
                    self.q_full.arrive()
                    yield
                if item >= S:
                    yield from wait(self.empty[item % S], item // S - 1, "loader, values' slot")
                if kind == "late":
                    late = (item % S, item, segment)
                    if me == 0:
                        slot, which = item % S, 0 if one_raw else item % S
                        self.copies.append(lambda slot=slot, item=item, which=which: (self.fill(slot, item, "all"), self.raw[which].arrive()))
                else:
                    put(kind, item)
                item += 1
                yield
        yield from settle()

    # -- the products
    def issuer(self):
        S, B = self.stages, self.buffers
        first_item = segs1 = 0
        s_buf = p_buf = p_use = 0
        s_turn, p_turn = [0, 0], [0, 0]
        for segment, (tiles, two) in enumerate(self.segments):
            yield from wait(self.q_full, segment, "issuer, queries")
            at = [0, 0]     # row tile and key tile of the next scores
            here = segment

            def scores():
                nonlocal s_buf
                (i, j), segment = at, here
                item = first_item + 2 * j
                if i == 0:
                    yield from wait(self.full[item % S], item // S, "issuer, keys")
                buf, bar = s_buf, self.s_full[i][(s_buf if self.form == "scores' barriers by buffer" else s_turn[i] % B)]
                last = i == int(two)

                def run():
                    require(self.queries.get("segment") == segment and all(w in self.queries for w in range(LOADERS)), "queries")
                    self.use(item % S, item, last)
                    require(not any(key[0] == buf for key in self.p), "p overwritten by scores", buf)
                    self.scores[buf] = (segment, i, j)
                self.pipe += [run, bar.arrive]
                if last:
                    self.pipe.append(self.empty[item % S].arrive)
                    if j + 1 == tiles:
                        self.pipe.append(self.q_empty.arrive)
                s_turn[i] += 1
                s_buf = (s_buf + 1) % B
                at[:] = [0, j + 1] if last else [1, j]

            for _ in range(B):
                if at[1] < tiles:
                    yield from scores()
            for j in range(tiles):
                item = first_item + 2 * j + 1
                yield from wait(self.full[item % S], item // S, "issuer, values")
                for i in range(1 + two):
                    if j == 0:
                        before = segs1 if i else segment
                        if before > 0:
                            yield from wait(self.o_empty[i], before - 1, "issuer, o")

                    def product(half, segment=segment, i=i, j=j, buf=p_buf, item=item, last=False):
                        def run():
                            self.use(item % S, item, last)
                            for w in range(QUARTERS):
                                require(self.p.pop((buf, half, w), None) == (segment, i, j), "p", buf, half, w)
                            if j == 0 and half == 0:
                                require(self.o_read[i] == QUARTERS, "o overwritten")
                                self.o_read[i] = 0
                            self.o[i] = (segment, j, half)
                        return run
                    yield from wait(self.p_half[p_buf], p_use, "issuer, half of p")
                    self.pipe += [product(0), self.pv_half[i][p_turn[i] % B].arrive]
                    yield from wait(self.p_full[p_buf], p_use, "issuer, p")
                    last = i == int(two)
                    self.pipe += [product(1, last=last), self.pv_done[i][p_turn[i] % B].arrive]
                    if last:
                        self.pipe.append(self.empty[item % S].arrive)
                    p_turn[i] += 1
                    p_buf += 1
                    if p_buf == B:
                        p_buf, p_use = 0, p_use + 1
                    if at[1] < tiles:
                        yield from scores()
            first_item += 2 * tiles
            segs1 += two

    # -- the softmax
    def softmax(self, warp):
        B, rnd = self.buffers, self.rnd
        i, quarter = warp // QUARTERS, warp % QUARTERS
        buf = turn = g = 0
        uses = [0] * B       # (of the barriers by buffer)
        for segment, (tiles, two) in enumerate(self.segments):
            s_buf, buf0 = (buf + i) % B, buf
            buf = (buf + (tiles << two)) % B
            if i > two:
                if segment >= SEGMENTS:
                    yield from wait(self.over[segment % SEGMENTS], segment // SEGMENTS - 1, "softmax, segment over")
                g += tiles
                for n in range(tiles):
                    uses[(buf0 + n) % B] += 1
                self.bad_read[segment] = self.bad_read.get(segment, 0) + 1
                self.over[segment % SEGMENTS].arrive()
                continue
            for j in range(tiles):
                if self.form == "scores' barriers by buffer":
                    mine = uses[s_buf]
                    for n in range(1 + two):
                        uses[(buf0 + j * (1 + two) + n) % B] += 1
                    mine = uses[s_buf] - 1
                    yield from wait(self.s_full[i][s_buf], mine, "softmax, scores")
                else:
                    yield from wait(self.s_full[i][turn % B], turn // B, "softmax, scores")
                require(self.scores[s_buf] == (segment, i, j), "scores", self.scores[s_buf], (segment, i, j))
                require(self.meta.get(g % META) == (g, two), "what is known of a tile")
                for half in range(2):
                    for _ in range(rnd.choice([0, 0, 1, 5])):
                        yield
                    if j + half > 0 and rnd.random() < 0.2:     # the reference rises
                        if j > 0:
                            yield from wait(self.pv_done[i][(turn - 1) % B], (turn - 1) // B, "softmax, o of the tile before")
                        if half > 0:
                            yield from wait(self.pv_half[i][turn % B], turn // B, "softmax, o of half a tile")
                        require(self.o[i] == ((segment, j, 0) if half else (segment, j - 1, 1)), "o", self.o[i], (segment, j, half))
                    require((s_buf, half, quarter) not in self.p, "p overwritten")
                    require(self.scores[s_buf] == (segment, i, j) and self.meta[g % META][0] == g, "a tile's scores went")
                    self.p[s_buf, half, quarter] = (segment, i, j)
                    (self.p_full if half else self.p_half)[s_buf].arrive()
                self.meta_read[g] += 1
                s_buf = (s_buf + 1 + two) % B
                turn += 1
                g += 1
            yield from wait(self.pv_done[i][(turn - 1) % B], (turn - 1) // B, "softmax, result")
            for _ in range(rnd.choice([0, 0, 5, 60])):
                yield
            require(self.o[i] == (segment, tiles - 1, 1), "result", self.o[i])
            self.o_read[i] += 1
            self.o_empty[i].arrive()
            for _ in range(rnd.choice([0, 0, 5, 60])):
                yield
            noted = self.bad[segment % SEGMENTS]
            require(noted[0] == segment, "values taken out", noted, segment)
            require("late" not in self.kinds[segment] or len(noted[1]) == LOADERS, "values taken out", noted)
            self.bad_read[segment] += 1
            self.over[segment % SEGMENTS].arrive()

    def run(self):
        rnd = self.rnd
        actors = [self.issuer()] + [self.loader(w) for w in range(LOADERS)] + [self.softmax(w) for w in range(SOFTMAX)]
        speeds = [rnd.choice([0.05, 0.3, 1.0]) for _ in range(len(actors) + 2)]
        if rnd.random() < 0.5:      # warps of a role together, or each on its own
            speeds[1:1 + LOADERS] = [speeds[1]] * LOADERS
        live, idle = set(range(len(actors))), 0
        while live or self.pipe or self.copies:
            which = rnd.randrange(len(actors) + 2)
            if rnd.random() > speeds[which]:
                continue
            idle += 1
            require(idle < 400000, "hangs")
            if which == len(actors):
                if self.pipe:
                    self.pipe.pop(0)()
            elif which == len(actors) + 1:
                if self.copies:
                    self.copies.pop(rnd.randrange(len(self.copies)))()
            elif which in live:
                try:
                    next(actors[which])
                except StopIteration:
                    live.discard(which)
        require(not self.p and not any(self.slot_busy) and all(n == QUARTERS for n in self.o_read), "something is left")


@pytest.mark.parametrize("dim", [64, 128])
def test_every_order_gives_each_role_what_it_waits_for(dim):
    for seed in range(70):
        Model(seed, dim).run()


@pytest.mark.parametrize("form", ["one barrier for checked values", "scores' barriers by buffer"])
def test_forms_that_are_wrong_are_found(form):
    """Two that the kernel once had: their phases come round again while someone is behind."""
    def wrong(seed):
        try:
            Model(seed, 64 if seed % 2 else 128, form).run()
        except Wrong:
            return True
        return False
    assert any(wrong(seed) for seed in range(150))
