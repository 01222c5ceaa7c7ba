"""Model of the roles of one CTA of the chunk attention kernel and of the
tensor-core decode, and of the barriers between them (CPU only): every random
interleaving has to end.

Barriers have phases and are waited for by parity alone, so a role that is two
phases behind another waits for good.  A context that ends inside a block leaves
V rows to be zeroed once they have landed.  That tile lands on a barrier of the
V warp's own, and the warp completes the stage when it has zeroed them; it does
so before it waits for an item that is not there yet.  With the zeroing announced
on a barrier that the MMA thread waits for ("announced"), short items put the V warp two
phases ahead, or leave it waiting for an item with a zeroing still to do.
"""
import random

import pytest

RING = 2                                            # item ring


class Bar:
    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        self.left -= 1
        assert self.left >= 0
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def done(self, parity):                         # the phase before the current one has this parity
        return (self.phase & 1) != (parity & 1)


def wait(bar, parity):
    while not bar.done(parity):
        yield


class Cta:
    """What both kernels share: the rings of K and V, the tensor core, the copies, softmax."""

    def __init__(self, kst, vst, seed, announced, converted=False):
        self.kst, self.vst, self.announced, self.converted = kst, vst, announced, converted
        self.rnd = random.Random(seed)
        full = 4 if converted else 1
        self.kf, self.ke = [Bar(full) for _ in range(kst)], [Bar(1) for _ in range(kst)]
        self.vf, self.ve = [Bar(full) for _ in range(vst)], [Bar(1) for _ in range(vst)]
        self.s, self.p, self.free = ([Bar(n) for _ in range(2)] for n in (1, 4, 4))
        self.o = [Bar(2 if converted else 1) for _ in range(2)]     # (the MMA thread's own arrival beside its commit)
        self.vz = Bar(1)
        self.queue, self.copies = [], []            # commits in issue order; copies that land in any
        self.jt = self.vzj = None

    def zero(self, st):
        """The V warp zeroes the rows of its pending tile."""
        if self.announced:
            yield from wait(self.vf[st.vzj % self.vst], (st.vzj // self.vst) & 1)
            self.vz.arrive()
        else:
            yield from wait(self.vz, st.zeroed & 1)
            st.zeroed += 1
            self.vf[st.vzj % self.vst].arrive()
        st.vzj = -1

    def stream(self, st, is_v, tiles, zero_last):
        """The TMA warp of K or V streams an item's (segment's) tiles."""
        nst, full, empty = (self.vst, self.vf, self.ve) if is_v else (self.kst, self.kf, self.ke)
        for t in range(tiles):
            last = is_v and zero_last and t == tiles - 1
            if st.vzj >= 0 and (st.jt >= st.vzj + self.vst or (last and not self.announced)):
                yield from self.zero(st)
            if st.jt >= nst:
                yield from wait(empty[st.jt % nst], ((st.jt // nst) - 1) & 1)
            self.copies.append(self.vz if last and not self.announced else full[st.jt % nst])
            yield
            if last:
                if st.vzj >= 0:
                    yield from self.zero(st)
                st.vzj = st.jt
            st.jt += 1

    def tensor_core(self):
        while True:
            if self.queue:
                self.queue.pop(0).arrive()
            yield

    def landing(self):
        while True:
            if self.copies:
                self.copies.pop(self.rnd.randrange(len(self.copies))).arrive()
            yield

    def ends(self, roles):
        roles = dict(roles, tensor=self.tensor_core(), landing=self.landing())
        left = set(roles) - {"tensor", "landing"}
        names = [n for n in roles for _ in range(self.rnd.choice([1, 1, 3, 20]))]
        for _ in range(150000):
            n = self.rnd.choice(names)
            if n in left or n in ("tensor", "landing"):
                try:
                    next(roles[n])
                except StopIteration:
                    left.discard(n)
                    if not left:
                        return True
        return False


class Stream:
    def __init__(self):
        self.jt, self.vzj, self.zeroed = 0, -1, 0


class Chunks(Cta):
    """Items (tiles of query tile 0, of query tile 1, rows to zero) through the item ring."""

    def run(self, items):
        readers = 15 if self.converted else 11
        self.items = items + [None]
        self.ifull, self.iempty = [Bar(1) for _ in range(RING)], [Bar(readers) for _ in range(RING)]
        self.qfull, self.qempty = [Bar(1) for _ in range(2)], [Bar(1) for _ in range(2)]
        roles = {"scheduler": self.scheduler(), "mma": self.mma()}
        if self.converted:
            roles.update({f"convert{c}": self.converter(c) for c in range(6)})
        else:
            roles.update(K=self.producer(False), V=self.producer(True))
        roles.update({f"softmax{x}.{w}": self.softmax(x) for x in range(2) for w in range(4)})
        return self.ends(roles)

    def take(self, j):
        yield from wait(self.ifull[j % RING], (j // RING) & 1)
        yield
        self.iempty[j % RING].arrive()
        return self.items[j]

    def scheduler(self):
        loads = [0, 0]
        for j, it in enumerate(self.items):
            if j >= RING:
                yield from wait(self.iempty[j % RING], ((j // RING) - 1) & 1)
            self.ifull[j % RING].arrive()
            if it is None:
                return
            for x in range(2 if it[1] else 1):
                if loads[x]:
                    yield from wait(self.qempty[x], (loads[x] - 1) & 1)
                self.copies.append(self.qfull[x])
                loads[x] += 1
                yield

    def mma(self):
        jt0 = zeroed = j = 0
        loads, weights, units = [0, 0], [0, 0], [0, 0]
        while True:
            it = yield from self.take(j)
            j += 1
            if it is None:
                return
            n, nT = it[:2], max(it[:2])
            zero_x = 0 if n[0] == nT else 1

            def qk(x, i):
                self.queue.append(self.s[x])
                if i == n[x] - 1:
                    self.queue.append(self.qempty[x])

            def pv(x, i):
                nonlocal zeroed
                jt = jt0 + i
                yield from wait(self.vf[jt % self.vst], (jt // self.vst) & 1)
                if self.announced and it[2] and i == nT - 1 and x == zero_x:
                    yield from wait(self.vz, zeroed & 1)
                    zeroed += 1
                yield from wait(self.p[x], weights[x] & 1)
                weights[x] += 1
                if i == 0:
                    if units[x]:
                        yield from wait(self.free[x], (units[x] - 1) & 1)
                    units[x] += 1
                if i == n[x] - 1:
                    self.queue.append(self.o[x])
                    if self.converted:
                        self.o[x].arrive()
            for i in range(nT):
                jt = jt0 + i
                if i == 0:
                    yield from wait(self.qfull[0], loads[0] & 1)
                    loads[0] += 1
                yield from wait(self.kf[jt % self.kst], (jt // self.kst) & 1)
                if i < n[0]:
                    qk(0, i)
                if n[1] and i:
                    yield from pv(1, i - 1)
                    self.queue.append(self.ve[(jt - 1) % self.vst])
                if i < n[1]:
                    if i == 0:
                        yield from wait(self.qfull[1], loads[1] & 1)
                        loads[1] += 1
                    qk(1, i)
                self.queue.append(self.ke[jt % self.kst])
                if i < n[0]:
                    yield from pv(0, i)
                    if not n[1]:
                        self.queue.append(self.ve[jt % self.vst])
            if n[1]:
                yield from pv(1, nT - 1)
                self.queue.append(self.ve[(jt0 + nT - 1) % self.vst])
            jt0 += nT

    def producer(self, is_v):
        st, j = Stream(), 0
        while True:
            if st.vzj >= 0 and not self.announced and not self.ifull[j % RING].done((j // RING) & 1):
                yield from self.zero(st)
            it = yield from self.take(j)
            j += 1
            if it is None:
                break
            yield from self.stream(st, is_v, max(it[:2]), it[2])
        if st.vzj >= 0:
            yield from self.zero(st)

    def converter(self, c):
        """Three warps a stream take the four slices of its tiles in turn."""
        nst, full, empty = (self.vst, self.vf, self.ve) if c >= 3 else (self.kst, self.kf, self.ke)
        w, jt, j = c % 3, 0, 0
        while True:
            it = yield from self.take(j)
            j += 1
            if it is None:
                return
            end = jt + max(it[:2])
            while jt < end:
                if jt >= nst:
                    yield from wait(empty[jt % nst], ((jt // nst) - 1) & 1)
                yield
                full[jt % nst].arrive()
                w += 3
                if w >= 4:
                    w, jt = w - 4, jt + 1

    def softmax(self, x):
        tiles = units = j = 0
        while True:
            it = yield from self.take(j)
            j += 1
            if it is None:
                return
            for _ in range(it[x]):
                yield from wait(self.s[x], tiles & 1)
                tiles += 1
                yield
                self.p[x].arrive()
            if it[x]:
                yield from wait(self.o[x], units & 1)
                units += 1
                yield
                self.free[x].arrive()


class Decode(Cta):
    """Segments (tiles, rows to zero), which every role knows; the tiles alternate between two halves."""

    def run(self, segments):
        self.segments = segments
        roles = {"mma": self.mma(), "K": self.producer(False), "V": self.producer(True)}
        roles.update({f"softmax{x}.{w}": self.softmax(x) for x in range(2) for w in range(4)})
        return self.ends(roles)

    def mma(self):
        jt = zeroed = 0
        weights, units, prev = [0, 0], [0, 0], None

        def pv(e):
            nonlocal zeroed
            t, first, last, zero = e
            x = t & 1
            yield from wait(self.vf[t % self.vst], (t // self.vst) & 1)
            if self.announced and zero:
                yield from wait(self.vz, zeroed & 1)
                zeroed += 1
            yield from wait(self.p[x], weights[x] & 1)
            weights[x] += 1
            if first:
                if units[x]:
                    yield from wait(self.free[x], (units[x] - 1) & 1)
                units[x] += 1
            self.queue.append(self.ve[t % self.vst])
            if last:
                self.queue.append(self.o[x])
        for n, zero in self.segments:
            for i in range(n):
                yield from wait(self.kf[jt % self.kst], (jt // self.kst) & 1)
                self.queue += [self.s[jt & 1], self.ke[jt % self.kst]]
                if prev:
                    yield from pv(prev)
                prev = (jt, i < 2, i >= n - 2, zero and i == n - 1)
                jt += 1
        if prev:
            yield from pv(prev)

    def producer(self, is_v):
        st = Stream()
        for n, zero in self.segments:
            yield from self.stream(st, is_v, n, zero)
        if st.vzj >= 0:
            yield from self.zero(st)

    def softmax(self, x):
        jt = tiles = units = 0
        for n, _ in self.segments:
            count = sum((jt + i) & 1 == x for i in range(n))
            jt += n
            for _ in range(count):
                yield from wait(self.s[x], tiles & 1)
                tiles += 1
                yield
                self.p[x].arrive()
            if count:
                yield from wait(self.o[x], units & 1)
                units += 1
                yield
                self.free[x].arrive()


def chunk_items(rnd):
    out = []
    for _ in range(rnd.randint(1, 7)):
        a = rnd.randint(1, 3)
        out.append((a, a + rnd.randint(0, 1) if rnd.random() < 0.6 else 0, rnd.random() < 0.5))
    return out


def segments(rnd):
    return [(rnd.choice([1, 1, 1, 2, 5]), rnd.random() < 0.7) for _ in range(rnd.randint(1, 10))]


@pytest.mark.parametrize("kst,vst,converted", [(4, 4, False), (3, 2, False), (4, 4, True), (2, 2, True)])
def test_chunks_end(kst, vst, converted):
    rnd = random.Random(kst)
    for seed in range(120):
        items = chunk_items(rnd)
        assert Chunks(kst, vst, seed, False, converted).run(items), items


@pytest.mark.parametrize("kst,vst", [(5, 4), (3, 2)])
def test_decode_ends(kst, vst):
    rnd = random.Random(kst)
    for seed in range(150):
        units = segments(rnd)
        assert Decode(kst, vst, seed, False).run(units), units


@pytest.mark.parametrize("kind,draw,kst,vst", [(Chunks, chunk_items, 4, 4), (Decode, segments, 5, 4)])
def test_the_model_finds_an_announced_zeroing_stuck(kind, draw, kst, vst):
    rnd = random.Random(1)
    assert not all(kind(kst, vst, seed, True).run(draw(rnd)) for seed in range(60))
