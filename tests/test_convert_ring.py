"""Model of the tile rings between the converting warps and the tensor core of
the E4M3 prefill and the tensor-core decode over row caches (CPU only).

Three warps (in the decode four) take the four 32-row slices of each K tile in
turn and as many those of each V tile; they fill the stages, and the MMA thread's products empty them.
Barriers have phases and are waited for by parity alone, so a wait is only right
if its phase is the current one or the one before.  Random interleavings of the roles must all end, and no
slice may be written while a product may still read its stage.
"""
import random

import pytest

# (stream, first slice, step) of each warp: slices 0-3 of a tile are K, 4-7 V
STREAMS = [(k, c, 3) for k in (0, 4) for c in range(3)]
FOUR = [(k, c, 4) for k in (0, 4) for c in range(4)]
MIXED = [(None, c, 6) for c in range(6)]


class Bar:
    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        self.left -= 1
        assert self.left >= 0
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def done(self, parity):                 # the wait by parity: the phase before the current one has this parity
        return (self.phase & 1) != (parity & 1)


def run(kst, vst, tiles, order, seed, warps=STREAMS):
    rnd = random.Random(seed)
    full = {"k": [Bar(4) for _ in range(kst)], "v": [Bar(4) for _ in range(vst)]}
    empty = {"k": [Bar(1) for _ in range(kst)], "v": [Bar(1) for _ in range(vst)]}
    nst = {"k": kst, "v": vst}
    holds = {"k": [-1] * kst, "v": [-1] * vst}       # tile whose products may still read the stage
    queue = []                                       # the tensor core: operations in issue order
    ready_s, ready_p = {}, {}                        # S of (x, tile) complete; P of (x, tile) written

    def warp(base, first, step):
        n = first                                    # the warp's slice of its stream (or of both, in turn)
        per = 8 if base is None else 4
        while n // per < tiles:
            jt, k = n // per, n % per + (base or 0)
            name = "v" if k & 4 else "k"
            st = jt % nst[name]
            while jt >= nst[name] and not empty[name][st].done(jt // nst[name] - 1):
                yield
            assert holds[name][st] in (-1, jt), f"{name} stage {st} written for tile {jt} while tile {holds[name][st]} is read"
            holds[name][st] = jt
            yield
            full[name][st].arrive()
            n += step

    def mma():
        for op in order(tiles):
            kind, x, i = op
            if kind == "qk":
                while not full["k"][i % kst].done(i // kst):
                    yield
                queue.append(("s", x, i))
            elif kind == "pv":
                while not full["v"][i % vst].done(i // vst) or (x, i) not in ready_p:
                    yield
                queue.append(("o", x, i))
            else:
                queue.append((kind, x, i))           # commit of a stage's empty barrier
            yield

    def tensor():
        for _ in order(tiles):
            while not queue:
                yield
            kind, x, i = queue.pop(0)
            if kind == "s":
                assert holds["k"][i % kst] == i
                ready_s[x, i] = True
            elif kind == "o":
                assert holds["v"][i % vst] == i
            else:
                m = kind[0]
                holds[m][i % nst[m]] = -1
                empty[m][i % nst[m]].arrive()
            yield

    def softmax(x):
        for kind, y, i in order(tiles):
            if kind == "qk" and y == x:
                while (x, i) not in ready_s:
                    yield
                ready_p[x, i] = True
                yield
    roles = [warp(*w) for w in warps] + [mma(), tensor(), softmax(0), softmax(1)]
    weights = [rnd.choice([1, 1, 1, 20]) for _ in roles]
    idle = 0
    while roles:
        n = rnd.choices(range(len(roles)), weights)[0]
        try:
            next(roles[n])
        except StopIteration:
            roles.pop(n), weights.pop(n)
            idle = 0
        idle += 1
        assert idle < 200000, "the roles wait for one another"


def prefill_order(tiles, two=True):
    ops = []
    for i in range(tiles):
        ops.append(("qk", 0, i))
        if two and i >= 1:
            ops += [("pv", 1, i - 1), ("v", 0, i - 1)]
        if two:
            ops.append(("qk", 1, i))
        ops += [("k", 0, i), ("pv", 0, i)]
        if not two:
            ops.append(("v", 0, i))
    if two:
        ops += [("pv", 1, tiles - 1), ("v", 0, tiles - 1)]
    return ops


def decode_order(tiles):
    ops = []
    for i in range(tiles):
        ops += [("qk", i & 1, i), ("k", 0, i)]
        if i:
            ops += [("pv", (i - 1) & 1, i - 1), ("v", 0, i - 1)]
    return ops + [("pv", (tiles - 1) & 1, tiles - 1), ("v", 0, tiles - 1)]


@pytest.mark.parametrize("kst,vst", [(2, 2), (4, 4)])
@pytest.mark.parametrize("two", [True, False])
def test_prefill_rings(kst, vst, two):
    for seed in range(60):
        run(kst, vst, 1 + seed % 23, lambda n: prefill_order(n, two), seed)


@pytest.mark.parametrize("kst,vst", [(1, 1), (3, 3)])
def test_decode_rings(kst, vst):
    for seed in range(60):
        run(kst, vst, 1 + seed % 23, decode_order, seed, warps=FOUR)
        run(kst, vst, 1 + seed % 23, decode_order, seed)


def test_the_model_finds_a_skipped_phase():
    """Warps that take K and V slices in turn skip tiles of a stream, and their
    waits take an older phase for the one they need."""
    with pytest.raises(AssertionError, match="written for tile|wait for one another"):
        for seed in range(200):
            run(1, 1, 20, decode_order, seed, warps=MIXED)
