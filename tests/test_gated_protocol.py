"""CPU model of two barrier protocols in the experts' kernel (csrc/experts.cu), run under random interleavings: the two
accumulators of a gated unit whose sums are formed in halves, and the scale bytes that four epilogue warps bring
together.  Waits test the parity of a phase, as the hardware's do: a wait that could pass a phase early or late shows up
as a stale read, an overwrite or a deadlock."""
import random

import pytest


class Barrier:
    """An mbarrier: `count` arrivals complete a phase; a wait on a parity passes unless the current phase has it."""

    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        assert self.left > 0
        self.left -= 1
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def passed(self, parity):
        return (self.phase & 1) != parity


def _run(roles, rng, limit=200000):
    """Steps generators that yield a condition to wait for (or None) until all of them end."""
    waiting = {i: None for i in range(len(roles))}
    live = list(waiting)
    for _ in range(limit):
        if not live:
            return
        ready = [i for i in live if waiting[i] is None or waiting[i]()]
        assert ready, "deadlock"
        i = rng.choice(ready)
        try:
            waiting[i] = next(roles[i])
        except StopIteration:
            live.remove(i)
    raise AssertionError("no end")


@pytest.mark.parametrize("steps", [1, 2, 5])
@pytest.mark.parametrize("seed", range(30))
def test_accumulators_of_halves(steps, seed):
    """MMA issuer and epilogue warps (both CTAs' arrive on one barrier): the first accumulator is free after the fold, the
    second after the stores; a unit's sums are read while they are its own."""
    units, warps = 7, 4
    full, empty = Barrier(1), [Barrier(warps), Barrier(warps)]
    # what the accumulators hold in each warp's lanes and columns: (unit, half) or ("sum", unit)
    acc = [[None] * warps, [None] * warps]
    folds = {u: 0 for u in range(units)}
    half = (steps + 1) // 2

    def issuer():
        aph = 0
        for u in range(units):
            yield lambda: empty[0].passed(aph ^ 1)
            assert u == 0 or folds[u - 1] == warps
            acc[0][:] = [(u, 0)] * warps
            for k in range(steps):
                if k == half:
                    yield lambda: empty[1].passed(aph ^ 1)
                    assert u == 0 or stored[u - 1] == warps
                    acc[1][:] = [(u, 1)] * warps
                yield None
            full.arrive()
            aph ^= 1

    stored = {u: 0 for u in range(units)}

    def epilogue(w):
        aph = 0
        for u in range(units):
            yield lambda: full.passed(aph)
            assert acc[0][w] == (u, 0)
            yield None
            if half < steps:
                assert acc[1][w] == (u, 1)
            acc[1][w] = ("sum", u)
            yield None
            assert acc[0][w] == (u, 0)
            folds[u] += 1
            empty[0].arrive()
            for _ in range(3):
                yield None
                assert acc[1][w] == ("sum", u)
            stored[u] += 1
            empty[1].arrive()
            aph ^= 1

    _run([issuer()] + [epilogue(w) for w in range(warps)], random.Random(seed))
    assert all(n == warps for n in stored.values())


@pytest.mark.parametrize("seed", range(30))
def test_scale_bytes_of_four_warps(seed):
    """Two buffers in turn, one barrier a unit: what a warp copies out is all four warps' bytes of this unit.  Units
    without columns for this half are passed over by all four alike."""
    rng = random.Random(seed)
    units = [rng.random() < 0.8 for _ in range(12)]
    bar, buffers = Barrier(4), [{}, {}]

    def warp(q):
        sph = 0
        for u, has_columns in enumerate(units):
            if not has_columns:
                continue
            for row in range(4):
                buffers[sph][q, row] = u
                yield None
            bar.arrive()
            yield lambda: bar.passed(sph)
            for other in range(4):  # this warp's quarter of the rows, every warp's byte
                assert buffers[sph][other, q] == u
                yield None
            sph ^= 1

    _run([warp(q) for q in range(4)], rng)


def test_the_model_finds_a_missing_buffer():
    """With one buffer instead of two a fast warp overwrites what a slow one still copies."""
    found = False
    for seed in range(50):
        rng = random.Random(seed)
        bar, buffer = Barrier(4), {}

        def warp(q):
            phase = 0
            for u in range(6):
                for row in range(4):
                    buffer[q, row] = u
                    yield None
                bar.arrive()
                yield lambda: bar.passed(phase)
                for other in range(4):
                    assert buffer[other, q] == u
                    yield None
                phase ^= 1

        try:
            _run([warp(q) for q in range(4)], rng)
        except AssertionError:
            found = True
    assert found
