"""CPU model of the accumulators of the gated block kept in 8 bits, fp16 (csrc/experts.cu), with what the model of
test_gated_protocol.py holds fixed: the two warps of a TMEM quarter share its columns, and the border between them follows
the live rows of each unit, so that a column changes hands from one unit to the next."""
import random
import re

import pytest

from tests.test_gated_protocol import Barrier, _run
from tests.test_warp_convergence import _body, _code

CHUNKS = 8  # of 32 columns


def _stale(steps, alternate, seed, units=9):
    """Whether some warp reads a chunk that is not its unit's.  alternate: a single half alternates between the accumulators;
    else it is copied into the second one."""
    rng = random.Random(seed)
    lives = [rng.randint(1, CHUNKS) for _ in range(units)]
    half = (steps + 1) // 2
    two = steps > 1
    fold = two or not alternate
    full, empty = [Barrier(1), Barrier(1)], [Barrier(2), Barrier(2)]
    acc = [[None] * CHUNKS, [None] * CHUNKS]
    found = []

    def issuer():
        a = aph = 0
        for u in range(units):
            yield lambda: empty[a].passed(aph ^ 1)
            d = a
            for k in range(steps):
                if two and k == half:
                    yield lambda: empty[1].passed(aph ^ 1)
                    d = 1
                acc[d] = [(u, k >= half)] * CHUNKS
                yield None
            full[a].arrive()
            a ^= not fold
            if a == 0:
                aph ^= 1

    def epilogue(w):
        a = aph = 0
        for u in range(units):
            yield lambda: full[a].passed(aph)
            mid = (lives[u] + 1) // 2
            mine = range(mid, lives[u]) if w else range(mid)
            read = a
            if fold:
                for c in mine:
                    if acc[0][c] != (u, False) or (two and acc[1][c] != (u, True)):
                        found.append((u, c))
                    acc[1][c] = ("sum", u)
                    yield None
                empty[0].arrive()
                read = 1
            for c in mine:
                if acc[read][c] != (("sum", u) if fold else (u, False)):
                    found.append((u, c))
                yield None
            empty[read].arrive()
            a ^= not fold
            if a == 0:
                aph ^= 1

    _run([issuer(), epilogue(0), epilogue(1)], rng)
    return bool(found)


@pytest.mark.parametrize("steps", [1, 2, 3, 5])
def test_columns_that_change_hands(steps):
    assert not any(_stale(steps, True, seed) for seed in range(300))


def test_one_half_copied_into_the_second_accumulator_goes_stale():
    """What nothing holds back at one step; at two the wait for the second accumulator does."""
    assert any(_stale(1, False, seed) for seed in range(300))
    assert not any(_stale(2, False, seed) for seed in range(300))


def test_the_kernel_folds_two_halves_only():
    """The kernel is the model's: it folds, and takes both accumulators for one unit, above one step of depth."""
    code = _body(_code("experts.cu"), r"experts_kernel\(const __grid_constant__")
    assert re.search(r"const bool halves = HALVES && a\.depth > kDepth;", code)
    assert len(re.findall(r"if \(!halves\) acc \^= 1;\s*if \(acc == 0\) aph \^= 1u;", code)) == 2
    assert re.search(r"if \(halves\) \{\s*fold_halves\(", code) and code.count("fold_halves(") == 1
    assert "const int half = halves ? second_half(w.steps) : -1;" in code
    assert "give_back(halves ? 1 : acc);" in code
