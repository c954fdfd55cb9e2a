"""The order in which the scans' warps hand tiles over, as a model on the CPU:
computing warps and the two control warps of a CTA take turns in any order, and
no warp may read another tile's state or wait on a phase that is gone.  The
numbers of tiles ahead and of slots are read from the kernels' source."""
import os
import random
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = open(os.path.join(ROOT, "nonlinear_rnn_newton_b200", "csrc", "glr.cuh")).read()


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def passed(self, parity):
        return (self.phase & 1) != parity


def run(tiles, slots, ahead, stages, stages_back, warps, rng):
    """One CTA over its tiles, a random schedule.  stages_back: a stage is given
    back when its tile has been run through (adjoint), else when folded (scan).
    Returns the wrong reads and whether anyone was left waiting."""
    sets = ahead + 1
    full, empty = [Barrier(1) for _ in range(stages)], [Barrier(warps) for _ in range(stages)]
    folded, entered = [Barrier(warps) for _ in range(sets)], [Barrier(1) for _ in range(slots)]
    passed = [Barrier(1), Barrier(1)]
    enter, maps, own, held = [[None] * warps for _ in range(slots)], [[None] * warps for _ in range(sets)], [None, None], {}
    wrong = []

    def load(n):
        held[n % stages] = n
        full[n % stages].arrive()

    def wait(barrier, turn):
        while not barrier.passed(turn & 1):
            yield

    def computing(w):
        def fold(n):
            yield from wait(full[n % stages], n // stages)
            if held[n % stages] != n:
                wrong.append(("stage", n))
            maps[n % sets][w] = n
            yield
            folded[n % sets].arrive()
            yield

        for n in range(min(ahead, tiles)):
            yield from fold(n)
        for n in range(tiles):
            if n + ahead < tiles:
                yield from fold(n + ahead)
            yield from wait(entered[n % slots], n // slots)
            yield
            if enter[n % slots][w] != n:
                wrong.append(("state", n, enter[n % slots][w]))
            if stages_back and held[n % stages] != n:
                wrong.append(("stage", n))
            yield
            empty[n % stages].arrive()
            yield

    def control(first):
        for n in range(first, tiles, 2):
            yield from wait(folded[n % sets], n // sets)
            if stages_back:
                if n >= ahead and n - ahead + stages < tiles:
                    yield from wait(empty[(n - ahead) % stages], (n - ahead) // stages)
                    load(n - ahead + stages)
            elif n + stages < tiles:
                load(n + stages)
            yield
            if n > 0:
                yield from wait(passed[(n - 1) & 1], (n - 1) >> 1)
                if own[(n - 1) & 1] != n - 1:
                    wrong.append(("own", n))
            for w in range(warps):
                enter[n % slots][w] = n
                yield
                if maps[n % sets][w] != n:
                    wrong.append(("map", n))
            own[n & 1] = n
            passed[n & 1].arrive()
            yield
            entered[n % slots].arrive()
            yield

    for n in range(min(tiles, stages)):
        load(n)
    live = [computing(w) for w in range(warps)] + [control(0), control(1)]
    speed = [rng.choice([1, 1, 5, 40]) for _ in live]
    for _ in range(20000):
        if not live or wrong:
            break
        i = rng.choices(range(len(live)), speed)[0]
        try:
            next(live[i])
        except StopIteration:
            del live[i], speed[i]
    return wrong, bool(live)


def layout(name):
    """(tiles ahead, stages, slots of the entering states) of a kernel."""
    body = re.search(r"struct " + name + r" \{(.*?)\n\};", SOURCE, re.S).group(1)
    ahead = int(re.search(r"kAhead = (\d+)", body).group(1))
    assert "kSets = kAhead + 1" in body
    slots = re.search(r"float2 enter\[(\w+)\]", SOURCE).group(1)
    assert re.search(r"entered\[" + slots + r"\]", SOURCE)
    return ahead, int(re.search(r"kStages = (\d+)", body).group(1)), ahead + 1 if slots == "NS" else int(slots)


@pytest.mark.parametrize("name,stages_back", [("GlrScanLayout", False), ("GlrAdjointLayout", True)])
def test_handover_in_any_order(name, stages_back):
    ahead, stages, slots = layout(name)
    for seed in range(400):
        rng = random.Random(seed)
        tiles = rng.randrange(1, 13)
        wrong, waiting = run(tiles, slots, ahead, stages, stages_back, 3, rng)
        assert not wrong and not waiting, (seed, tiles, wrong)


def test_the_model_finds_too_few_slots():
    """Two slots behind two tiles ahead: a late warp reads the state of a later tile, or waits for ever."""
    found = [run(6, 2, 2, 5, True, 3, random.Random(seed)) for seed in range(400)]
    assert any(wrong for wrong, _ in found) and any(waiting for _, waiting in found)
