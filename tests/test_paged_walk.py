"""The waits of the paged decode's scoring SM as a model on the host: the warps that load queries and keys, move
the queries and issue the products, over parts of a few tiles, under random schedules.  A barrier shows only the
parity of its phase, so a wait is right only if it passes on the phase that it means, and memory may be
written only when what it held has been read.  The model's waits are those of csrc/paged_tc.cu, by name."""
import random

import pytest

STAGES, GROUPS, MOVERS, BOXES = 2, 3, 4, 9


class Broken(AssertionError):
    pass


class Barrier:
    def __init__(self, arrivals):
        self.arrivals, self.pending, self.done = arrivals, arrivals, 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.done, self.pending = self.done + 1, self.arrivals

    def passes(self, parity):
        return self.done & 1 != parity   # the phase of that parity next to the open one is complete


def wait(bar, phase):
    """Waits for `phase` (-1: passes on a fresh barrier) by its parity, as the hardware can."""
    while not bar.passes(phase & 1):
        yield
    if bar.done != phase + 1:
        raise Broken("phase %d of a barrier that has completed %d" % (phase, bar.done))


def walk(parts, rng, used_stages_only=True, wait_behind=False):
    """`parts`: tiles of each part.  `used_stages_only`: a part completes the phases of the stages that it uses, not
    of both.  `wait_behind`: instead, a one-tile part waits for the other stage's phase behind its load."""
    kfree = [Barrier(MOVERS) for _ in range(STAGES)]
    qfull, qready, qfree = Barrier(1), Barrier(MOVERS), Barrier(2)
    gfull = [[Barrier(1) for _ in range(GROUPS)] for _ in range(STAGES)]
    gempty = [[Barrier(1) for _ in range(GROUPS)] for _ in range(STAGES)]
    box = [None] * BOXES                                       # the part whose queries box j holds
    stage_of_box = [0, 0, 0, 0, None, 1, 1, 1, 1]              # box 4 lies in both
    covers = [[j for j in range(BOXES) if stage_of_box[j] in (s, None)] for s in range(STAGES)]
    late = []                                                  # completions of loads and products, in any order

    def producer(g):
        n, uses = 0, [0] * STAGES
        for part, tiles in enumerate(parts):
            for i in range(tiles):
                s = n & 1
                yield from wait(gempty[s][g], (n >> 1) - 1)
                if i < STAGES:
                    yield from wait(kfree[s], uses[s] if used_stages_only else part)
                    uses[s] += 1
                for j in covers[s]:
                    box[j] = ("keys", n)
                late.append(gfull[s][g].arrive)
                n += 1
                yield
            if wait_behind and tiles < STAGES:
                yield from wait(kfree[n & 1], part)

    def queries():
        for part in range(len(parts)):
            yield from wait(qfree, part - 1)

            def land(part=part):
                box[:] = [part] * BOXES
                qfull.arrive()
            late.append(land)
            yield

    def mover():
        n = 0
        for part, tiles in enumerate(parts):
            yield from wait(qfull, part)
            for j in range(BOXES):
                if box[j] != part:
                    raise Broken("box %d of part %d holds %s" % (j, part, box[j]))
                yield
                if j in (4, 8) and (not used_stages_only or tiles >= STAGES or (n & 1) == (j == 8)):
                    kfree[j == 8].arrive()
            qready.arrive()
            n += tiles

    def issuer(s):
        n = 0
        for part, tiles in enumerate(parts):
            yield from wait(qready, part)
            used = []
            for _ in range(tiles):
                if n & 1 == s:
                    for g in range(GROUPS):
                        yield from wait(gfull[s][g], n >> 1)
                        late.append(gempty[s][g].arrive)
                        used.append(late[-1])
                n += 1

            while any(u in late for u in used):   # a commit completes behind the products in front of it
                yield
            qfree.arrive()

    running = [producer(g) for g in range(GROUPS)] + [queries()] + [mover() for _ in range(MOVERS)] + [issuer(0), issuer(1)]
    weight = [rng.choice([1, 1, 20]) for _ in running] + [rng.choice([1, 20])]
    idle = 0
    while running:
        k = rng.choices(range(len(running) + 1), weight)[0]
        if k == len(running):
            if late:
                late.pop(rng.randrange(len(late)))()
                idle = 0
            continue
        before = len(late)
        try:
            next(running[k])
        except StopIteration:
            del running[k], weight[k]
            idle = 0
        idle = 0 if len(late) != before else idle + 1
        if idle > 5000:
            raise Broken("no progress")


PARTS = [[1] * 12, [1, 2] * 6, [1, 1, 3, 1, 2, 1, 5, 1, 1, 2], [2, 3, 2, 1, 1, 4, 1], [1, 1, 1, 2, 7, 1, 1]]


@pytest.mark.parametrize("parts", PARTS)
def test_every_wait_is_for_its_own_phase(parts):
    for seed in range(40):
        walk(parts, random.Random(seed))


@pytest.mark.parametrize("parts,wait_behind", [(p, False) for p in PARTS] + [(PARTS[0], True)])
def test_a_phase_that_is_not_waited_for_is_found(parts, wait_behind):
    """Where every part completes both stages' phases, the model finds a test that passes a phase early; a wait
    behind the load would come two phases late instead."""
    with pytest.raises(Broken):
        for seed in range(100):
            walk(parts, random.Random(seed), used_stages_only=False, wait_behind=wait_behind)
