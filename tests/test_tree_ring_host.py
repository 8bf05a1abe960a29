"""A model of the key ring of the attention's tile kernel, on the host: three
stages, filled in order by asynchronous copies that may land in any order, and
two consumers that take alternate tiles.  Barriers are the hardware's: a wait
names a phase's parity, and passes when the barrier is in a phase of the other
parity, so it cannot tell a phase from the one two before."""
import random

import pytest

STAGES, INFOS = 3, 8


class Barrier:
    """One arrival a phase (and, for a fill, its bytes)."""

    def __init__(self):
        self.phase, self.arrived, self.bytes = 0, False, 0

    def passes(self, parity):
        return (self.phase & 1) != parity

    def arrive(self, expect=0):
        assert not self.arrived, "an arrival more than the barrier counts"
        self.arrived = True
        self.bytes += expect
        self._turn()

    def land(self, n):
        self.bytes -= n
        self._turn()

    def _turn(self):
        if self.arrived and self.bytes == 0:
            self.phase, self.arrived = self.phase + 1, False


def run(r, tiles, figures_first):
    """One random schedule: true if every consumer found its own tile's keys in
    its stage, false if one did not or a barrier was overrun."""
    full = [Barrier() for _ in range(STAGES)]
    free = [Barrier() for _ in range(STAGES)]
    info = [Barrier() for _ in range(INFOS)]
    holds, flying = [None] * STAGES, []
    slow = r.choice([0.02, 0.2, 1.0])            # how readily a copy lands

    def copier():
        for m in range(tiles):
            while not free[m % STAGES].passes((m // STAGES & 1) ^ 1):
                yield
            full[m % STAGES].arrive(1)
            flying.append(m)
            yield
            info[m % INFOS].arrive()
            yield

    def consumer(first):
        for m in range(first, tiles, 2):
            while figures_first and not info[m % INFOS].passes(m // INFOS & 1):
                yield
            while not full[m % STAGES].passes(m // STAGES & 1):
                yield
            assert holds[m % STAGES] == m, "keys of another tile"
            free[m % STAGES].arrive()
            yield

    roles = [copier(), consumer(0), consumer(1)]
    try:
        while roles:
            role = r.choice(roles)
            try:
                next(role)
            except StopIteration:
                roles.remove(role)
            if flying and r.random() < slow:
                m = flying.pop(r.randrange(len(flying)))
                holds[m % STAGES] = m
                full[m % STAGES].land(1)
    except AssertionError:
        return False
    return True


def test_the_stage_alone_does_not_tell_its_tile():
    r = random.Random(1)
    assert not all(run(r, 12, False) for _ in range(400))


@pytest.mark.parametrize("tiles", [1, 2, 3, 4, 12, 41])
def test_with_the_tiles_figures_every_wait_is_for_its_tile(tiles):
    r = random.Random(tiles)
    assert all(run(r, tiles, True) for _ in range(400))
