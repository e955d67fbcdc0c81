"""The input ring of the layer's tensor-core kernel, modelled: a producer, loads that land
in any order, transform teams that take the chunks in turn, and the MMA issue, with barriers
whose waits see a phase's parity alone.  No wait may let a role pass before its own phase is
complete, whatever the order of events, and every run must end.

The roles' waits are those of csrc/tc_fwd.cuh: the producer on empty (the phase before), a
team on empty (the phase before) where the ring is odd and two teams share it, then on full,
the MMA issue on tready.
"""

import random

import pytest


class Bar:
    """An mbarrier: phases complete after ``count`` arrivals; a wait tests a parity."""

    def __init__(self, count=1):
        self.count, self.left, self.done = count, count, 0  # done: phases completed

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.done = self.count, self.done + 1

    def passes(self, parity):
        return (self.done - 1) % 2 == parity  # the last completed phase has that parity


def run(stages, teams, chunks, guard, rng):
    """True if every wait passed in its own phase; False at the first that did not."""
    full, tready, empty = ([Bar() for _ in range(stages)] for _ in range(3))
    flying, at = [], {"load": 0, "mma": 0, **{t: t for t in range(teams)}}

    def wait(bar, phase):  # None: not yet; else whether the phase is really complete
        return (bar.done > phase) if bar.passes(phase % 2) else None

    def step(role):
        """What the role does next; None if it waits."""
        c = at[role]
        if c >= chunks:
            return None
        s, k = c % stages, c // stages
        if role == "load":
            ok = wait(empty[s], k - 1)
            if ok:
                flying.append(s)
        elif role == "mma":
            ok = wait(tready[s], k)
            if ok:
                empty[s].arrive()
        else:
            if guard and teams == 2 and stages % 2:
                ok = wait(empty[s], k - 1)
                if not ok:
                    return ok
            ok = wait(full[s], k)
            if ok:
                tready[s].arrive()
        if ok:
            at[role] = c + (teams if isinstance(role, int) else 1)
        return ok

    idle = 0
    roles = list(at)
    while at["mma"] < chunks:
        if flying and rng.random() < 0.4:
            full[flying.pop(rng.randrange(len(flying)))].arrive()
            idle = 0
            continue
        ok = step(rng.choice(roles))
        if ok is False:
            return False
        idle = 0 if ok else idle + 1
        assert idle < 10000, "a role waits for ever"
    return True


@pytest.mark.parametrize("teams", [1, 2])
@pytest.mark.parametrize("stages", range(2, 9))
def test_no_wait_passes_early(stages, teams):
    rng = random.Random(stages * 10 + teams)
    assert all(run(stages, teams, rng.randint(1, 40), True, rng) for _ in range(400))


@pytest.mark.parametrize("stages", [3, 5])
def test_the_model_sees_a_missing_wait(stages):
    rng = random.Random(stages)
    assert not all(run(stages, 2, 40, False, rng) for _ in range(400))
