"""The paged form's producers, checked on the host (no GPU).

Several producer warps share out a key tile's copies; each waits, before the loads of group g (V_{g-3} and
K_g), for the score commit of group g - kStages / 2, which frees their ring slots.  Commits rotate over six
barriers, waited for by parity.  This module restates the rules (as test_pipeline_protocol does for the
contiguous producer) and checks that (1) that commit is never earlier than the groups that consumed the
slots' last tiles, and is itself free of deadlock, (2) under random interleavings a producer that
issues at least one copy of every tile never finds a barrier two phases ahead of the one it waits for, and
(3) a warp that issued none could, which is why such warps take no part."""
import numpy as np
import pytest

from test_pipeline_protocol import K_SCOMMITS, group_of_load


def first_waiting_group(stages):
    """The first group whose second load reuses a ring slot: loads 2 g - 3 and 2 g - 2."""
    return next(g for g in range(3, 100) if 2 * g - 2 >= stages)


@pytest.mark.parametrize("stages", [6, 10])
def test_commit_covers_both_ring_slots(stages):
    g0 = first_waiting_group(stages)
    assert g0 - stages // 2 == 1  # the producer's counter starts at group 1
    for g in range(g0, 2000):
        waited = g - stages // 2
        for load in (2 * g - 3, 2 * g - 2):
            if load >= stages:
                assert group_of_load(load - stages) <= waited
        assert waited < g - 1  # issued two groups before: no wait for what is still to be loaded
    for g in range(g0):  # groups before it reuse no slot
        assert (g if g < 3 else 2 * g - 2) < stages


def simulate(stages, groups, issues, rng):
    """One CTA.  issues[w]: whether producer w has a copy of every tile.  Returns the largest number of
    phases that a waited-for barrier was ahead (1: the phase waited for; 2: it would be missed)."""
    done = 0                      # groups whose score commit has arrived
    at = [0] * len(issues)        # next group of each producer
    worst = 0
    start = first_waiting_group(stages)

    def phases(barrier):          # completed phases of a commit barrier
        return (done - barrier + K_SCOMMITS - 1) // K_SCOMMITS

    while done < groups or min(at) < groups:
        moves = []
        if done < groups and all(a > done for a, i in zip(at, issues) if i):
            moves.append(-1)
        for w, g in enumerate(at):
            if g < groups and (g < start or done > g - stages // 2):
                moves.append(w)
        assert moves, "deadlock"
        m = moves[rng.integers(len(moves))] if rng.random() < 0.5 else moves[0]
        if m < 0:
            done += 1
            continue
        g = at[m]
        if g >= start:
            waited = g - stages // 2
            worst = max(worst, phases(waited % K_SCOMMITS) - waited // K_SCOMMITS)
        at[m] += 1
    return worst


@pytest.mark.parametrize("stages", [6, 10])
@pytest.mark.parametrize("producers", [1, 2, 3])
def test_issuing_producers_stay_within_the_phase(stages, producers):
    for seed in range(60):
        assert simulate(stages, 80, [True] * producers, np.random.default_rng(seed)) <= 1


@pytest.mark.parametrize("stages", [6, 10])
def test_a_producer_without_copies_could_fall_behind(stages):
    assert max(simulate(stages, 80, [True, False], np.random.default_rng(seed)) for seed in range(60)) >= 2
