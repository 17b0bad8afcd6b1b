"""The ring of packed tiles that a step of many rows over a 4-bit cache fills by TMA and
empties with two groups of warps, on the host: a model of its barriers over the kernel's own
order of items, slots and parities (mha_debug_q4_ring), with copies that land in any order."""
import random

import numpy as np
import pytest

from tests.test_cache_host import lib  # noqa: F401


def ring_of(lib, slots, tiles):  # noqa: F811
    loads, keys, values = (np.full((n, w), -1, dtype=np.int32) for n, w in ((2 * tiles, 4), (tiles, 3), (tiles, 3)))
    lib.mha_debug_q4_ring(slots, tiles, *(a.ctypes.data for a in (loads, keys, values)))
    return loads.tolist(), (keys.tolist(), values.tolist())


def run(slots, tiles, loads, waits, rng):
    """One schedule.  A copy is issued in order, into a slot whose last item is emptied, and
    lands at any later time.  A group's wait passes when the phase of its parity is the one
    before the barrier's current one.  Keys of tile t are unpacked when the scores of t - 2 are
    formed, which come behind the products of t - 4; values of t when the products of t - 2
    are, which come behind the scores of t - 1.  Copies land late as a rule, so that warps
    run into every wait as early as they can."""
    issued, landed, emptied = 0, set(), set()
    phases = {}                                  # completed, of each barrier
    done, passed = [0, 0], [False, False]
    late = {x: rng.random() for x in range(2 * tiles)}
    while min(done) < tiles:
        actions = []
        if issued < 2 * tiles and (issued < slots or issued - slots in emptied):
            actions.append("issue")
        for group in (0, 1):
            t = done[group]
            if t == tiles:
                continue
            _, bar, parity = waits[group][t]
            if passed[group]:
                if done[1 - group] >= (t - 3 if group == 0 else min(tiles, t)):
                    actions.append(("finish", group))
            elif phases.get(bar, 0) & 1 != parity:
                actions.append(("pass", group))
        flying = [x for x in range(issued) if x not in landed]
        if not actions or rng.random() < 0.1:
            assert actions or flying, "nothing can go on"
            if flying:
                x = max(flying, key=lambda y: late[y])
                landed.add(x)
                phases[loads[x][3]] = phases.get(loads[x][3], 0) + 1
                continue
        action = rng.choice(actions)
        if action == "issue":
            issued += 1
        elif action[0] == "pass":
            group = action[1]
            item = waits[group][done[group]][0]
            assert item in landed, f"{'kv'[group]}{done[group]} passes before item {item} has landed"
            assert max(x for x in range(issued) if loads[x][0] == loads[item][0]) == item, "the slot holds another item"
            passed[group] = True
        else:
            group = action[1]
            emptied.add(waits[group][done[group]][0])
            done[group] += 1
            passed[group] = False
    assert issued == 2 * tiles and len(landed) == issued


@pytest.mark.parametrize("slots", [3, 4, 8])
def test_every_wait_finds_its_item(lib, slots):  # noqa: F811
    for tiles in range(1, 15):
        loads, waits = ring_of(lib, slots, tiles)
        assert sorted((v, t) for _, v, t, _ in loads) == [(v, t) for v in (0, 1) for t in range(tiles)]
        for group in (0, 1):
            for t, (item, bar, parity) in enumerate(waits[group]):
                assert loads[item][1:] == [group, t, bar] and parity in (0, 1)
        rng = random.Random(1000 * slots + tiles)
        for _ in range(150):
            run(slots, tiles, loads, waits, rng)


@pytest.mark.parametrize("slots", [3, 4])
def test_the_model_finds_a_barrier_of_both_groups(lib, slots):  # noqa: F811
    """One barrier to a slot, for both groups' items, lets a group pass early."""
    loads, waits = ring_of(lib, slots, 10)
    loads = [[s, v, t, s] for s, v, t, _ in loads]
    shared = [[[x, x % slots, x // slots & 1] for x, _, _ in group] for group in waits]
    rng = random.Random(slots)
    with pytest.raises(AssertionError, match="passes before"):
        for _ in range(500):
            run(slots, 10, loads, shared, rng)
