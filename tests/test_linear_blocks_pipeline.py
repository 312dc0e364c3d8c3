"""Host-side model of the accumulators' round in moe_w4a16_linear_blocks.

Per K chunk the multiplying warp issues MMAs into the next of `accs`
accumulators and commits; every adding warp of every CTA reads that chunk's
accumulator and hands it back.  The last chunk's of a tile is kept for the sums
and handed back only when the tile is finished.  MMAs finish in order, at any
time after they are issued.  Random interleavings are run; a warp may stop, and
the others' waits then run out, at any moment (pace) or once nothing else
moves.  The model checks that no accumulator is written before every adder has
read and released it, that a tile's sums are of its own chunks in order, that
everything ends, and that no MMA is in flight at the end.
"""
import random

import pytest


def run(ctas, warps, tiles, nk, accs, stop, seed):
    """(chunks added up per warp, MMAs in flight at the end)"""
    rnd = random.Random(seed)
    total = tiles * nk
    adders = [(c, w) for c in range(ctas) for w in range(warps)]
    released = [0] * accs                 # arrivals of the accumulator's barrier, over all phases
    need = len(adders)
    issued = done = 0
    holds = [None] * accs                 # the chunk in an accumulator
    readers = [set() for _ in range(accs)]
    state = {a: ["wait", 0] for a in adders}   # wait for chunk i / finish a tile / end
    added = {a: [] for a in adders}
    mul = "run"
    while True:
        steps, late = [], []              # late: waits that could run out
        if done < issued:
            steps.append(("mma done",))
        if mul == "run":
            k, slot = issued, issued % accs
            if k == total or stop == ("mul", k):
                steps.append(("mul close",))
            elif k < accs or released[slot] >= need * (k // accs):
                steps.append(("issue",))
            else:
                late.append(("mul close",))
        elif mul == "close" and done == issued:
            steps.append(("mul end",))    # waits for the MMAs it issued
        for a in adders:
            what, i = state[a]
            if what == "wait":
                if i == total or stop == (a, i):
                    steps.append(("add end", a))
                elif done > i:
                    steps.append(("read", a))
                else:
                    late.append(("add end", a))
            elif what == "finish":
                steps.append(("finish", a))
        if not steps and not late:
            break
        stopped = stop is not None
        step = rnd.choice(steps) if steps and not (stopped and late and rnd.random() < 0.02) else rnd.choice(late)
        if step[0] == "mma done":
            done += 1
        elif step[0] == "issue":
            slot = issued % accs
            assert holds[slot] is None or len(readers[slot]) == need, "written before it was read"
            holds[slot], readers[slot] = issued, set()
            issued += 1
        elif step[0] == "mul close":
            mul = "close"
        elif step[0] == "mul end":
            mul = "end"
        elif step[0] == "add end":
            state[step[1]] = ["end", 0]
        elif step[0] == "read":
            a = step[1]
            i = state[a][1]
            assert holds[i % accs] == i, "another chunk's sums"
            added[a].append(i)
            if (i + 1) % nk == 0:
                state[a] = ["finish", i]
            else:
                readers[i % accs].add(a)
                released[i % accs] += 1
                state[a] = ["wait", i + 1]
        elif step[0] == "finish":         # reads the sums back from the accumulator, then hands it back
            a = step[1]
            i = state[a][1]
            assert holds[i % accs] == i, "the sums were written over"
            readers[i % accs].add(a)
            released[i % accs] += 1
            state[a] = ["wait", i + 1]
    assert mul == "end" and all(s[0] == "end" for s in state.values())
    return added, issued - done


@pytest.mark.parametrize("ctas,warps", [(1, 4), (2, 3)])
@pytest.mark.parametrize("accs", [2, 4])
@pytest.mark.parametrize("tiles,nk", [(1, 1), (5, 1), (3, 2), (2, 3), (2, 7), (1, 9)])
def test_every_chunk_is_added_once(ctas, warps, accs, tiles, nk):
    for seed in range(40):
        added, left = run(ctas, warps, tiles, nk, accs, None, seed)
        assert left == 0 and all(v == list(range(tiles * nk)) for v in added.values())


@pytest.mark.parametrize("accs", [2, 4])
@pytest.mark.parametrize("tiles,nk", [(4, 1), (2, 5)])
@pytest.mark.parametrize("who", ["mul", (0, 0), (1, 2)])
@pytest.mark.parametrize("at", [0, 1, 3])
def test_a_warp_that_stops_leaves_nothing_behind(accs, tiles, nk, who, at):
    for seed in range(40):
        added, left = run(2, 3, tiles, nk, accs, (who, at), seed)
        assert left == 0 and all(v == list(range(len(v))) for v in added.values())
