"""Host-side model of how the CTAs of moe_w4a16_linear end.

One CTA (up to 64 tokens) or a pair that shares its MMAs: in each CTA a warp
loads chunks into a ring of stages, one warp issues the MMAs of all CTAs and
commits every stage's release, which arrives in each CTA on its own.  Copies
land, MMAs finish (in order) and releases arrive at any time; random
interleavings of these and of the warps' steps are run.  A warp may stop after
some chunks; another's wait on it may then run out: the pipelines' own waits
at any moment (their limit may be short), the closing ones only when nothing
else can happen any more (their limit is a second).

When all warps of all CTAs are through, nothing may be on its way to their
shared memory and no MMA may be in flight.  closing=False is a way to end that
does not hold this: a loading warp that waits for its copies only where it
gave up itself, a multiplying warp that does not wait for its MMAs.
"""
import random

import pytest


def run(ctas, chunks, stages, stop_mma, stop_load, closing, seed):
    """(copies on their way, releases on their way, MMAs in flight) when the CTAs end."""
    rnd = random.Random(seed)
    pace = rnd.random()                   # of the warps beside the copies, MMAs and releases
    issued = [0] * ctas                   # chunks each loading warp has asked for
    copies = set()                        # (cta, chunk) on their way
    mma = 0                               # chunks the MMAs of which are issued
    done = 0                              # .. and finished
    releases = set()                      # (cta, chunk) finished, not yet arrived
    arrived = [set() for _ in range(ctas)]
    load = ["run"] * ctas                 # run -> close -> end
    mul = "run"
    while True:
        engine = [("land", c) for c in copies]
        if done < mma:
            engine.append(("finish",))
        engine += [("release", r) for r in releases]
        steps, late = [], []              # late: waits of a second running out
        for c in range(ctas):
            i = issued[c]
            if load[c] == "run":
                if i == chunks or i == stop_load.get(c, -1):
                    steps.append(("close", c))
                elif i < stages or i - stages in arrived[c]:
                    steps.append(("load", c))
                else:
                    steps.append(("close", c))          # the wait ran out
            elif load[c] == "close":
                last = range(max(0, i - stages), i)     # of each filled stage the last chunk
                if closing:
                    ready = all(j in arrived[c] for j in last)
                else:
                    ready = i == chunks or not any(copy[0] == c for copy in copies)
                (steps if ready else late).append(("end", c))
        if mul == "run":
            if mma == chunks or mma == stop_mma:
                steps.append(("mclose",))
            elif all(issued[c] > mma and (c, mma) not in copies for c in range(ctas)):
                steps.append(("mma",))
            else:
                steps.append(("mclose",))               # the wait ran out
        elif mul == "close":
            (steps if not closing or done == mma else late).append(("mend",))
        normal = stop_mma < 0 and not stop_load         # nobody gives up: no wait runs out
        if normal:
            steps = [s for s in steps if not (s[0] == "close" and issued[s[1]] < chunks) and
                     not (s[0] == "mclose" and mma < chunks)]
        if all(s == "end" for s in load) and mul == "end":
            return len(copies), len(releases), mma - done
        move = rnd.choice(steps if steps and (not engine or rnd.random() < pace) else engine or late)
        kind = move[0]
        if kind == "land":
            copies.remove(move[1])
        elif kind == "finish":
            releases |= {(c, done) for c in range(ctas)}
            done += 1
        elif kind == "release":
            releases.remove(move[1])
            arrived[move[1][0]].add(move[1][1])
        elif kind == "load":
            copies.add((move[1], issued[move[1]]))
            issued[move[1]] += 1
        elif kind == "close":
            load[move[1]] = "close"
        elif kind == "end":
            load[move[1]] = "end"
        elif kind == "mma":
            mma += 1
        else:
            mul = "close" if kind == "mclose" else "end"


STOPS = [(-1, {}), (0, {}), (2, {}), (-1, {0: 2}), (-1, {0: 0}), (-1, {0: 5}), (6, {0: 7})]


@pytest.mark.parametrize("ctas", [1, 2])
@pytest.mark.parametrize("chunks,stages", [(1, 3), (3, 3), (8, 3), (11, 5)])
def test_nothing_is_on_its_way_when_the_ctas_end(ctas, chunks, stages):
    for stop_mma, stop_load in STOPS + [(-1, {1: 2}), (-1, {0: 2, 1: 2})]:
        if any(c >= ctas for c in stop_load):
            continue
        for seed in range(60):
            assert run(ctas, chunks, stages, stop_mma, stop_load, True, seed) == (0, 0, 0)


@pytest.mark.parametrize("ctas", [1, 2])
def test_the_model_sees_a_ring_that_is_left_too_early(ctas):
    normal = [run(ctas, 8, 3, -1, {}, False, seed) for seed in range(200)]
    assert any(r[1] for r in normal)                                   # releases
    stopped = [run(ctas, 3, 3, 1, {}, False, seed) for seed in range(200)]
    assert any(r[0] for r in stopped) and any(r[2] for r in stopped)   # copies, MMAs
