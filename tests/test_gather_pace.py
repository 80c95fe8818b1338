"""Warps that gather rows into a ring of stages (csrc/grouped.cuh), modelled: a barrier's
wait tells phases apart by their parity alone, so a warp must not fall two of them
behind. One that has rows in a tile cannot, as the products wait for its copies; one
that has none can, and must not go by the barriers there. And the code keeps to that."""

import os
import random
import re

import fine_grained_moe_gb300 as fgm

CSRC = os.path.join(os.path.dirname(fgm.__file__), "csrc")


def run(rng, skips, stages, tiles, lazy):
    """The weights' warp (0) and a warp of rows (1) that has some in only some tiles; the products free a stage when
    both have copied for it. skips: the second leaves tiles without rows out. Returns whether all stages passed."""
    has = [rng.random() < 0.5 for _ in range(tiles)]
    steps = [rng.randint(1, 3 * stages) for _ in range(tiles)]
    rows = [h for h, s in zip(has, steps) for _ in range(s)]         # whether warp 1 has rows in a stage
    free = [0] * stages                                              # completed phases of each place
    copied, done, passed, left = [0, 0], 0, 0, False                 # stages each has gone through; products; what warp 0 found free

    def seems_free(n):
        return n < stages or (free[n % stages] - 1) & 1 == (n // stages - 1) & 1

    idle = 0
    while idle < 100:
        idle += 1
        who = 2 if rng.random() < 0.4 else int(rng.random() < (lazy if idle < 50 else 0.5))
        if who == 2:
            if done < copied[0] and (not rows[done] or done < copied[1]):
                free[done % stages] += 1
                done, idle = done + 1, 0
            continue
        n = copied[who]
        if n == len(rows):
            continue
        if who == 1 and skips and not rows[n]:
            copied[1], left, idle = n + 1, True, 0
            continue
        if passed > n if who == 1 and left else seems_free(n):
            left = left and who != 1
            if who == 0:
                passed = n + 1
            if who == 0 or rows[n]:
                assert n < stages or done > n - stages, "a copy into a stage in use"
            copied[who], idle = n + 1, 0
    return done == len(rows)


def test_warps_without_rows_follow_the_weights():
    rng = random.Random(5)
    assert all(run(rng, True, rng.randint(1, 12), rng.randint(1, 12), lazy) for lazy in (0.5, 0.1, 0.01, 0.99) for _ in range(500))


def test_the_model_sees_a_warp_that_falls_behind():
    rng = random.Random(5)
    assert not all(run(rng, False, rng.randint(1, 12), rng.randint(1, 12), 0.01) for _ in range(500))


def test_the_code_leaves_such_tiles_out():
    code = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "grouped.cuh")).read())
    gather = code[code.index("if (p.src) {"):code.index("copy_gathered(ring")]
    skip, back, wait = (gather.index(s) for s in ("place.skip(steps, stages)", "wait.passed(&sh.passed, n", "wait(&sh.empty[place.slot]"))
    assert skip < back < wait
