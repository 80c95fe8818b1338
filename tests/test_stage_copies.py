"""The end of the copies of a CTA pair whose warps bring parts of a stage (weights and
rows, csrc/grouped.cuh), counted as in csrc/pair_copies.h, against a model: warps that
stop at any stage, products that free a stage, copies that land when they like. The
kernel leaves when the phases that are left are complete; no copy may land after that.
(On a GPU the case needs a wait that runs out, which no test forces.)"""

import ctypes
import os
import random
import shutil
import subprocess

import pytest

import fine_grained_moe_gb300 as fgm
from test_pair_copies import Barrier

CSRC = os.path.join(os.path.dirname(fgm.__file__), "csrc")


@pytest.fixture(scope="module")
def count(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("stage")
    (d / "p.cpp").write_text(
        '#include "pair_copies.h"\nusing namespace fgm::score;\n'
        'extern "C" void left(const uint32_t *issued, int n, uint32_t stages, uint32_t *o)\n'
        "{ StagesLeft l; for (int i = 0; i < n; ++i) l.warp(issued[i]); o[0] = l.first(stages); o[1] = l.to; }\n"
        'extern "C" uint32_t sent(uint32_t first, uint32_t bytes, uint32_t steps, uint32_t issued, uint32_t n)\n'
        "{ return sent_bytes({first, bytes}, steps, issued, n); }\n")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, "-o", str(d / "p.so"), str(d / "p.cpp")], check=True)
    lib = ctypes.CDLL(str(d / "p.so"))
    lib.sent.restype = ctypes.c_uint32

    def left(issued, stages):
        o = (ctypes.c_uint32 * 2)()
        lib.left((ctypes.c_uint32 * len(issued))(*issued), len(issued), stages, o)
        return tuple(o)
    return left, lib.sent


NOTES = 12             # tiles that a warp's notes hold, and the longest ring


def size(tile, w):
    """Bytes of warp w's copies for a stage of a tile: weights alike in both CTAs, rows by the tile (none in some)."""
    return 64 if w < 2 else (tile * 7 + w // 2 * 5) % 4 * 16


def run(count, rng, total, stages, steps, warps, by_weights=False):
    """Warps 0 and 1 bring the CTAs' weights, the others rows in turn of the CTAs, for tiles of `steps` stages. Returns
    what was in flight when the kernel left, whether it waited for what nobody sent, and how far the warps were apart."""
    left, sent = count
    full = [Barrier() for _ in range(stages)]
    at, alive, done, consumer = [0] * warps, [True] * warps, 0, True      # at: the stage that a warp is at
    issued = [0] * warps                                         # and how far it has copied
    notes = [[(0xFFFFFFFF, 0)] * NOTES for _ in range(warps)]
    flying = []
    named = lambda n: sum(size(n // steps, w) for w in range(warps))      # noqa: E731
    give_up = rng.random() < 0.9
    for _ in range(rng.randint(0, 30 * total * warps)):          # (then every wait that is left runs out)
        what = rng.random()
        if what < 0.6:
            w = rng.randrange(warps)
            n = at[w]
            b = size(n // steps, w)
            if alive[w] and n < total and b == 0:                # (no rows: nothing to wait for)
                at[w] += steps
            elif alive[w] and n < total and n - stages < done:
                if w == 0:
                    full[n % stages].arrive(named(n))
                flying.append((n, b))
                if n % steps == 0:
                    notes[w][n // steps % NOTES] = (n, b)
                at[w] = issued[w] = n + 1
            elif give_up and rng.random() < 0.05:
                alive[w] = False
        elif what < 0.85 and flying:
            n, b = flying.pop(rng.randrange(len(flying)))
            full[n % stages].land(b)
        elif consumer:
            if done < total and full[done % stages].phase > done // stages:
                done += 1
            elif give_up and rng.random() < 0.02:
                consumer = False
        if give_up and rng.random() < 0.02:
            alive[rng.randrange(warps)] = False
    first, to = left(issued[:2] if by_weights else issued, stages)
    for n in range(first, to):
        if by_weights and min(issued[:2]) > n:                   # (a stage that both CTAs' weights were copied for counts as whole)
            continue
        total_sent = 64 * ((n < issued[0]) + (n < issued[1]))
        total_sent += sum(sent(*note, steps, issued[w], n) for w in range(2, warps) for note in notes[w])
        if n >= issued[0]:
            assert full[n % stages].phase == n // stages, "arrives in the wrong phase"
            full[n % stages].arrive(total_sent)
        elif total_sent != named(n):
            assert full[n % stages].phase == n // stages, "makes up for the wrong phase"
            full[n % stages].land(named(n) - total_sent)
    rng.shuffle(flying)
    while not all(full[n % stages].phase > n // stages for n in range(first, to)):
        if not flying:
            return 0, True, max(issued) - min(issued)
        n, b = flying.pop()
        full[n % stages].land(b)
    return len(flying), False, max(issued) - min(issued)


@pytest.mark.parametrize("warps", [4, 14])          # rows by a warp of each CTA, and gathered by six
def test_no_copy_outlives_the_pair(count, warps):
    rng = random.Random(warps)
    apart = set()
    for _ in range(1500):
        steps = rng.choice([1, 1, 2, 3, 5, 15, 22])
        flying, stuck, d = run(count, rng, steps * rng.randint(1, 30 // steps), rng.choice([1, 2, 4, 8, 12]), steps, warps)
        assert flying == 0 and not stuck
        apart.add(d)
    assert 0 in apart and 12 in apart               # all together, and as far apart as the longest ring allows


@pytest.mark.parametrize("warps", [4, 14])
def test_the_model_sees_a_count_of_weights_alone(count, warps):
    """Going by the weights' copies leaves rows in flight, or waits for rows that nobody sent."""
    rng = random.Random(warps)
    ends = [run(count, rng, 2 * rng.randint(1, 15), rng.choice([1, 2, 4, 8, 12]), 2, warps, True) for _ in range(1500)]
    assert any(e[0] for e in ends) and any(e[1] for e in ends)
