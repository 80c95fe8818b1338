"""The end of a CTA pair's copies (csrc/pair_copies.h) against a model of the pair:
two CTAs that issue copies into a ring on one set of barriers, the products that
free a stage, waits that run out at any point, and copies that land when they like.
The kernel leaves when the barriers' phases that pair_end names are complete; no
copy may land after that. (On a GPU the case needs a wait that runs out, which no
test forces.)"""

import ctypes
import random
import shutil
import subprocess

import pytest

import os

import fine_grained_moe_gb300 as fgm

CSRC = os.path.join(os.path.dirname(fgm.__file__), "csrc")


@pytest.fixture(scope="module")
def pair_end(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("pair")
    (d / "p.cpp").write_text('#include "pair_copies.h"\nextern "C" void pair_end(uint32_t a, uint32_t b, uint32_t s, uint32_t *o)\n'
                             "{ fgm::score::PairEnd e = fgm::score::pair_end(a, b, s); o[0] = e.first; o[1] = e.only_from; o[2] = e.to; }\n")
    subprocess.run(["g++", "-O1", "-shared", "-fPIC", "-I", CSRC, "-o", str(d / "p.so"), str(d / "p.cpp")], check=True)
    f = ctypes.CDLL(str(d / "p.so")).pair_end

    def call(a, b, s):
        o = (ctypes.c_uint32 * 3)()
        f(a, b, s, o)
        return tuple(o)
    return call


class Barrier:
    """One arrival and a byte count to a phase; bytes may land before they are expected."""

    def __init__(self):
        self.phase, self.arrived, self.bytes = 0, False, 0

    def settle(self):
        if self.arrived and self.bytes == 0:
            self.phase, self.arrived = self.phase + 1, False

    def arrive(self, expect):
        assert not self.arrived, "a second arrival in a phase"
        self.arrived = True
        self.bytes += expect
        self.settle()

    def land(self, n):
        self.bytes -= n
        self.settle()


def size(n, r):
    """Bytes of a CTA's n-th copy (fewer where it has no rows to copy)."""
    return 48 if r == 0 or n % 7 < 4 else 32


def run(pair_end, rng, total, stages):
    """One run; returns what was still in flight when the kernel left, how far the
    CTAs were apart, and whether it waited for what nobody issued."""
    full = [Barrier() for _ in range(stages)]
    issued, alive, done, consumer = [0, 0], [True, True], 0, True      # done: copies whose products are through
    flying = []
    give_up = rng.random() < 0.8

    def issue(r):
        n = issued[r]
        if n >= total or n - stages >= done:       # nothing left, or the stage is not free yet
            return False
        if r == 0:
            full[n % stages].arrive(size(n, 0) + size(n, 1))
        flying.append((n, size(n, r)))
        issued[r] += 1
        return True

    for _ in range(rng.randint(0, 40 * total)):     # (then every wait that is left runs out)
        what = rng.random()
        if what < 0.5:
            r = rng.randrange(2)
            if alive[r] and not issue(r) and issued[r] < total and give_up and rng.random() < 0.05:
                alive[r] = False
        elif what < 0.75 and flying:
            n, b = flying.pop(rng.randrange(len(flying)))
            full[n % stages].land(b)
        elif consumer:
            if done < total and full[done % stages].phase > done // stages:
                done += 1
            elif give_up and rng.random() < 0.02:
                consumer = False
        if give_up and rng.random() < 0.01:
            alive[rng.randrange(2)] = False
    first, only_from, to = pair_end(issued[0], issued[1], stages)
    for n in range(only_from, to):
        assert full[n % stages].phase == n // stages, "makes up for the wrong phase"
        if n < issued[0]:
            full[n % stages].land(size(n, 1))
        else:
            full[n % stages].arrive(size(n, 1))
    # the rest lands in any order; the kernel leaves as soon as the phases are complete
    rng.shuffle(flying)
    while not all(full[n % stages].phase > n // stages for n in range(first, to)):
        if not flying:
            return 0, issued[1] - issued[0], True
        n, b = flying.pop()
        full[n % stages].land(b)
    return len(flying), issued[1] - issued[0], False


def test_no_copy_outlives_the_pair(pair_end):
    rng = random.Random(7)
    apart = set()
    for _ in range(3000):
        left, d, stuck = run(pair_end, rng, rng.randint(1, 40), rng.choice([1, 2, 3, 6, 12]))
        assert left == 0 and not stuck
        apart.add(d)
    assert min(apart) < 0 < max(apart) and 0 in apart      # either CTA ahead, and neither


def test_the_model_sees_a_count_of_one_cta_alone(pair_end):
    """Waiting for the first CTA's copies only, as counted there, leaves some of the
    second's in flight, or waits for what the second never issued."""
    rng = random.Random(7)
    ends = [run(lambda a, b, s: pair_end(a, a, s), rng, rng.randint(1, 40), rng.choice([1, 2, 3, 6, 12])) for _ in range(3000)]
    assert max(e[0] for e in ends) > 0 and any(e[2] for e in ends)


@pytest.mark.parametrize("a,b,s,want", [(0, 0, 3, (0, 0, 0)), (5, 5, 3, (2, 5, 5)), (2, 4, 3, (1, 2, 4)), (7, 4, 12, (0, 4, 7))])
def test_ends(pair_end, a, b, s, want):
    assert pair_end(a, b, s) == want
