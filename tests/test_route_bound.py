"""The bound within which routing sums logits again, against the documented error of an
addition of the tensor pipe."""

import os
import re

import fine_grained_moe_gb300 as fgm
import prompt64 as p64

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(fgm.__file__)))
HIDDEN, CHUNK, STEP = 2816, 256, 16        # elements of K: all, between readings of the accumulator, of one addition


def test_near_logits_are_bounded():
    code = open(os.path.join(ROOT, "fine_grained_moe_gb300", "csrc", "route.cuh")).read()
    header = open(os.path.join(ROOT, "include", "fgm.h")).read()
    add = 2.0 ** -int(re.search(r"each addition within 2\^-(\d+)\s*\*?\s*of a partial sum", header).group(1))
    assert add == p64.ADD
    chunks = HIDDEN // CHUNK
    # a chunk's additions are each within `add` of the chunk's absolute sum; the chunks' sums (also those of a split K,
    # which is cut between chunks) are added in fp32: one rounding a chunk; |x| from fp32 squares: 2^-12 of itself
    worst = (CHUNK // STEP * add + chunks * 2.0 ** -24) * (1 + 2.0 ** -12)
    bound = float.fromhex(re.search(r"kLogitError = (0x[0-9a-fp.-]+)f;", code).group(1))
    assert worst <= bound < 1.1 * worst
    assert re.search(r"gap = [^;]*2\.0f \* \(kLogitError \* ", code)
