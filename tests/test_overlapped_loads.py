"""Kernels that launch_overlapped starts may live while the kernel before them still
writes: what they read is not constant for their lifetime, so the read-only load
path (__ldg, ld.global.nc, pointers promised not to alias) is closed to them. The
embedding table is a weight, which no kernel writes."""

import os
import re

import fine_grained_moe_gb300 as fgm

CSRC = os.path.join(os.path.dirname(fgm.__file__), "csrc")


def units_that_overlap():
    """Sources of every translation unit that calls launch_overlapped, with the headers they include."""
    seen = set()

    def take(name):
        path = os.path.join(CSRC, name)
        if name in seen or not os.path.exists(path):
            return
        seen.add(name)
        for inc in re.findall(r'#include "([^"]+)"', open(path).read()):
            take(inc)
    for f in sorted(os.listdir(CSRC)):
        if f.endswith(".cu") and "launch_overlapped(" in open(os.path.join(CSRC, f)).read():
            take(f)
    return {f: open(os.path.join(CSRC, f)).read() for f in sorted(seen)}


def test_the_units_are_found():
    assert {"kv_append.cuh", "kv_attn.cuh", "logprobs.cuh", "lm_score.cuh"} <= set(units_that_overlap())


def test_no_read_only_loads_but_of_weights():
    for name, text in units_that_overlap().items():
        code = re.sub(r"//[^\n]*", "", text)
        for load in re.findall(r"__ldg\(([^;]*);", code):
            assert load.startswith("er[j]"), f"{name}: __ldg({load}"      # a word's row of the embedding
        assert not re.search(r"\.nc\b|__restrict__|__ldlu|__nv_ldg", code), name


def test_tensor_memory_is_taken_behind_the_wait():
    """A kernel that holds tensor memory while it waits for the one before it to end
    would hang with one that lets it start before taking its own."""
    found = 0
    for name, text in units_that_overlap().items():
        code = re.sub(r"//[^\n]*", "", text)
        if "tcgen05.alloc" in code and "griddepcontrol.wait" in code:
            for kernel in code.split("__global__")[1:]:
                if "tcgen05.alloc" in kernel:
                    found += 1
                    assert kernel.index("griddepcontrol.wait") < kernel.index("tcgen05.alloc"), name
    assert found == 2
