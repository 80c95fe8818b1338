"""What include/fgm.h promises of bf16 activations as two E4M3 terms, for every bf16 element
under every largest element of a row: the steps of csrc/moe_rows.cuh in plain torch. (Powers
of two of the row do not matter: rows whose largest element lies in [128, 256).)"""

import os
import re

import torch

import fine_grained_moe_gb300 as fgm

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(fgm.__file__))), "include", "fgm.h")


def promise():
    text = re.sub(r"\s*\*\s+", " ", open(HEADER).read())
    m = re.search(r"x enters exactly where an element is 2\^-(\d+) of its row's largest or more, the others to 2\^-(\d+) of that", text)
    return 2.0 ** -int(m.group(1)), 2.0 ** -int(m.group(2))


def e4m3(v):
    return v.to(torch.float8_e4m3fn).float()


def test_every_element_of_every_row():
    exact, error = promise()
    v = torch.arange(1, 0x4380, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()      # all below 256
    v = v[v >= 2.0 ** -40]
    t1 = e4m3(v)
    off = (v - t1 - e4m3(v - t1)).abs()
    worst = 0.0
    for m in range(128):
        largest = 128.0 + m
        in_row = v <= largest
        assert (off[in_row & (v >= exact * largest)] == 0).all(), largest
        assert (off[in_row] <= error * largest).all(), largest
        worst = max(worst, float((off[in_row] / largest).max()))
    assert worst == error                           # and no tighter one holds
    assert any((off[(v >= exact / 2 * m) & (v <= m)] != 0).any() for m in range(128, 256))
