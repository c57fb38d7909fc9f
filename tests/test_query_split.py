"""A query as the sum of two e4m3 numbers (attention of large trees on the 8-bit cache): what that loses, over every significand
a bf16 can have, and that the header says so."""
import os
import re

import numpy as np

from oracle import fp8_cache as fc

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "pkv.h")


def e4m3(x):
    return fc.E4M3[fc.round_e4m3(x)]


def test_two_parts():
    significands = 1 + np.arange(128) / 128
    y = np.concatenate([[0.0], *[significands * 2.0 ** e for e in range(-14, 8)]])      # bf16, the row's largest in [128, 256)
    high = e4m3(y)
    off = np.abs(y - (high + e4m3(y - high)))
    exact, worst = 0.0, 0.0                            # of the largest: from where on all are exact, and the most any is off
    for largest in 128 * significands:
        here = y <= largest
        worst = max(worst, off[here].max() / largest)
        exact = max(exact, y[here & (off > 0)].max() / largest)
    assert worst == 2.0 ** -17
    assert 2.0 ** -9 * (1 - 2.0 ** -7) <= exact < 2.0 ** -9
    assert np.array_equal(e4m3(-y), -high)             # either sign alike


def test_the_header_says_so():
    with open(HEADER) as f:
        text = re.sub(r"\s*\n \* ?", " ", f.read())
    said = re.search(r"split into two e4m3 parts, exact from 2\^-(\d+) of the row's largest element and off by at most 2\^-(\d+) of it", text)
    assert said and said.groups() == ("9", "17")
