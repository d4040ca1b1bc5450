"""How far include/fa.h says that the elements of a 4-bit cache are off, over every rounding
border of the scales."""
import os
import re

import torch

import four_reference as ref

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "fa.h")


def worst(largest):
    """For groups with these largest magnitudes, the largest error of an element at most that
    large, in parts of it: at a border between two numbers, on either side, or the largest."""
    s = ref.scales()[ref.scale_of(largest)]
    u = torch.tensor(ref.U, dtype=torch.float64)
    off = torch.zeros_like(largest)
    for border in [(a + b) / 2 for a, b in zip(ref.U, ref.U[1:])] + [1e9]:
        for near in (1 - 2.0 ** -40, 1, 1 + 2.0 ** -40):
            x = torch.minimum(s * border * near, largest)
            held = torch.where(s > 0, u[ref.nearest((x / s.clamp_min(2.0 ** -17)).clamp_max(6), u)] * s, 0)
            off = torch.maximum(off, (x - held).abs() / largest)
    return off


def test_the_bounds_that_the_header_states():
    text = " ".join(open(HEADER).read().replace("\n *", " ").split())
    m = re.search(r"off by at most ([\d.]+) of its group's largest, by ([\d.]+) where that is below 6 \* 2\^-14, and by 1/3 "
                  r"below 9 \* 2\^-17\. A group whose largest is 6 \* 2\^-18 or less is held as zeros, and magnitudes above 61440", text)
    assert m
    s = ref.scales()
    borders = 6 * torch.cat([(s[1:] + s[:-1]) / 2, s[1:]])              # where scales change, and what they hold exactly
    largest = torch.cat([2.0 ** torch.linspace(-19, 15.906, 100001, dtype=torch.float64)]
                        + [borders * near for near in (1 - 2.0 ** -40, 1, 1 + 2.0 ** -40)])
    largest = largest[largest <= 61440]
    zeros = largest <= 6 * 2.0 ** -18
    assert bool((ref.scale_of(largest[zeros]) == 0).all()) and bool((ref.scale_of(largest[~zeros]) > 0).all())
    largest = largest[~zeros]
    off = worst(largest)
    bound = torch.where(largest < 9 * 2.0 ** -17, 1 / 3, torch.where(largest < 6 * 2.0 ** -14, float(m[2]), float(m[1])))
    assert bool((off <= bound + 2.0 ** -39).all())
    # and no bound is far from what happens
    for lo, hi, b in ((6 * 2.0 ** -18, 9 * 2.0 ** -17, 1 / 3), (9 * 2.0 ** -17, 6 * 2.0 ** -14, float(m[2])), (6 * 2.0 ** -14, 61441, float(m[1]))):
        assert float(off[(largest > lo) & (largest < hi)].max()) > 0.97 * b
