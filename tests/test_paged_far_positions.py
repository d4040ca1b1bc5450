"""The angles of kv_append() at far positions, against exact rational arithmetic,
for frequencies over the whole range that it takes."""
import math
import os
import random
import re
from fractions import Fraction

import pytest
import torch

import exact_tiled_attention_23_gb300 as fa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TWO_PI = 2 * Fraction(31415926535897932384626433832795028841971693993751058209749445923, 10 ** 64)
MASK = (1 << 64) - 1


def constants():
    with open(os.path.join(ROOT, "exact_tiled_attention_23_gb300", "csrc", "fa_append.cu")) as f:
        return [int(x, 16) for x in re.search(r"kInvTwoPiHi = (0x\w+)ull, kInvTwoPiLo = (0x\w+)ull", f.read()).groups()]


def test_the_constant_is_one_over_two_pi():
    hi, lo = constants()
    assert (hi << 64) + lo == int((1 << 128) / TWO_PI)


def test_a_frequency_in_turns_is_good_to_its_last_bit():
    """The kernel's integer steps, with the constants of its source."""
    hi_c, lo_c = constants()
    rng = random.Random(1)
    for _ in range(2000):
        e, m = rng.randint(1, 142), rng.randint(1 << 23, (1 << 24) - 1)       # f = m 2^(e - 150)
        if rng.random() < 0.02:
            e, m = 143, 1 << 23                                               # 65536, the largest
        part = m * hi_c & MASK
        lo = (part + (m * lo_c >> 64)) & MASK
        hi = ((m * hi_c >> 64) + (lo < part)) & MASK
        shift = 150 - e
        F = (lo >> shift | hi << (64 - shift) & MASK) if shift < 64 else hi >> (shift - 64) if shift < 128 else 0
        exact = Fraction(m) * Fraction(2) ** (e - 150) / TWO_PI * (1 << 64)
        off = (exact - F) % (1 << 64)
        assert off < 1 or off > (1 << 64) - Fraction(1, 1000), (e, m, float(off))


@pytest.mark.gpu
@pytest.mark.parametrize("offset", [0, 1 << 31, (1 << 36) + 12345, (1 << 40) - 7, 1 << 40])
def test_angles_of_far_positions(offset):
    """cos and sin are off by 2 pi n 2^-64 and 2^-22 (the angle's fp32 form, the
    function's error and the product), and rounded once to fp16."""
    fa.build()
    D, length, rng = 64, 9, random.Random(offset)
    n = offset + length - 1
    freq = [65536.0, -65536.0, 65535.996, 40000.5, 1.0, -0.75, 3.14159265, 0.0, 1e-30, 2.0 ** -20]
    freq += [rng.choice([-1, 1]) * 2.0 ** rng.uniform(-12, 16) for _ in range(D // 2 - len(freq))]
    freq = torch.tensor(freq, dtype=torch.float32)
    pool = torch.zeros((1, 1, 16, D), dtype=torch.float16, device="cuda")
    cache = fa.PagedKV(pool, pool.clone(), torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
                       torch.tensor([length], dtype=torch.int32, device="cuda"))
    x = torch.zeros((1, 1, 1, D), dtype=torch.float16)
    x[..., :D // 2] = 1                             # (1, 0) turns into (cos, sin)
    out = fa.kv_append(cache, x.cuda(), x.cuda(), q=x.cuda(), inv_freq=freq.cuda(), position_offset=offset)
    got = out.cpu().double()[0, 0, 0]
    for p in range(D // 2):
        a = Fraction(float(freq[p])) * n
        a = float(a - TWO_PI * round(a / TWO_PI))
        off = 2 * math.pi * n * 2.0 ** -64 + 2.0 ** -22
        for value, want in ((got[p], math.cos(a)), (got[D // 2 + p], math.sin(a))):
            bound = off + 2.0 ** -11 * (abs(want) + off) + 2.0 ** -25
            assert abs(float(value) - want) <= bound, (p, float(freq[p]), n, float(value), want)
