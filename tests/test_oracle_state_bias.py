"""How far the 8-bit second moment lies above the 32-bit one, followed over
thousands of steps with the oracle's rounding.

The code of r is rounded without bias, r^2 gains the rounding's variance each
step. A step moves r by d = (1 - b2) (g^2 - r^2) / (2 r), far less than the
distance q between codes, so r goes to the neighbouring code with probability
|d| / q and E[r^2] grows by |d| (q - |d|) beyond the true step. In the steady
state that stands against the decay (1 - b2) (E[r^2] - E[g^2]):

    E[r^2] / E[g^2] - 1  =  q / (2 r) * E|g^2 / r^2 - 1|     (to first order in |d| / q)

whatever b2. q / r is between 1/15 and 1/8 for codes from 2^-6 on (r from
1/28672 of the block's largest on), and grows below, where codes are 2^-9
apart; E|x^2 - 1| = 4 phi(1) = 0.968 for a standard normal x.
"""
import math

import numpy as np
import pytest

from oracle import optim as OO

NORMAL = 4 * math.exp(-0.5) / math.sqrt(2 * math.pi)


def follow(sizes, b2, steps, seed):
    """Means of the decoded r^2, of v in 64 bits, and of the right-hand side over
    the second part of a run, by size: blocks of one element of 1 and 63 of the
    size, with normal gradients."""
    rng = np.random.default_rng(seed)
    blocks = 24
    n = 64 * blocks * len(sizes)
    sigma = np.repeat(np.array(sizes), 64 * blocks)
    sigma[::64] = 1.0
    v = sigma ** 2
    r2 = v.copy()
    got, want, law = np.zeros(n), np.zeros(n), np.zeros(n)
    kept = 0
    for t in range(1, steps + 1):
        g2 = (sigma * rng.standard_normal(n)) ** 2
        if t > steps // 4:
            r = np.sqrt(r2)
            y = r / np.repeat(np.ldexp(1.0, OO.scales_of(r) - 127), 64)
            q = np.ldexp(1.0, np.maximum(np.frexp(y)[1] - 1, -6) - 3)
            got += r2
            want += v
            law += 0.5 * q / y * np.abs(g2 - r2)
            kept += 1
        v = b2 * v + (1 - b2) * g2
        r = np.sqrt(b2 * r2 + (1 - b2) * g2)
        s = OO.scales_of(r)
        lo, hi, pos = OO.encode_levels(r, s, rng.integers(0, 65536, n), True)
        r2 = (np.where(pos >= 1, hi, lo) * np.repeat(np.ldexp(1.0, s - 127), 64)) ** 2
    small = np.ones(n, dtype=bool)
    small[::64] = False
    cut = lambda x: np.array([p[m].sum() for p, m in zip(np.split(x, len(sizes)), np.split(small, len(sizes)))])  # noqa: E731
    return cut(got) / cut(want) - 1, cut(law) / cut(want)


@pytest.mark.parametrize("b2,steps", [(0.99, 3000), (0.999, 6000)])
def test_second_moments_from_codes_lie_a_few_per_cent_above(b2, steps):
    """Sizes from the block's largest to 1e-4 of it. The sampling error: r^2 and v
    see the same gradients; what separates them is a walk of about 0.2 of r^2
    with a memory of 1 / (1 - b2) steps, over 63 * 24 elements and 2250 or 4500
    steps (22 or 4.5 memories), 0.2 / sqrt(1512 * 4.5) = 0.0024 at most; four of
    these. The law leaves out |d| / q (4 % of it at b2 = 0.99) and the spread of r
    over neighbouring codes: a quarter."""
    bias, law = follow([1.0, 0.3, 1e-2, 1e-3, 1e-4], b2, steps, 1)
    noise = 4 * 0.0024
    print(b2, bias, law)
    assert (np.abs(bias - law) <= 0.25 * law + noise).all()
    assert (bias >= 0.75 * NORMAL / 30 - noise).all() and (bias <= 1.25 * NORMAL / 16 + noise).all()


def test_second_moments_far_below_their_blocks_largest():
    """1e-5 of the largest: one to three steps of 2^-9 above 0, where r^2 may lie
    half above v, and no code is 0."""
    bias, _ = follow([1e-5], 0.99, 3000, 2)
    print(bias)
    assert 0.1 <= bias[0] <= 1.0
