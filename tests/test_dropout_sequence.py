"""How the dropout masks of different seeds, sites and steps are related, as
the header states it."""

import os
import re

import numpy as np
import pytest

from oracle import matrices as O

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = open(os.path.join(ROOT, "include", "dopt.h")).read()
MOVE = 0x144CBC89


def key(seed, site, t):
    return seed + site * 0x510E527F + t * 0x6A09E667


def moved(a, b):
    """Pairs by which b's numbers are moved against a's, nearest to 0."""
    d = (key(*b) - key(*a)) * MOVE % 2**32
    return d if d < 2**31 else d - 2**32


def test_the_headers_constant():
    assert MOVE * 0x9E3779B9 % 2**32 == 1 and "(key' - key) * 0x144CBC89 pairs" in HEADER


@pytest.mark.parametrize("a,b", [((5, 3, 11), (5, 22, 7)), ((5, 3, 11), (5, 16, 11)), ((5, 3, 11), (5, 3, 54)), ((5, 3, 11), (123456789, 0, 2)),
                                 ((0, 0, 0), (2**32 - 1, 2**32 - 1, 10**12))])
def test_masks_are_one_sequence_moved(a, b):
    n = np.arange(4000)
    far = (n // 2 + moved(a, b)) % 2**32 * 2 + n % 2  # elements of a
    assert np.array_equal(O.random16(n, *b), O.random16(far, *a))


def test_the_headers_examples():
    text = re.sub(r"\s*\n \* ", " ", HEADER)
    assert "site + 19 at t - 4 is moved by 4122407 pairs, site + 13 by 39608715, t + 43 by 5865525" in text
    assert [abs(moved((7, 2, 50), b)) for b in ((7, 21, 46), (7, 15, 50), (7, 2, 93))] == [4122407, 39608715, 5865525]
