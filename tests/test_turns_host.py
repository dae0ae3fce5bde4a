"""Frequencies as fractions of a turn: rounded once, without a GPU."""

import math
from fractions import Fraction

import numpy as np
import pytest


@pytest.fixture(scope="module")
def sdl():
    from structured_decay_linear_gb300 import build as nvbuild
    nvbuild.build()
    import structured_decay_linear_gb300 as s
    s.library()
    return s


def test_turns_are_rounded_once(sdl):
    """Half a unit of 2^-64, and what two numbers of 53 bits leave of 1 / (2 pi) and its products, below 2^-9 of one for
    frequencies up to 2 pi (a rounding of 2^-54 turns' rest, 2^-107, and the constant's, 2^-110, both times 2^64)."""
    pi = Fraction(314159265358979323846264338327950288419716939937510582097494, 10 ** 59)
    r = np.random.default_rng(0)
    f = np.concatenate([np.logspace(-18, math.log10(6.28), 3000), 10000.0 ** (-2 * np.arange(64) / 128), r.uniform(0, 6.28, 3000),
                        [0.0, 0.5, 1.0, math.pi, 2 * math.pi, 2.0 ** -64, 2.0 ** -62]])
    t = np.zeros(len(f), np.uint64)
    assert sdl.dplr_nr_turns(f.ctypes.data, len(f), t.ctypes.data) == 0
    for x, got in zip(f, t):
        off = abs(Fraction(float(x)) / (2 * pi) % 1 * 2 ** 64 - int(got))
        assert min(off, 2 ** 64 - off) <= Fraction(1, 2) + Fraction(1, 512), x
