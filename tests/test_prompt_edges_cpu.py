"""Host-side arithmetic and limits of the operators of a prompt's layer where values and sizes meet their ends (no GPU)."""
import math
import random
from fractions import Fraction

import pytest

from exact_circle import circle
import weight_streaming_q4_gb300 as q4
from weight_streaming_q4_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return q4.lib()


def test_turns_of_a_position_are_exact():
    """Every bit of a frequency's turns is right: what is off by one unit of 2^-64 here is off by 2^-33 of a turn at the farthest position."""
    rng, two_pi = random.Random(3), circle()
    freqs = [1.0, 0.794, 2.0, 3.7, 30.0, 100.0, -3.0, 2 * math.pi, math.pi, -2 * math.pi, 1e-6, -1e-12, 1e-30, 5e-324, 0.0, -0.0, 2.0 ** 60, -(2.0 ** 60), math.nextafter(2.0 ** 60, 0)]
    freqs += [rng.choice((-1, 1)) * math.exp(rng.uniform(-45, 41)) for _ in range(400)]
    for at in range(0, len(freqs), 100):
        part = freqs[at:at + 100]
        for got, f in zip(q4.Rope.of(512, part).turn, part):
            want = Fraction(f) / two_pi * 2 ** 64
            off = (got - want) % 2 ** 64
            assert min(off, 2 ** 64 - off) <= Fraction(5, 8), f


@pytest.mark.parametrize("freq", [math.nextafter(2.0 ** 60, math.inf), -1e19, 1e300])
def test_frequencies_whose_turns_are_not_known_are_refused(freq):
    with pytest.raises(q4.Q4Error):
        q4.Rope.of(8, [1.0, freq])
