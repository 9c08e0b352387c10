"""The turns per position of the rotary frequencies against exact fractions, on the CPU."""
import math

import numpy as np
import pytest

import split_kv_decode_distattention_gb300 as dattn
from split_kv_decode_distattention_gb300 import _build

import _block_ref as ref


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return dattn.load_library()


def _off(freqs):
    """Units of 2^-64 of a turn between the library's turns and the exact ones."""
    n = len(freqs)
    freqs = list(freqs) + [0.0] * (-n % 8)
    r = dattn.Rotation(2 * len(freqs), inv_freq=freqs)
    out = []
    for t, f in zip(list(r._turns)[:n], freqs):
        d = (ref.Fraction(t) - ref.Fraction(f) / ref.TWO_PI * 2 ** 64) % 2 ** 64
        out.append(float(min(d, 2 ** 64 - d)))
    return out


def test_turns_are_right_to_the_last_bit():
    rng = np.random.default_rng(7)
    sets = [dattn.dattn_rope_frequencies(128, b) for b in (1e4, 5e5, 1e6)]
    sets += [np.exp2(rng.uniform(-40, 31.9, 64)) * rng.choice([-1, 1], 64) for _ in range(8)]
    sets += [[1.0, -1.0, 2 * math.pi, math.pi, -math.pi / 2, 0.0, -0.0, 1e-30, 5e-324, 2.0 ** 32 - 1,
              -2.0 ** -64, 7.0]]
    for f in sets:
        # rounded to nearest, of a quotient that is itself right to 2^-8 of a unit or better
        assert max(_off(f)) <= 0.5 + 2.0 ** -7


def test_angles_of_far_positions():
    """p times the turns, mod one turn: within 2^31 half units, 2^-34 of a turn, at any position."""
    f = dattn.dattn_rope_frequencies(128, 500000.0)
    turns = list(dattn.Rotation(128, inv_freq=f)._turns)
    for p in (2 ** 31 - 1, -2 ** 31, 10 ** 9 + 7, 123456):
        for t, x in zip(turns, f):
            d = (ref.Fraction(p * t, 2 ** 64) - p * (ref.Fraction(x) / ref.TWO_PI)) % 1
            assert min(d, 1 - d) <= 2.0 ** -34 * (1 + 2.0 ** -6)


def test_turns_of_any_finite_frequency_are_taken():
    for f in (1e308, -1e308, 2.0 ** 64, -2.0 ** 63, 1e20):
        dattn.Rotation(16, inv_freq=[f] * 8)
