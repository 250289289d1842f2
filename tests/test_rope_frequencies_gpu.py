"""The rotation at frequencies of any size: angles far beyond what a product in
64 bits keeps, against whole-number arithmetic."""

from fractions import Fraction
from math import pi

import numpy as np
import pytest
import torch

from attention_flashattention_fwd_04_b200 import api

pytestmark = pytest.mark.gpu


def two_pi(bits):
    """2 pi * 2^bits, rounded down: Machin's 16 atan(1/5) - 4 atan(1/239), doubled, in whole numbers."""
    one = 1 << (bits + 32)

    def arctan_of_inverse(n):
        total, term, k = 0, one // n, 0
        while term:
            total += term // (2 * k + 1) * (-1) ** k
            term //= n * n
            k += 1
        return total

    return 2 * (16 * arctan_of_inverse(5) - 4 * arctan_of_inverse(239)) >> 32


CIRCLE = Fraction(two_pi(400), 1 << 400)


def angle(position, freq):
    """position * freq less whole turns, to the last bit of a double."""
    a = Fraction(int(position)) * Fraction(float(freq))
    return float(a - CIRCLE * (a // CIRCLE))


def test_the_circle():
    assert abs(float(CIRCLE) - 2 * pi) < 1e-15 and angle(1, 2 * pi) == pytest.approx(2 * pi, abs=1e-15)


@pytest.mark.parametrize("freq", [15.7, 6.5, -15.7, 1e3, 1e8, -1e8, 123456789.0625, 1e12, 2.0 ** 53 + 2, 1e18, 2.0 ** 62 - 2.0 ** 9, 1e-9, 5e-300])
@pytest.mark.parametrize("adjacent", [False, True])
def test_large_frequencies_at_far_positions(freq, adjacent):
    """Unit pairs, so that the outputs are the cosines and sines: off by a rounding to bf16 and a few 2^-24."""
    d = 64
    freqs = [freq * (1.0 - j / 64.0) for j in range(d // 2)]
    spec = api.rope_spec(d, inv_freq=freqs, adjacent_pairs=adjacent)
    where = [2 ** 31 - 1, -2 ** 31, 16777217, 123456789, -7, 1, 0]
    x = torch.zeros(len(where), 1, d, dtype=torch.bfloat16)
    first = slice(0, d, 2) if adjacent else slice(0, d // 2)
    second = slice(1, d, 2) if adjacent else slice(d // 2, d)
    x[..., first] = 1.0
    out, _ = api.attn_rope(x.cuda(), None, torch.tensor([where], dtype=torch.int32).cuda(), spec)
    out = out.double().cpu().numpy()[:, 0]
    for i, p in enumerate(where):
        a = np.array([angle(p, f) for f in freqs])
        for got, want in ((out[i, first], np.cos(a)), (out[i, second], np.sin(a))):
            assert np.all(np.abs(got - want) <= 2.0 ** -9 * 2 * np.abs(want) + 2.0 ** -20), (p, np.abs(got - want).max())
