"""The oracle of the paged cache at the ends of its range, on the CPU."""
from fractions import Fraction

import numpy as np

from oracle import paged as ref


def test_the_oracle_takes_keys_of_any_size():
    """The exponent of the K scale by rational arithmetic: the smallest e with x^2 + z^2 <= (448 2^e)^2."""
    def smallest(x, z):
        top = Fraction(x) ** 2 + Fraction(z) ** 2
        return next(e for e in range(-72, 121) if e == 120 or top <= (448 * Fraction(2) ** e) ** 2)

    g = np.random.default_rng(0)
    sizes = [(1.75 * 2.0 ** e, 0.0) for e in (-64, -63, 0, 63, 64, 90, 127)] + [(1.7578125 * 2.0 ** e, 0.0) for e in (-64, -63, 60, 64, 90)]
    sizes += [(m * 2.0 ** e, n * 2.0 ** e) for e in (-80, -66, -64, -63, -1, 30, 62, 64, 66, 99, 126)
              for m, n in np.round(g.uniform(1, 2, (20, 2)) * 128) / 128]
    for x, z in sizes:
        k = np.zeros((1, 64))
        k[0, 3], k[0, 35] = x, z
        assert ref._smallest(ref.k_reach(k, 32)[0]) == smallest(x, z), (x, z)
