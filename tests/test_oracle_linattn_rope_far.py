"""The oracle's angles at positions far from zero against decimal arithmetic
of 80 digits.  An angle below 2 pi is rounded three times (the part of a turn,
2 pi and their product): 3 x 2^-53 x 2 pi < 2^-48."""
from decimal import Decimal, localcontext

import numpy as np
import pytest

from oracle import linattn_oracle as R

PI = "3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798"


@pytest.mark.parametrize("position", [0, 1, -1, 4097, 2 ** 31 - 1, -(2 ** 31), 123456789012, 2 ** 40 + 12345, 2 ** 52 + 2 ** 31,
                                      -(2 ** 52)])
def test_angles_are_exact(position):
    freqs = 10000.0 ** (-2.0 * np.arange(32) / 64)
    got = R.rope_angles([[position]], freqs)[0, 0]
    with localcontext() as c:
        c.prec = 80
        turn = 2 * Decimal(PI)
        for f, a in zip(freqs, got):
            want = Decimal(position) * Decimal(float(f)) % turn   # of the position's sign
            d = abs(want - Decimal(float(a)))
            assert min(d, abs(turn - d), abs(2 * turn - d)) < Decimal(2) ** -48, (position, f)


def test_rotation_by_a_far_angle():
    freqs = np.array([0.7, 1e-3])
    x = np.array([1.0, 2.0, -3.0, 0.5]).reshape(1, 1, 1, 4)
    far, near = 2 ** 51 + 1, 5
    a, b = (R.rope_angles([[p]], freqs)[0, 0] for p in (far, near))
    y = R.rope_ref(x, [[far]], freqs)[0, 0, 0]
    for i in range(2):
        c, s = np.cos(a[i]), np.sin(a[i])
        assert y[i] == pytest.approx(x[0, 0, 0, i] * c - x[0, 0, 0, i + 2] * s, abs=1e-14)
        assert y[i + 2] == pytest.approx(x[0, 0, 0, i] * s + x[0, 0, 0, i + 2] * c, abs=1e-14)
    # a turn onwards and back is none
    z = R.rope_ref(R.rope_ref(x, [[far]], freqs), [[far]], freqs, inverse=True)
    np.testing.assert_allclose(z, x, atol=1e-14)
    assert b[0] == pytest.approx(3.5)
