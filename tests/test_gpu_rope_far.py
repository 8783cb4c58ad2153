"""The bound that csa_rope.h gives for its angles, at far positions and for
frequencies past the usual ones: |p| (2^-64 + |f| 2^-61 / (2 pi)) + 2^-33 turns,
against rational arithmetic.

The pair (1, 0) turns into the cosine and the sine. An angle that is off by t
turns moves them by at most 2 pi t; beside it stands what test_gpu_rope.py
counts for an element, 2^-20.9 of |a| + |b| = 1.
"""
import math
from fractions import Fraction

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459")
FREQS = [1.0, 0.7310585786300049, 0.5, 1e-3, 2.0 ** -31, 3.0, -6.25, 1e3, -700.1, 2.0 ** 20, 1.4e6, -2.0 ** 26 - 1.0]


@pytest.fixture(scope="module")
def gsk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_softmax_kv_gb300 as g
    g.build()
    return g


def turns_off(p, f):
    return abs(p) * (2.0 ** -64 + abs(f) * 2.0 ** -61 / (2 * math.pi)) + 2.0 ** -33


@pytest.mark.parametrize("pos", [1, 4097, 2 ** 20 + 1, 2 ** 31 - 1, 2 ** 31 - 12345, -2 ** 31, -2 ** 30 - 7, 2 ** 40 + 3])
def test_angles_of_far_positions(gsk, pos):
    f = torch.tensor(FREQS, dtype=torch.float64, device="cuda")
    x = torch.zeros(1, 1, 2 * len(FREQS), device="cuda")
    x[..., 0::2] = 1.0
    y = gsk.csa_rope(x, f, torch.tensor([pos], device="cuda"))[0, 0].double().cpu().numpy()
    for i, v in enumerate(FREQS):
        turn = float((Fraction(pos) * Fraction(v) / TWO_PI) % 1)
        want = np.array([math.cos(2 * math.pi * turn), math.sin(2 * math.pi * turn)])
        tol = 2 * math.pi * turns_off(pos, v) + 2.0 ** -20.9
        assert (np.abs(y[2 * i:2 * i + 2] - want) <= tol).all(), (v, y[2 * i:2 * i + 2], want, tol)


def test_bounds_that_the_header_names():
    assert turns_off(2 ** 31, 1.0) < 2.0 ** -31
    assert turns_off(2 ** 31, 2.0 ** 20) < 2.0 ** -12
    assert turns_off(2 ** 20, 1.0) < 2.0 ** -32
