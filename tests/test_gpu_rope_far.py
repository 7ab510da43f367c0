"""Rotary positions at the largest positions and frequencies, against angles reduced exactly."""
from fractions import Fraction

import numpy as np
import pytest

import fp8_fine_grained_amd as fp8
from tests.test_gpu_kv import dev, held, host, ints

pytestmark = pytest.mark.gpu

TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798")


def turned(x, positions, freqs, interleaved, scale, inverse):
    """x [T][H][rot] in float64; every angle brought below a whole turn in rational numbers first."""
    T, _, rot = x.shape
    left = np.zeros((T, rot // 2))
    for t in range(T):
        for i in range(rot // 2):
            angle = int(positions[t]) * Fraction(float(freqs[i]))
            left[t, i] = float(angle - TWO_PI * round(angle / TWO_PI))
    c, s = np.cos(left)[:, None] * scale, np.sin(left)[:, None] * (-scale if inverse else scale)
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:])
    y, size = np.zeros_like(x), np.abs(a) + np.abs(b)
    if interleaved:
        y[..., 0::2], y[..., 1::2] = a * c - b * s, b * c + a * s
        return y, np.repeat(size, 2, -1)
    y[..., :rot // 2], y[..., rot // 2:] = a * c - b * s, b * c + a * s
    return y, np.concatenate([size, size], -1)


@pytest.mark.parametrize("most", [1.0, 5.0, 1000.0, 2.0 ** 32])
@pytest.mark.parametrize("interleaved,inverse", [(False, False), (True, True)])
def test_far_positions(most, interleaved, inverse):
    """Angles up to 2^63 radians keep the error of near ones."""
    rng = np.random.default_rng(int(most))
    T, H, rot = 12, 3, 64
    pos = np.concatenate([[0, 1, 2 ** 31 - 1], rng.integers(2 ** 30, 2 ** 31, T - 3)])
    freqs = np.concatenate([[most], rng.uniform(most / 2, most, rot // 2 - 1)]).astype(np.float32)
    x = rng.standard_normal((T, H, rot)).astype(np.float32)
    out, _ = fp8.rope(dev(x), None, ints(pos), dev(freqs), interleaved, 1.25, inverse)
    want, size = turned(x.astype(np.float64), pos, freqs, interleaved, 1.25, inverse)
    held(host(out) - want, 2.0 ** -21 * 1.25 * size + 2.0 ** -24 * np.abs(want), "rope")
