"""Pins of the plain forms of the rotary positions, the norm before them and the prefill, and the
frequencies, which the host computes."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest

from linear_attention_02_gb300 import _native
from oracle import serving as ref

lib = _native.lib
# 2 pi to 60 digits (Machin's formula in whole numbers)


def _two_pi():
    def arctan_inv(n, one):
        total = term = one // n
        k, sign = 3, -1
        while term:
            term //= n * n
            total += sign * (term // k)
            k, sign = k + 2, -sign
        return total
    one = 10 ** 70
    return Fraction(2 * 4 * (4 * arctan_inv(5, one) - arctan_inv(239, one)), one)


def _freqs(rot, base=10000.0, scaling=0, factor=1.0, olen=0.0, fast=32.0, slow=1.0):
    buf, mag = (ctypes.c_uint64 * (rot // 2))(), ctypes.c_float()
    assert lib.la_rotary_frequencies(rot, base, scaling, factor, olen, fast, slow, buf, ctypes.byref(mag)) == 0
    return list(buf), mag.value


NAMES = ["none", "linear", "base", "by_parts"]


@pytest.mark.parametrize("rot", [2, 6, 20, 64, 128])
@pytest.mark.parametrize("scaling", range(4))
def test_frequencies(rot, scaling):
    f, mag = _freqs(rot, 10000.0, scaling, 8.0, 4096.0)
    theta, m = ref.rotary_theta(rot, 10000.0, NAMES[scaling], 8.0, 4096)
    assert abs(mag - m) <= 2.0 ** -24 * m
    two_pi = _two_pi()
    for u, t in zip(f, theta):
        # the angles are doubles: a few roundings of 2^-53 each side (power, factor, ramp), then a unit of 2^-64
        want = Fraction(float(t)) / two_pi
        assert abs(Fraction(u, 1 << 64) - want) <= 8 * Fraction(1, 1 << 53) * want + Fraction(1, 1 << 64)


def test_frequencies_of_whole_angles_are_exact():
    # theta_0 = 1: the whole part of 2^64 / 2 pi, to the nearest
    u, _ = _freqs(2)
    assert abs(Fraction(u[0], 1 << 64) - 1 / _two_pi()) <= Fraction(1, 1 << 64)


def test_scaled_frequencies():
    one, _ = ref.rotary_theta(8)
    lin, _ = ref.rotary_theta(8, scaling="linear", factor=4.0)
    np.testing.assert_allclose(lin, one / 4)
    bas, _ = ref.rotary_theta(8, scaling="base", factor=4.0)
    assert bas[0] == 1 and abs(bas[3] * 4 - one[3]) < 1e-15  # the slowest pair is slowed by the factor
    par, mag = ref.rotary_theta(8, base=1e6, scaling="by_parts", factor=4.0, original_len=2000)
    one, _ = ref.rotary_theta(8, base=1e6)
    assert par[0] == one[0] and abs(par[3] - one[3] / 4) < 1e-20  # 318 turns, and a third of one
    assert abs(mag - (1 + 0.1 * math.log(4))) < 1e-15


def test_frequency_refusals():
    f = lib.la_rotary_frequencies
    buf, mag = (ctypes.c_uint64 * 64)(), ctypes.c_float()
    inv, uns = _native.LA_ERR_INVALID_ARG, _native.LA_ERR_UNSUPPORTED
    m = ctypes.byref(mag)
    for rot in (0, -2, 7, 130):
        assert f(rot, 1e4, 0, 1, 0, 32, 1, buf, m) == inv
    for base in (0.5, 0.0, -1e4, math.inf, math.nan):
        assert f(64, base, 0, 1, 0, 32, 1, buf, m) == inv
    assert f(64, 1e4, 4, 1, 0, 32, 1, buf, m) == uns
    for factor in (0.5, math.nan, math.inf):
        assert f(64, 1e4, 1, factor, 0, 32, 1, buf, m) == inv
    assert f(64, 1e4, 3, 2, 0, 32, 1, buf, m) == inv and f(64, 1e4, 3, 2, 4096, 1, 1, buf, m) == inv
    assert f(64, 1e300, 2, 1e300, 0, 32, 1, buf, m) == inv
    assert f(64, 1e4, 0, 1, 0, 32, 1, None, m) == inv and f(64, 1e4, 0, 1, 0, 32, 1, buf, None) == inv


def test_phases_are_exact_at_any_position():
    f, _ = _freqs(4, 10000.0)
    for p in (0, 1, 12345, 2 ** 20 + 1, 2 ** 31 - 1):
        a = ref.rotary_angles(f, [p])[0]
        for u, x in zip(f, a):
            turns = Fraction(p * u, 1 << 64) % 1
            assert abs(Fraction(float(x)) - turns * _two_pi()) < Fraction(1, 1 << 48)


def test_rotary_by_hand():
    a = np.array([math.pi / 2, math.pi])
    x = np.array([1.0, 2.0, 3.0, 4.0, 5.0])
    np.testing.assert_allclose(ref.rotary(x, a, "half", 2.0), [-6, -4, 2, -8, 5], atol=1e-14)
    np.testing.assert_allclose(ref.rotary(x, a, "interleaved"), [-2, 1, -3, -4, 5], atol=1e-14)
    # turning back undoes it, and products of two rows depend on the distance of their positions alone
    r = np.random.RandomState(1)
    q, k, th = r.randn(8), r.randn(8), ref.rotary_theta(8)[0]
    np.testing.assert_allclose(ref.rotary(ref.rotary(q, 7 * th), -7 * th), q)
    for lay in ("half", "interleaved"):
        d = [ref.rotary(q, (p + 5) * th, lay) @ ref.rotary(k, p * th, lay) for p in (0, 3, 100)]
        np.testing.assert_allclose(d, d[0])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_norm_gradient_by_differences(layout):
    r = np.random.RandomState(2)
    x, dy, w, a = r.randn(3, 6), r.randn(3, 6), r.randn(6), r.randn(3, 2)
    dx, dw = ref.norm_rotary_backward(x, dy, w, a, layout, 1.25, 0.1)
    f = lambda x, w: (dy * ref.norm_rotary(x, w, a, layout, 1.25, 0.1)).sum()  # noqa: E731
    h = 1e-6
    for i in range(18):
        e = np.zeros(18)
        e[i] = h
        assert abs((f(x + e.reshape(3, 6), w) - f(x - e.reshape(3, 6), w)) / (2 * h) - dx.reshape(-1)[i]) < 1e-8
    for i in range(6):
        e = np.zeros(6)
        e[i] = h
        assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - dw[i]) < 1e-8


def test_prefill_against_the_decode_step():
    # a chunk of one token over what is cached is the decode step that appends the same row
    r = np.random.RandomState(3)
    K, V, q = r.randn(6, 2, 4, 8), r.randn(6, 2, 4, 8), r.randn(3, 4, 8)
    table, lens = [[0, 2, -1], [1, 3, 5], [4, -1, -1]], [5, 10, 0]
    for window in (0, 3):
        out, lse, _ = ref.paged_prefill(q, K, V, table, lens, [0, 1, 2, 3], window)
        k = np.array([K[table[i][n // 4], :, n % 4] for i, n in enumerate(lens)])
        v = np.array([V[table[i][n // 4], :, n % 4] for i, n in enumerate(lens)])
        o, e = ref.paged_decode(q, k, v, K, V, table, lens, window)
        np.testing.assert_allclose(out, o)
        np.testing.assert_allclose(lse, e)


def test_prefill_by_hand():
    # equal keys: the prefix mean of the values, within the window
    K, V = np.ones((2, 1, 2, 1)), np.arange(4.0).reshape(2, 1, 2, 1)
    out, lse, _ = ref.paged_prefill(np.ones((3, 1, 1)), K, V, [[0, 1]], [1], [0, 3], 0, 1.0)
    np.testing.assert_allclose(out[:, 0, 0], [0.5, 1, 1.5])
    np.testing.assert_allclose(lse[:, 0], 1 + np.log([2, 3, 4]))
    out, _, _ = ref.paged_prefill(np.ones((3, 1, 1)), K, V, [[0, 1]], [1], [0, 3], 2, 1.0)
    np.testing.assert_allclose(out[:, 0, 0], [0.5, 1.5, 2.5])
