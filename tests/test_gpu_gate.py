"""The gate's arithmetic by itself: far below zero, where its factors are smaller than FP32's normal numbers and its value
is not, and the slope where 1 - s is small.

The products are made exact (one token-independent number each), so what is left is the gate and one rounding.
"""
import numpy as np
import pytest

import mlp_ref as R
from test_gpu_mlp import gated_backward, gated_forward, rounded

pytestmark = pytest.mark.gpu
U = R.U32
TINY = 2.0 ** -149   # FP32's smallest step
FAR = {"silu": [-80.0, -87.0, -87.5, -88.0, -88.5, -89.0, -90.0, -91.0],
       "gelu_tanh": [-9.5, -9.75, -9.9375, -10.0, -10.0625, -10.125],
       "gelu": [-12.5, -13.0, -13.125, -13.1875, -13.25]}


def backward(gate, up, dh, fn, dt):
    """dg and du where dy W is dh everywhere."""
    T, f = gate.shape
    dy, W = np.zeros((T, 16)), np.zeros((16, f))
    dy[:, 0], W[0] = dh, 1.0
    return gated_backward(dy, W, gate, up, fn, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("fn", sorted(FAR))
def test_far_below_zero(fn, dt):
    """Scaled by 2^40, so that no output is denormal.  A factor below 2^-126 is off by its own step: s, e and 1 / (1 + e) e
    by TINY each, erfc and the exponential by a few, times at most 1 + 2 |g| z' (z' below 8) on their way."""
    g = rounded(np.array([FAR[fn]]), dt)
    f, big = g.shape[1], 2.0 ** 40
    a, slope = R.gate(g, fn)
    rel = R.gate_error(g, fn) + 8 * U
    step = 16 * TINY * (1 + 2 * np.abs(g) * 8)
    assert (np.abs(a).min() > 2.0 ** -127) or fn == "gelu"
    dg, du = backward(g, np.ones_like(g), big, fn, dt)
    want = big * slope
    # a' = s + g z' s (1 - s): the sum of the terms' sizes, each with its error
    assert (np.abs(dg - want) <= 2 * rel * np.abs(want) + big * step + 1.01 * R.half_step(want, dt)).all()
    want = big * a
    assert (np.abs(du - want) <= rel * np.abs(want) + big * step + 1.01 * R.half_step(want, dt)).all()
    out = gated_forward(np.zeros((3, 16)), np.zeros((f, 16)), np.zeros((f, 16)), fn, dt, bg=g[0], bu=np.full(f, big))
    assert (np.abs(out["h"] - want) <= rel * np.abs(want) + big * step + 1.01 * R.half_step(want, dt)).all()


@pytest.mark.parametrize("fn", ["silu", "gelu_tanh"])
def test_slope_where_the_gate_is_almost_open(fn):
    """FP32.  expf is off by 2 units in the last place (4 U) and by its argument's error (z is 6 roundings of its size for the
    tanh form, none for SiLU); 1 + e, the reciprocal (a unit, 2 U) and the product behind it add 4 U.  a' has s once and
    g z' s (1 - s) with both and four more roundings."""
    g = rounded(np.linspace(-20, 20, 4001)[None, :], "f32")
    z, dz = (g, 1.0) if fn == "silu" else (R_Z * (g + 0.044715 * g ** 3), R_Z * (1 + 3 * 0.044715 * g * g))
    e = np.exp(-np.abs(z))
    s, o = np.where(z >= 0, 1.0, e) / (1 + e), np.where(z >= 0, e, 1.0) / (1 + e)
    es = (8 + (0 if fn == "silu" else 6 * np.abs(z))) * U   # of s and of 1 - s
    dg, du = backward(g, np.ones_like(g), 1.0, fn, "f32")
    a, slope = R.gate(g, fn)
    # where s is near 1 its error is that of e, which is 1 - s of it
    ss = np.where(z >= 0, es * o + 3 * U, es) * s
    term = np.abs(g * dz) * s * o
    assert (np.abs(dg - slope) <= ss + (2 * es + 8 * U) * term + 2 * U * np.abs(slope) + 1e-37).all()
    assert (np.abs(du - a) <= np.abs(g) * ss + 2 * U * np.abs(a) + 1e-37).all()


R_Z = 2.0 * np.sqrt(2.0 / np.pi)
