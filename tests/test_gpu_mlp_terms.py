"""FP32 operands as three BF16 terms: every product of terms that is taken, on either side and in either layout of the second
operand.  Whole numbers are compared bit for bit; random numbers by the size of the error."""
import numpy as np
import pytest

import mlp_ref as R
from test_gpu_mlp import gated_backward, gated_forward, input_grad, linear, normal

pytestmark = pytest.mark.gpu
BIG = (1 << 17) + 1   # up to 18 bits: three terms
SHAPES = [(1, 1, 1), (3, 129, 257), (130, 513, 96), (257, 40, 136), (300, 1100, 200), (5, 2500, 300)]


def all_products(x, W, W2):
    """Every call's sums of x with the rows of W and W2."""
    V, V2, n = np.ascontiguousarray(W.T), np.ascontiguousarray(W2.T), W.shape[0]
    want, want2 = x @ W.T, x @ W2.T
    assert max(np.abs(want).max(), np.abs(want2).max()) < 2 ** 24
    assert np.array_equal(linear(x, W, "f32"), want)
    out = gated_forward(x, W, W2, "silu", "f32")
    assert np.array_equal(out["gate"], want) and np.array_equal(out["up"], want2)
    assert np.array_equal(input_grad(x, V, "f32"), want)
    assert np.array_equal(input_grad(x, V, "f32", x[::-1].copy(), V2), want + want2[::-1])
    dg, _ = gated_backward(x, V, np.zeros_like(want), np.full_like(want, 2.0), "silu", "f32")   # a'(0) = 1/2
    assert np.array_equal(dg, want)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_three_terms_of_the_second_operand(shape):
    T, k, n = shape
    rng = np.random.default_rng(T + k + n)
    x = rng.integers(-1, 2, (T, k)).astype(float)
    W, W2 = (rng.integers(-BIG, BIG + 1, (n, k)).astype(float) for _ in range(2))
    for w in (W, W2):   # in 50 of the k places, anywhere: sums of two pairs stay below 2^24
        w[:, rng.permutation(k)[50:]] = rng.integers(-1, 2, (n, max(k - 50, 0)))
    all_products(x, W, W2)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_two_terms_on_both_sides(shape):
    """11 bits by 11 bits in two places: the first terms' products, both mixed ones and the second terms'."""
    T, k, n = shape
    rng = np.random.default_rng(T + 3 * k + n)
    x, W, W2 = np.zeros((T, k)), np.zeros((n, k)), np.zeros((n, k))
    for at in {0, k // 2, k - 1}:
        x[:, at] = rng.integers(512, 1024, T) * 2 + 1
    pick = sorted({0, k // 2, k - 1})[-2:]
    W[:, pick] = rng.integers(512, 1024, (n, len(pick))) * 2 + 1
    W2[:, pick[:1]] = -(rng.integers(512, 1024, (n, 1)) * 2 + 1)
    all_products(x, W, W2)


@pytest.mark.parametrize("shape", [(64, 200, 264), (300, 1021, 130), (70, 4096, 96)], ids=str)
def test_error_of_random_products(shape):
    """Frobenius norm of the error over the result's.  A block of 64 k ends with the four steps of the first terms, each cut by
    at most a unit in the last place (2 U) of a sum no larger than the block's; what is left out, the additions to
    nearest and the output's rounding are random and below a tenth of that together: 8 U."""
    T, k, n = shape
    rng = np.random.default_rng(k)
    x, W = normal(rng, T, k), normal(rng, n, k)
    V, most = np.ascontiguousarray(W.T), 1.05 * 8 * R.U32

    def error(got, want):
        return np.linalg.norm(got - want) / np.linalg.norm(want)

    want = x @ W.T
    assert error(linear(x, W, "f32"), want) <= most
    assert error(input_grad(x, V, "f32"), want) <= most
    out = gated_forward(x, W, -W, "silu", "f32")
    assert error(out["gate"], want) <= most and error(out["up"], -want) <= most
    dg, _ = gated_backward(x, V, np.zeros_like(want), np.full_like(want, 2.0), "silu", "f32")
    assert error(dg, want) <= most
    x2, W2 = normal(rng, T, k), normal(rng, n, k)
    want = want + x2 @ W2.T
    assert error(input_grad(x, V, "f32", x2, np.ascontiguousarray(W2.T)), want) <= most
