"""How the products sum: after how many terms a sum is rounded to nearest, and the segments of a forward product that keeps
h in 8 bits.  Whole numbers throughout, so every comparison is bit for bit."""
import math

import numpy as np
import pytest
import torch

import act_ref as A
from fac_whitening_gb300 import gift as G
from test_gpu_mlp import gated_backward, gated_forward, input_grad, linear, rounded

pytestmark = pytest.mark.gpu


def terms(k, kept):
    """The most terms that are summed before a rounding to nearest."""
    if not kept:
        return 1024
    b = -(-k // 64)
    return 64 * max(2, min(16, 1 + b // 8, math.floor(math.sqrt(b) + 0.5)))


def long_sums(k, most, n, seed):
    """x (k) and W (n x k) whose sums are exact when they are rounded to nearest every `most` terms or sooner, and are not when
    much longer sums are truncated.  Products are positive and close to 2^24 / most: `most` of them fit into FP32's 24 bits,
    a third more do not.  An FP32 sum past 2^24 holds even numbers only, and every 16 products have an odd sum, so each
    later step of an MMA loses at least 1, whether products or their sum are cut.  64 products sum to a multiple of 64, so
    what is added to nearest stays exact to 2^30.  The last 64 places hold few large products that take the total, but
    for 64 to 192, away again; those are multiples of 64 below 2^30 too, exact wherever the cut falls.  Results: 64 + 64 (n % 3)."""
    rng = np.random.default_rng(seed)
    top = 2 ** 24 // most
    w_top = min(255, top // 255)
    w_low = w_top - w_top // 8
    assert w_top >= 40 and k % 64 == 0
    x = rng.integers(112, 128, k) * 2 + 1.0                       # odd, 225 to 255
    W = np.floor(rng.uniform(w_low, w_top, (n, k)) / 2) * 2 + 1.0   # odd
    W = np.minimum(W, w_top - (1 - w_top % 2))
    W[:, 5::16] -= 1                                              # one even product of 16: the sum is odd
    x[0::64] = 1                                                  # the place that makes 64 products a multiple of 64
    W[:, 0::64] = 0
    rest = (W * x).reshape(n, -1, 64).sum(2)
    W[:, 0::64] = (-rest) % 64 + 64
    assert (W[:, 0::64] % 2 == 1).all()                           # so the first 16's sum is odd as well
    x[k - 64:], W[:, k - 64:] = 0, 0
    total = W @ x
    left = total - (64 + 64 * (np.arange(n) % 3))
    assert (left > 0).all() and left.max() < 2 ** 30
    for j in range(3):                                            # eight bits each: BF16 holds them
        part = np.floor(left / 2.0 ** (6 + 8 * j)) % 256
        x[k - 64 + j], W[:, k - 64 + j] = 2.0 ** (6 + 8 * j), -part
    assert (W @ x == 64 + 64 * (np.arange(n) % 3)).all()
    assert (W * x)[:, :most].sum(1).max() < 2 ** 24
    return x, W


# n: a whole tile of columns and odd ones
@pytest.mark.parametrize("T,n", [(3, 131), (260, 48)], ids=str)
@pytest.mark.parametrize("k", [512, 1536, 4096, 12480, 32768])
def test_a_kept_forward_product_rounds_its_sums_often_enough(k, T, n):
    x, W = long_sums(k, terms(k, True), n, k)
    want = np.broadcast_to(W @ x, (T, n))
    X = np.broadcast_to(x, (T, k)).copy()
    for fmt in ("e4m3", "e5m2"):
        out = gated_forward(X, W, W[::-1].copy(), "silu", "bf16", fmt=fmt)
        assert out["status"] == 0
        assert np.array_equal(out["gate"], want) and np.array_equal(out["up"], want[:, ::-1])


@pytest.mark.parametrize("k", [1024, 4096, 12480])
def test_products_round_their_sums_often_enough(k):
    T, n = 70, 96
    x, W = long_sums(k, 1024, n, k)
    X, V = np.broadcast_to(x, (T, k)).copy(), np.ascontiguousarray(W.T)
    want = np.broadcast_to(W @ x, (T, n))
    out = gated_forward(X, W, W, "silu", "bf16")
    assert np.array_equal(out["gate"], want) and np.array_equal(out["up"], want)
    assert np.array_equal(linear(X, W, "bf16"), want)
    assert np.array_equal(input_grad(X, V, "bf16"), want)
    assert np.array_equal(input_grad(X, V, "bf16", X, V), 2 * want)
    dg, _ = gated_backward(X, V, np.zeros((T, n)), np.full((T, n), 2.0), "silu", "bf16")   # a'(0) = 1/2
    assert np.array_equal(dg, want)


# k of the first segment only, of a last one of one stage or of a part of it, and of many; one tile, and nine
@pytest.mark.parametrize("sms", [None, 2], ids=["", "one-pair"])
@pytest.mark.parametrize("off", [False, True], ids=["aligned", "unaligned"])
@pytest.mark.parametrize("T,n", [(40, 48), (600, 272)], ids=str)
@pytest.mark.parametrize("k", [100, 256, 320, 769, 1536, 2000, 4096])
def test_segments_of_a_kept_forward_product(k, T, n, off, sms):
    """gate, up, h, codes and scales from whole numbers.  The gates are at least 20, where a(g) = g in FP32."""
    c = None
    if sms:
        c = G.Context(torch.cuda.current_device())
        G.gift_set_option(c, G.OPT_SMS, sms)
    rng = np.random.default_rng(k + T)
    x, W, W2 = (rng.integers(-m, m + 1, s).astype(float) for m, s in ((8, (T, k)), (1, (n, k)), (1, (n, k))))
    bias = rng.integers(2000, 2101, n).astype(float)
    g, u = x @ W.T + bias, x @ W2.T
    h = g * u
    assert g.min() >= 20 and np.abs(h).max() < 2 ** 24
    for fmt in ("e4m3", "e5m2"):
        out = gated_forward(x, W, W2, "silu", "bf16", bg=bias, fmt=fmt, off=off, c=c)
        assert out["status"] == 0
        for key, want in (("gate", g), ("up", u), ("h", h)):
            assert np.array_equal(out[key], rounded(want, "bf16")), key
        codes, scales = A.encode(h, fmt)
        assert np.array_equal(out["scales"], scales) and np.array_equal(out["codes"], codes)
