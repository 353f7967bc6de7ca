"""Values at the ends of FP32's range through the layer norm and the weight gradient: a result is right or is
reported, never quietly something else.  Tolerances as in test_gpu_act.py."""
import numpy as np
import pytest
import torch

import act_ref as R
from fac_whitening_gb300 import gift as G
from test_gpu_act import DT, forward, host, weight_grad
from gpu_util import DEV

pytestmark = pytest.mark.gpu


# one width for each way a row is held: element and wide accesses, one to four pieces per lane, and the
# rows that are read again
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("d", [200, 256, 1536, 4096, 16400, 40000])
def test_norm_forward_reports_a_variance_beyond_fp32(d, dt):
    # every element is finite and so is the mean; the squared deviations (1e50) are not FP32 values
    x = torch.as_tensor(np.random.default_rng(d).standard_normal((5, d))).to(DT[dt])
    x[3, ::2], x[3, 1::2] = 1e25, -1e25
    y, mean, rstd, _, _, st = forward(x.to(DEV), None, None, 1e-5)
    assert st == G.ERR_NONFINITE
    # the other rows are what they are without it
    x[3] = 0.0
    y0, _, _, _, _, st = forward(x.to(DEV), None, None, 1e-5)
    keep = [0, 1, 2, 4]
    assert st == 0 and torch.equal(y[keep], y0[keep])


@pytest.mark.parametrize("d", [200, 256, 1536, 4096, 16400, 40000])
def test_norm_forward_of_large_rows_within_fp32(d):
    # deviations of 1e16: sums of d squares up to 4e36 stay below FP32's largest value
    x = torch.as_tensor(np.random.default_rng(d).uniform(-1e16, 1e16, (3, d))).float()
    y, _, rstd, _, _, st = forward(x.to(DEV), None, None, 1e-5)
    wy, _, wm, wr = R.norm_forward(x.double().numpy(), None, None, 1e-5)
    N = d + 8
    tol_m = N * R.U32 * np.abs(x.double().numpy()).mean(axis=1) * wr   # the mean's error in units of a deviation
    assert st == 0
    assert np.all(np.abs(host(rstd) - wr) <= wr * (N * R.U32 + tol_m + 4 * R.U32))
    assert np.all(np.abs(host(y) - wy) <= np.abs(wy) * ((N + 8) * R.U32 + tol_m[:, None]) + tol_m[:, None])


# ---- weight gradient: FP32 gradients at the ends of the range ---------------------------------------------
# the small product; the tensor cores with db from the group of ones; with db by the pass over delta
WIDE_RANGE_SHAPES = [(130, 40, 400), (300, 264, 528), (1100, 1024, 4864)]


def _rows_of_ones(T, d, seed):
    """A checkpoint of values +-1 and 0 (every 7th column of every third token)."""
    v = np.random.default_rng(seed).choice([-1.0, 1.0], (T, d))
    v[::3, ::7] = 0.0
    codes, scales = R.encode(v, "e4m3")
    return v, torch.as_tensor(codes).to(DEV), torch.as_tensor(scales).to(DEV)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", WIDE_RANGE_SHAPES, ids=str)
def test_weight_grad_infinite_gradient_follows_the_formula(shape, dt):
    T, d_out, d_in = shape
    delta = np.random.default_rng(T).integers(-3, 4, (T, d_out)).astype(np.float64)
    delta[T // 3, 1], delta[T - 1, d_out - 1], delta[5, 7] = np.inf, -np.inf, np.nan
    v, codes, scales = _rows_of_ones(T, d_in, d_out)
    dW, db = weight_grad(torch.as_tensor(delta).to(DEV, DT[dt]), codes, scales, "e4m3", d_in)
    finite = np.where(np.isfinite(delta), delta, 0.0)
    want, wb = R.weight_grad(finite, v)
    for o, t in ((1, T // 3), (d_out - 1, T - 1)):      # Inf * v: an infinity of v's sign, NaN where v is 0
        with np.errstate(invalid="ignore"):
            want[o] = delta[t, o] * v[t]
        wb[o] = delta[t, o]
    want[7], wb[7] = np.nan, np.nan
    assert np.array_equal(host(dW), want, equal_nan=True)
    assert np.array_equal(host(db), wb, equal_nan=True)


@pytest.mark.parametrize("shape", WIDE_RANGE_SHAPES, ids=str)
def test_weight_grad_of_the_largest_fp32_gradients(shape):
    # above 3.3961e38 an FP32 value rounds to infinity in BF16; one such token an output, whose sums (the values
    # are 0 and +-1) are that value itself: three products, at most 2u from truncation each
    T, d_out, d_in = shape
    delta = np.zeros((T, d_out), dtype=np.float32)
    big = np.array([3.4028234e38, -3.4028234e38, 3.3961776e38, -3.4e38, 3.39e38, 3.2e38], dtype=np.float32)
    at = np.arange(d_out) % T
    delta[at, np.arange(d_out)] = big[np.arange(d_out) % len(big)]
    v, codes, scales = _rows_of_ones(T, d_in, d_out)
    dW, db = weight_grad(torch.as_tensor(delta).to(DEV), codes, scales, "e4m3", d_in)
    want, wb = R.weight_grad(delta.astype(np.float64), v)
    assert np.all(np.abs(host(dW) - want) <= 6 * R.U32 * np.abs(want))
    assert np.all(np.abs(host(db) - wb) <= 6 * R.U32 * np.abs(wb))


@pytest.mark.parametrize("shape", WIDE_RANGE_SHAPES, ids=str)
def test_weight_grad_of_the_smallest_fp32_gradients(shape):
    # below 2^-110 the third term ends at BF16's smallest step, 2^-133: half of it is lost an element at most.
    # One token an output, as above
    T, d_out, d_in = shape
    rng = np.random.default_rng(T)
    delta = np.zeros((T, d_out), dtype=np.float32)
    at = np.arange(d_out) % T
    delta[at, np.arange(d_out)] = np.ldexp(rng.uniform(1, 2, d_out), rng.integers(-126, -100, d_out))
    v, codes, scales = _rows_of_ones(T, d_in, d_out)
    dW, db = weight_grad(torch.as_tensor(delta).to(DEV), codes, scales, "e4m3", d_in)
    want, wb = R.weight_grad(delta.astype(np.float64), v)
    assert np.all(np.abs(host(dW) - want) <= 6 * R.U32 * np.abs(want) + 2.0 ** -134 * np.abs(v).max())
    assert np.all(np.abs(host(db) - wb) <= 6 * R.U32 * np.abs(wb) + 2.0 ** -134)
