"""The 64-bit statements the GPU tests compare with, against torch on the CPU and differences."""
import numpy as np
import pytest
import torch

import act_ref as R


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_checkpoint_reference_against_torch_casts(fmt):
    f8 = torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((40, 300)) * np.exp(3 * rng.standard_normal((40, 300)))).astype(np.float32)
    x[0], x[1, :5] = 0.0, -0.0
    codes, scales = R.encode(x, fmt)
    inv = np.ldexp(1.0, 127 - np.repeat(scales.astype(int), 128, axis=1)[:, :300])
    want = torch.tensor(x.astype(np.float64) * inv).float().to(f8).view(torch.uint8).numpy()
    assert np.array_equal(codes, want)
    v = R.decode(codes, scales, fmt)
    assert np.array_equal(v, torch.tensor(v).to(torch.bfloat16).double().numpy())   # exact in BF16
    amax = np.abs(x.astype(np.float64))[:, :128].max(axis=1)
    k = scales[:, 0].astype(int) - 127
    fmax = R.magnitudes(fmt)[-1]
    live = amax > 0
    assert np.all(amax[live] <= fmax * 2.0 ** k[live]) and np.all(amax[live] > fmax * 2.0 ** (k[live] - 1))


def test_checkpoint_reference_extremes():
    for fmt, emax in R.EMAX.items():
        x = np.array([[3.4e38, 1.0], [1e-38, 0.0], [np.nan, 1.0], [np.inf, 0.0]])
        s = R.scale_bytes(x, fmt)[:, 0]
        assert list(s) == [127 + 127 - emax, 17, 255, 255]
        assert np.isfinite(R.decode(*R.encode(x[:2], fmt), fmt)).all()


def test_norm_reference_against_differences():
    rng = np.random.default_rng(2)
    T, d, eps = 3, 17, 1e-5
    x, g, b = rng.standard_normal((T, d)), 1 + 0.2 * rng.standard_normal(d), rng.standard_normal(d)
    w = rng.standard_normal((T, d))
    _, n, _, rstd = R.norm_forward(x, g, b, eps)
    dx, dg, db = R.norm_backward(w, n, g, rstd)

    def loss(x, g, b):
        return float((w * R.norm_forward(x, g, b, eps)[0]).sum())

    for arr, grad, args in ((x, dx, lambda e: (x + e, g, b)), (g, dg, lambda e: (x, g + e, b)),
                            (b, db, lambda e: (x, g, b + e))):
        v = rng.standard_normal(arr.shape)
        h = 1e-5
        diff = (loss(*args(h * v)) - loss(*args(-h * v))) / (2 * h)
        assert abs(diff - (grad * v).sum()) <= 1e-6 * max(1.0, abs(diff))
    tx = torch.tensor(x, requires_grad=True)
    torch.nn.functional.layer_norm(tx, (d,), torch.tensor(g), torch.tensor(b), eps).mul(torch.tensor(w)).sum().backward()
    assert np.allclose(tx.grad.numpy(), dx, rtol=1e-10, atol=1e-12)
