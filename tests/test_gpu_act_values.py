"""Values at the ends of FP32's range through the layer norm and the weight gradient: a result is right or is
reported, never quietly something else.  Tolerances as in test_gpu_act.py."""
import numpy as np
import pytest
import torch

import act_ref as R
from fac_whitening_gb300 import gift as G
from test_gpu_act import DT, forward, host
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
