"""Host-side checks of the feed-forward calls: refusals that need no GPU, and the plain statements by themselves."""
import ctypes

import numpy as np
import pytest

import mlp_ref as R
from fac_whitening_gb300 import gift as G


def _lib_or_skip():
    try:
        return G.lib()
    except RuntimeError as e:  # not built in this checkout
        pytest.skip(str(e))


def test_null_context_is_rejected():
    lib = _lib_or_skip()
    n, bf16, e4m3, bad = None, G.DTYPE["bf16"], G.FMT["e4m3"], G.ERR_INVALID_ARG
    for op in ("gated_forward", "gated_backward", "linear_forward", "input_grad", "dropout_backward"):
        assert lib.gift_act_workspace_bytes(n, G.OP[op], bf16, 4, 4, 4) == ctypes.c_size_t(-1).value
    assert lib.gift_gated_forward(n, n, bf16, 4, 4, n, n, 4, n, n, 0, n, n, n, e4m3, n, n, n, 0, n, n) == bad
    assert lib.gift_gated_backward(n, n, bf16, 4, 4, n, 4, n, n, 0, n, n, n, 0, n, n) == bad
    assert lib.gift_linear_forward(n, n, bf16, 4, 4, n, 4, n, n, 0.0, n, 0, n, n, 0, n, n) == bad
    assert lib.gift_input_grad(n, n, n, n, n, bf16, 4, 4, 4, n, n, 0, n, n) == bad
    assert lib.gift_dropout_forward(n, n, bf16, 4, 4, n, n, 0.0, n, 0, n, n) == bad
    assert lib.gift_dropout_backward(n, n, bf16, 4, 4, 0.0, n, 0, n, n, n, 0, n) == bad


def test_binding_refuses_what_the_kernels_would_misread():
    import torch

    class Cuda:   # stands in for a device tensor (no GPU here)
        is_cuda = True

        def __init__(self, n, dtype):
            self.t = torch.empty(n, dtype=dtype)
            self.shape, self.dtype = self.t.shape, dtype

        def __getattr__(self, name):
            return getattr(self.t, name)

    assert G._rng(None) is None
    assert isinstance(G._rng(Cuda(2, torch.int64)), int)
    for bad in (Cuda(2, torch.int32), Cuda(3, torch.int64), Cuda(2, torch.float64)):
        with pytest.raises(ValueError, match="64-bit"):
            G._rng(bad)
    with pytest.raises(ValueError, match="device memory"):
        G._rng(torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="Wg"):
        G._buf(Cuda(7, torch.bfloat16), 8, "Wg", torch.bfloat16)
    with pytest.raises(ValueError, match="Wg"):
        G._buf(Cuda(8, torch.float16), 8, "Wg", torch.bfloat16)


def test_philox_known_answers():
    # the generator's published test vectors (counter, key -> output)
    for c, k, want in (
            ([0] * 4, [0] * 2, [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
            ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
            ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
             [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1])):
        assert [int(v) for v in R.philox([np.uint64(x) for x in c], k)] == want


def test_dropped_share_and_independence_of_the_reference_mask():
    T, d, p = 512, 1024, 0.1
    a, b, c = (R.keep(T, d, p, 1 << 60, s, site) for s, site in ((5, 0), (5, 1), (6, 0)))
    n, q = T * d, R.threshold(p) / 65536
    for m in (a, b, c):
        assert abs(np.mean(~m) - q) < 5 * np.sqrt(q * (1 - q) / n)
    for x, y in ((a, b), (a, c)):   # both dropped as often as independent bits are
        assert abs(np.mean(~x & ~y) - q * q) < 5 * np.sqrt(q * q / n)


@pytest.mark.parametrize("fn", ["silu", "gelu", "gelu_tanh"])
def test_gate_slope_is_the_derivative(fn):
    g = np.linspace(-8, 8, 4001)
    h = 1e-5
    a, slope = R.gate(g, fn)
    diff = (R.gate(g + h, fn)[0] - R.gate(g - h, fn)[0]) / (2 * h)
    assert np.abs(diff - slope).max() < 1e-9   # h^2 / 6 times the third derivative, and rounding over h
    assert np.abs(slope).max() < 1.13
