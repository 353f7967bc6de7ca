"""The wait budget is the pipeline's: the launch that prepares a product's operands, beside which the product's kernel starts, does
not use it up."""
import numpy as np
import pytest
import torch

from fac_whitening_gb300 import gift as G
from gpu_util import DEV, status

pytestmark = pytest.mark.gpu
T, K, N = 200_000, 99, 72
BUDGET = 400_000   # clocks: about 200 us


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("op", ["gated_forward", "gated_backward", "linear", "input_grad"])
def test_preparing_the_operands_uses_up_no_wait(op, dt):
    """On two SMs each of the 128 warps that prepare operands makes over 1500 spans, one after the other, each at least a
    trip to memory: a millisecond.  A pipeline's wait is over after a tile's product or its epilogue, some microseconds."""
    c = G.Context(torch.cuda.current_device())
    G.gift_set_option(c, G.OPT_SMS, 2)
    G.gift_set_option(c, G.OPT_BARRIER_WAIT, BUDGET)
    rng = np.random.default_rng(1)
    put = lambda x: torch.as_tensor(x.astype(np.float64)).to(DEV, dt)  # noqa: E731
    x, W = put(rng.integers(-3, 4, (T, K))), put(rng.integers(-1, 2, (N, K)))
    V = W.t().contiguous()
    want = (x.double() @ V.double()).to(dt)
    y, other, third = (torch.empty(T, N, dtype=dt, device=DEV) for _ in range(3))
    zero, two, st = torch.zeros(T, N, dtype=dt, device=DEV), torch.full((T, N), 2.0, dtype=dt, device=DEV), status()
    ws = lambda name, a, b: torch.empty(G.gift_act_workspace_bytes(c, name, dt, T, a, b), dtype=torch.uint8, device=DEV)  # noqa: E731,E501
    for _ in range(3):   # the first call loads the kernels
        y.fill_(0.5)
        if op == "gated_forward":
            G.gift_gated_forward(c, x, W, W, "silu", third, gate=y, up=other, ws=ws("gated_forward", N, K), status=st)
        elif op == "gated_backward":   # at gate 0: a' = 1/2
            G.gift_gated_backward(c, x, V, zero, two, "silu", y, other, ws=ws("gated_backward", K, N), status=st)
        elif op == "linear":
            G.gift_linear_forward(c, x, W, y, residual=zero, ws=ws("linear_forward", N, K), status=st)
        else:
            G.gift_input_grad(c, x, V, y, ws=ws("input_grad", K, N), status=st)
        assert int(st.item()) == 0 and torch.equal(y, want)
