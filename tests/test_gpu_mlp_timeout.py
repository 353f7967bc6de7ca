"""The products' bounded waits end: with a small wait budget the kernel reports GIFT_ERR_TIMEOUT, ends with none of its
copies or products in flight, and the same context then computes the right result (no GPU fault, no hang).

A budget of 0 gives up at the first wait that is not over within a few microseconds.  On a context of two SMs the
operands' preparation takes far longer than that (each of its 128 warps copies over a hundred spans, one after the
other, each at least a trip to memory), and the product's kernel starts beside it on the idle SMs: the call always reports.
On the whole GPU, and with longer budgets, it gives up in the middle of the pipeline or not at all; either way the call
ends, and a status of 0 means the right answer.
"""
import numpy as np
import pytest
import torch

from fac_whitening_gb300 import gift as G
from gpu_util import DEV, status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("op", ["gated_forward", "gated_backward", "linear", "input_grad"])
@pytest.mark.parametrize("shape", [(20000, 99, 144), (3000, 263, 528), (1100, 777, 1024)], ids=str)
def test_waits_run_out_and_the_context_survives(shape, op, dt):
    T, k, n = shape
    c = G.Context(torch.cuda.current_device())
    few = T == 20000
    if few:
        G.gift_set_option(c, G.OPT_SMS, 2)
    rng = np.random.default_rng(T)
    put = lambda x: torch.as_tensor(x.astype(np.float64)).to(DEV, dt)  # noqa: E731
    x, W = put(rng.integers(-3, 4, (T, k))), put(rng.integers(-1, 2, (n, k)))
    V = W.t().contiguous()
    want = x.double() @ V.double()
    new = lambda: torch.empty(T, n, dtype=dt, device=DEV)  # noqa: E731
    ws = lambda name, a, b: torch.empty(G.gift_act_workspace_bytes(c, name, dt, T, a, b), dtype=torch.uint8, device=DEV)  # noqa: E731,E501
    y, other, third, zero, two = new(), new(), new(), torch.zeros(T, n, dtype=dt, device=DEV), new()
    two.fill_(2.0)
    if op == "gated_forward":
        w = ws("gated_forward", n, k)
        call = lambda st: G.gift_gated_forward(c, x, W, W, "silu", third, gate=y, up=other, ws=w, status=st)  # noqa: E731
    elif op == "gated_backward":   # at gate 0: a' = 1/2
        w = ws("gated_backward", k, n)
        call = lambda st: G.gift_gated_backward(c, x, V, zero, two, "silu", y, other, ws=w, status=st)  # noqa: E731
    elif op == "linear":
        w = ws("linear_forward", n, k)
        call = lambda st: G.gift_linear_forward(c, x, W, y, residual=zero, ws=w, status=st)  # noqa: E731
    else:
        w = ws("input_grad", k, n)
        call = lambda st: G.gift_input_grad(c, x, V, y, ws=w, status=st)  # noqa: E731

    def run(budget):
        G.gift_set_option(c, G.OPT_BARRIER_WAIT, budget)
        y.fill_(0.5)
        st = status()
        call(st)
        torch.cuda.synchronize()
        return int(st.item())

    def right():
        return torch.equal(y, want.to(dt))

    assert run(2_000_000_000) == 0 and right()   # loads the kernels
    for budget in (0, 500, 2000, 20000):
        st = run(budget)
        assert st == G.ERR_TIMEOUT if few and budget == 0 else st in (0, G.ERR_TIMEOUT)
        assert st or right()
        assert run(2_000_000_000) == 0 and right()
