"""The weight gradient's bounded waits end: with a small wait budget the tensor-core kernel reports
GIFT_ERR_TIMEOUT, ends with none of its copies or products in flight, and the same context then
computes the right gradient (no GPU fault, no hang).

A budget of 0 gives up at the first wait that is not over within a few microseconds.  On a context of two SMs the
operands' preparation takes far longer than that (each of its 128 warps copies 156 rows, one after the other,
each at least a trip to memory), and the product's kernel starts beside it on the idle SMs: the call always
reports.  On the whole GPU, and with longer budgets, it gives up in the middle of the pipeline or not at all;
either way the call ends, and a status of 0 means the right answer.
"""
import numpy as np
import pytest
import torch

import act_ref as R
from fac_whitening_gb300 import gift as G
from gpu_util import DEV, status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(20000, 263, 272), (20000, 99, 528), (3000, 264, 528), (1100, 100, 4864)], ids=str)
def test_waits_run_out_and_the_context_survives(shape, dt):
    T, d_out, d_in = shape
    c = G.Context(torch.cuda.current_device())
    few = T == 20000
    if few:
        G.gift_set_option(c, G.OPT_SMS, 2)
    rng = np.random.default_rng(T)
    delta = torch.as_tensor(rng.integers(-3, 4, (T, d_out))).to(DEV, dt)
    codes, scales = R.encode(rng.integers(-7, 8, (T, d_in)).astype(np.float64), "e4m3")
    v = torch.as_tensor(R.decode(codes, scales, "e4m3")).to(DEV)
    want, wb = delta.double().t() @ v, delta.double().sum(0)
    codes, scales = torch.as_tensor(codes).to(DEV), torch.as_tensor(scales).to(DEV)
    dW, db = torch.empty(d_out, d_in, device=DEV), torch.empty(d_out, device=DEV)
    ws = torch.empty(G.gift_act_workspace_bytes(c, "weight_grad", dt, T, d_out, d_in), dtype=torch.uint8, device=DEV)

    def call(budget):
        G.gift_set_option(c, G.OPT_BARRIER_WAIT, budget)
        st = status()
        G.gift_weight_grad(c, delta, codes, scales, "e4m3", dW, db=db, ws=ws, status=st)
        torch.cuda.synchronize()
        return int(st.item())

    def right():
        return torch.equal(dW.double(), want) and torch.equal(db.double(), wb)

    assert call(2_000_000_000) == 0 and right()   # loads the kernels
    for budget in (0, 500, 2000, 20000):
        st = call(budget)
        assert st == G.ERR_TIMEOUT if few and budget == 0 else st in (0, G.ERR_TIMEOUT)
        assert st or right()
        assert call(2_000_000_000) == 0 and right()
