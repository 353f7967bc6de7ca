"""Conditions that only the device sees in the checkpointed layer's passes reach the example's caller."""
import pytest
import torch

from fac_whitening_gb300 import gift as G
from test_gpu_example import _example

pytestmark = pytest.mark.gpu


def test_a_nonfinite_row_reaches_the_status_word():
    ex = _example()
    T, d, o = 64, 256, 32
    x = torch.randn(T, d, device="cuda")
    x[5, 7] = float("nan")
    kept = {"status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    ones, W = torch.ones(d, device="cuda"), torch.randn(o, d, device="cuda").requires_grad_()
    ex.NormLinear.apply(x, ones, torch.zeros(d, device="cuda"), W, G.Context(torch.cuda.current_device()), kept)
    assert int(kept["status"].item()) == G.ERR_NONFINITE


@pytest.mark.parametrize("call", ["gift_layernorm_forward", "gift_weight_grad", "gift_layernorm_backward"])
def test_training_stops_on_a_reported_condition(call, monkeypatch):
    ex = _example()
    plain = getattr(ex.G, call)

    def reporting(*a, **kw):
        plain(*a, **kw)
        if kw.get("status") is not None:
            kw["status"].fill_(G.ERR_TIMEOUT)

    monkeypatch.setattr(ex.G, call, reporting)
    with pytest.raises(G.GiftError) as e:
        ex.train(tokens=256, d_in=256, d_out=64, steps=1)
    assert e.value.status == G.ERR_TIMEOUT
