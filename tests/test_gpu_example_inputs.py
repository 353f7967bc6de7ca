"""What the checkpointed layer's example gives the codec: the factor is that of the linear layer's inputs
a = gamma n + beta (not of the norm's rows n), of replica 0's batch."""
import pytest
import torch

from test_gpu_example import _example

pytestmark = pytest.mark.gpu


def _record(ex, monkeypatch):
    """Every layer-norm output and every activation matrix that reaches the factor refresh, in order."""
    outs, acts = [], []
    forward, update = ex.G.gift_layernorm_forward, ex.G.gift_factor_update

    def norm(ctx, x, gamma, beta, eps, y, **kw):
        forward(ctx, x, gamma, beta, eps, y, **kw)
        outs.append((y.detach().float().clone(), gamma.detach().clone(), beta.detach().clone()))

    def refresh(ctx, fac, a, **kw):
        acts.append(a.detach().float().clone())
        update(ctx, fac, a, **kw)

    monkeypatch.setattr(ex.G, "gift_layernorm_forward", norm)
    monkeypatch.setattr(ex.G, "gift_factor_update", refresh)
    return outs, acts


def test_the_factor_is_that_of_the_layers_inputs(monkeypatch):
    ex = _example()
    outs, acts = _record(ex, monkeypatch)
    ones, zeros = torch.ones, torch.zeros
    # a trained norm's gain and offset instead of the first step's 1 and 0
    gen = torch.Generator(device="cuda").manual_seed(5)
    r = lambda n: torch.randn(n, device="cuda", generator=gen)  # noqa: E731
    def parameter(plain, value):
        return lambda *n, **kw: value(*n).requires_grad_() if kw.get("requires_grad") else plain(*n, **kw)

    monkeypatch.setattr(torch, "ones", parameter(ones, lambda n: 1.5 + 0.5 * r(n)))
    monkeypatch.setattr(torch, "zeros", parameter(zeros, lambda n: 2.0 * r(n)))
    replicas = 2
    ex.train(tokens=512, d_in=256, d_out=64, steps=2, replicas=replicas)
    assert len(outs) == 2 * replicas and len(acts) == 2
    for step, a in enumerate(acts):
        y, gamma, beta = outs[replicas * step]
        # y = gamma n + beta rounded to BF16; a is that of the checkpoint's n, an E4M3 code each (2^-4 of n, and
        # 2^-17 of its group's largest, below 16 for these rows, where codes are subnormal), rounded to BF16
        n = ((y - beta) / gamma).abs()
        bound = gamma.abs() * (n * 2.0 ** -4 + 2.0 ** -13) + 2.0 ** -7 * (y.abs() + gamma.abs() * n + beta.abs())
        assert ((a - y).abs() <= bound).all()
