"""The checkpointed layer's training steps run end to end and learn."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import checkpointed_layer
    finally:
        sys.path.pop(0)
    return checkpointed_layer


def test_training_with_8_bit_checkpoints_and_the_codec():
    losses, error, kept = _example().train(tokens=1024, d_in=512, d_out=128, steps=6)
    assert losses[-1] < 0.5 * losses[0]
    # E4M3 rounds an element by 2^-4 at most; mapping back stretches that by at most T_A's condition,
    # sqrt(mu_1 / sigma) < 4 for these activations
    assert error < 0.25
    assert kept < 0.52 * 2 * 1024 * 512       # half of the BF16 input, and scales


def test_gradients_of_the_checkpointed_layer_match_the_plain_ones():
    ex = _example()
    from fac_whitening_gb300 import gift as G
    gen = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    T, d, o = 300, 520, 136
    x, W = r(T, d).requires_grad_(), (0.1 * r(o, d)).requires_grad_()
    gamma, beta = (1 + 0.1 * r(d)).requires_grad_(), (0.1 * r(d)).requires_grad_()
    w = r(T, o)
    (ex.NormLinear.apply(x, gamma, beta, W, G.Context(torch.cuda.current_device()), {}) * w).sum().backward()
    got = [p.grad.clone() for p in (x, gamma, beta, W)]
    for p in (x, gamma, beta, W):
        p.grad = None
    ((torch.nn.functional.layer_norm(x, (d,), gamma, beta, 1e-5) @ W.t()) * w).sum().backward()
    # an E4M3 checkpoint rounds each kept value by up to 2^-4: 2^-4 / sqrt(3) of its size at random
    for a, p in zip(got, (x, gamma, beta, W)):
        assert (a - p.grad).norm() <= 0.04 * p.grad.norm()
