"""The gated block's example: it runs, and its gradients are the block's."""
import math
import os
import sys

import numpy as np
import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

import mlp_ref as R  # noqa: E402
from gpu_util import ctx  # noqa: E402

pytestmark = pytest.mark.gpu


def test_example_runs():
    import gated_block as E
    losses, error = E.train(tokens=300, d=64, f=160, steps=2)
    assert len(losses) == 2 and all(math.isfinite(v) for v in losses)
    assert 0 < error < 0.2   # E4M3: half a step of four significant bits at most, 2^-4, of each whitened value's share


def test_example_gradients():
    """Against the block in 64 bits.  BF16 activations are off by at most 2^-8 each and the checkpoints by 2^-4, so with
    every rounding on the way the input's gradient, which meets n's checkpoint in the norm only, and the weights'
    are held to 2^-4 of their norm, biases and gain to the same."""
    import gated_block as E
    T, d, f, p, site = 200, 64, 144, 0.25, 5
    params, r = E.parameters(d, f, 3)
    x = r(T, d).to(torch.bfloat16).requires_grad_()
    dy = r(T, d).to(torch.bfloat16)
    rng = torch.tensor([11, 4], dtype=torch.int64, device="cuda")
    kept = {"status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    y = E.GatedBlock.apply(x, *params, ctx(), p, rng, site, kept)
    got = torch.autograd.grad(y, [x, *params], dy)
    assert int(kept["status"].item()) == 0
    q = [t.detach().double().requires_grad_() for t in [x, *params]]
    x64, gamma, beta, Wg, Wu, W, b = q
    n = torch.nn.functional.layer_norm(x64, (d,), gamma, beta, 1e-5)
    h = torch.nn.functional.silu(n @ Wg.t()) * (n @ Wu.t())
    keep = torch.as_tensor(R.keep(T, d, p, 11, 4, site)).cuda()
    v = h @ W.t() + b
    want_y = x64 + torch.where(keep, v / (1 - R.threshold(p) / 65536), torch.zeros_like(v))
    want = torch.autograd.grad(want_y, q, dy.double())
    assert ((y.double() - want_y).norm() / want_y.norm()).item() < 2.0 ** -6
    for g, w in zip(got, want):
        assert ((g.double() - w).norm() / w.norm()).item() < 2.0 ** -4
    assert np.isfinite(got[0].float().cpu().numpy()).all()
