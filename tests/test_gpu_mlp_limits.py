"""The feed-forward calls at the ends of what they take."""
import pytest
import torch

from fac_whitening_gb300 import gift as G
from gpu_util import DEV, ctx

pytestmark = pytest.mark.gpu
MOST = 1 << 30


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("op,n_is_out", [("gated_forward", True), ("linear_forward", True), ("gated_backward", False),
                                         ("input_grad", False)])
def test_no_workspace_for_an_output_of_too_many_tiles(op, n_is_out, dt):
    """2^31 - 1 tiles of 256 x 64 at the most.  Host arithmetic only; nothing is launched."""
    def size(T, n, k):
        return G.gift_act_workspace_bytes(ctx(), op, dt, T, *((n, k) if n_is_out else (k, n)))

    # 2^9 tiles of 64 columns by 2^22 of 256 rows are one too many, and so is much more
    for T, n in ((MOST, 64 * 512), (MOST, MOST), (MOST - 255, 64 * 511 + 1), (256 * 128, MOST)):
        with pytest.raises(G.GiftError):
            size(T, n, 16)
    for T, n in ((MOST, 64 * 511), (MOST - 256, 64 * 512), (1, MOST), (MOST, 1)):
        assert size(T, n, 16) >= 0
    # terms of FP32, or copies of BF16 rows that TMA cannot read: the token and a row of the weights, 2 bytes a number
    assert size(1, 1, MOST) >= 4 * MOST


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_the_residual_stream_may_be_the_input_but_not_the_output_too(dt):
    """y = x + x W^T: y in a buffer of its own is right, in x's place it is refused (other tiles still read x)."""
    T, d = 300, 64
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randint(-8, 9, (T, d), device=DEV, generator=g).to(dt)
    W = torch.randint(-1, 2, (d, d), device=DEV, generator=g).to(dt)
    ws = torch.empty(G.gift_act_workspace_bytes(ctx(), "linear_forward", dt, T, d, d), dtype=torch.uint8, device=DEV)
    y, want = torch.empty_like(x), (x.double() + x.double() @ W.double().t()).to(dt)
    G.gift_linear_forward(ctx(), x, W, y, residual=x, ws=ws)
    assert torch.equal(y, want)
    kept = x.clone()
    with pytest.raises(G.GiftError):
        G.gift_linear_forward(ctx(), x, W, x, residual=x, ws=ws)
    with pytest.raises(G.GiftError):
        G.gift_linear_forward(ctx(), x[:d], W, W, residual=x[:d], ws=ws)
    assert torch.equal(x, kept)
