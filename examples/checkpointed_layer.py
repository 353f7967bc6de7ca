"""A training step whose activations wait for the backward pass in 8 bits, with GIFT behind it.

One layer, norm -> linear -> squared error, for R data-parallel replicas modelled on one GPU:

  forward    gift_layernorm_forward keeps the normalised rows as an 8-bit checkpoint; nothing else
             of the layer's input is kept;
  backward   gift_weight_grad makes the linear layer's weight gradient from the checkpoint (the norm's
             gain and offset folded in), gift_layernorm_backward the norm's own gradients from it;
  codec      the layer's K-FAC factor from replica 0's inputs (the checkpoint's values with the norm's
             gain and offset), then every replica's weight gradient whitened, packed to E4M3,
             averaged and mapped back (GIFT's Algorithm 1).

    python examples/checkpointed_layer.py [--tokens 4096] [--d-in 1536] [--d-out 384] [--steps 10]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from fac_whitening_gb300 import gift as G  # noqa: E402

FMT, EPS = "e4m3", 1e-5


class NormLinear(torch.autograd.Function):
    """y = norm(x; gamma, beta) W^T, keeping an 8-bit checkpoint of the norm's rows between the passes.
    `kept` gets the checkpoint; its "status" word, where there is one, gets what only the device sees."""

    @staticmethod
    def forward(c, x, gamma, beta, W, ctx, kept):
        T, d = x.shape
        dev = x.device
        cb, sb = G.gift_act_sizes(FMT, T, d)
        codes, scales = torch.empty(cb, dtype=torch.uint8, device=dev), torch.empty(sb, dtype=torch.uint8, device=dev)
        y, rstd = torch.empty_like(x), torch.empty(T, device=dev)
        G.gift_layernorm_forward(ctx, x, gamma, beta, EPS, y, rstd=rstd, fmt=FMT, codes=codes, scales=scales,
                                 status=kept.get("status"))
        c.save_for_backward(codes, scales, rstd, gamma, beta, W)
        c.ctx, c.status = ctx, kept.get("status")
        kept["bytes"] = codes.numel() + scales.numel() + 4 * T
        kept["checkpoint"], kept["gain"], kept["offset"] = (codes, scales), gamma.detach(), beta.detach()
        return y @ W.to(x.dtype).t()

    @staticmethod
    def backward(c, delta):
        codes, scales, rstd, gamma, beta, W = c.saved_tensors
        delta = delta.contiguous()
        T, d_out = delta.shape
        d, dev = W.shape[1], delta.device
        new = lambda n: torch.empty(max(n, 1), dtype=torch.uint8, device=dev)  # noqa: E731
        dW = torch.empty_like(W)
        G.gift_weight_grad(c.ctx, delta, codes, scales, FMT, dW, gamma=gamma, beta=beta, status=c.status,
                           ws=new(G.gift_act_workspace_bytes(c.ctx, "weight_grad", delta.dtype, T, d_out, d)))
        dy = delta @ W.to(delta.dtype)
        dx, dgamma, dbeta = torch.empty_like(dy), torch.empty_like(gamma), torch.empty_like(beta)
        G.gift_layernorm_backward(c.ctx, dy, codes, gamma, rstd, dx, dgamma, dbeta, scales=scales, fmt=FMT,
                                  status=c.status,
                                  ws=new(G.gift_act_workspace_bytes(c.ctx, "layernorm_backward", dy.dtype, T, d, d)))
        return dx, dgamma, dbeta, dW, None, None


def layer_inputs(ctx, kept, T, d_in, status):
    """What the linear layer read, a = gamma n + beta in BF16, from the checkpoint of the norm's rows n."""
    n = torch.empty(T, d_in, device=kept["gain"].device)
    G.gift_act_decode(ctx, *kept["checkpoint"], FMT, n, status=status)
    return torch.addcmul(kept["offset"], n, kept["gain"]).to(torch.bfloat16)


def average_through_codec(ctx, grads, kept, T):
    """The replicas' weight gradients whitened with the factor of the activations that `kept` stands for (one
    factor for all of them: a single decode maps the average back), packed to E4M3, averaged and mapped
    back."""
    d_out, d_in = grads[0].shape
    dev = grads[0].device
    new = lambda n: torch.empty(max(n, 256), dtype=torch.uint8, device=dev)  # noqa: E731
    status = kept["status"]
    acts = layer_inputs(ctx, kept, T, d_in, status)
    fac = G.Factor.empty("lowrank", d_out, d_in, planes=True)
    G.gift_factor_update(ctx, fac, acts, seed=1, status=status,
                         ws=new(G.gift_workspace_bytes(ctx, "factor_update", "lowrank", "e4m3", "tensor", d_out, d_in, T)))
    codes = [torch.empty(d_out, d_in, dtype=torch.uint8, device=dev) for _ in grads]
    scales = [torch.empty(1, device=dev) for _ in grads]
    G.gift_encode_replicas(ctx, fac, grads, "e4m3", "tensor", codes, scales, status=status,
                           ws=new(G.gift_workspace_bytes(ctx, "encode", "lowrank", "e4m3", "tensor", d_out, d_in)))
    out = torch.empty(d_out, d_in, device=dev)
    G.gift_reduce_decode(ctx, fac, codes, scales, "e4m3", "tensor", d_out, d_in, out, status=status,
                         ws=new(G.gift_workspace_bytes(ctx, "reduce_decode", "lowrank", "e4m3", "tensor", d_out, d_in)))
    return out


def train(tokens=4096, d_in=1536, d_out=384, steps=10, replicas=2, lr=0.1, seed=0):
    """Runs the steps; returns the losses, the codec's relative error, and the bytes kept per replica."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    r = lambda *s: torch.randn(*s, device=dev, generator=gen)  # noqa: E731
    ctx = G.Context(torch.cuda.current_device())
    W = (0.02 * r(d_out, d_in)).requires_grad_()
    gamma, beta = torch.ones(d_in, device=dev, requires_grad=True), torch.zeros(d_in, device=dev, requires_grad=True)
    goal = 0.02 * r(d_out, d_in)
    chan = torch.exp(0.2 * r(d_in))
    xs = [(r(tokens, d_in) * chan).to(torch.bfloat16) for _ in range(replicas)]
    with torch.no_grad():   # the goal sees normalised rows
        norm = lambda x: (x.float() - x.float().mean(1, keepdim=True)) / x.float().std(1, keepdim=True)  # noqa: E731
        ys = [norm(x) @ goal.t() for x in xs]
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    losses, error, kept = [], 0.0, [{"status": status} for _ in range(replicas)]
    for _ in range(steps):
        gW, total = [], 0.0
        for x, y, k in zip(xs, ys, kept):
            W.grad = None
            out = NormLinear.apply(x, gamma, beta, W, ctx, k)
            loss = (out.float() - y).square().mean()
            loss.backward()
            gW.append(W.grad)
            total += loss.item() / replicas
        avg = average_through_codec(ctx, gW, kept[0], tokens)
        if int(status.item()):   # of the passes as well as the codec
            raise G.GiftError(int(status.item()), "a training step")
        exact = sum(gW) / replicas
        error = ((avg - exact).norm() / exact.norm()).item()
        with torch.no_grad():
            for p, g in ((W, avg), (gamma, gamma.grad / replicas), (beta, beta.grad / replicas)):
                p -= lr * g * (d_out if p is W else 1.0)
        gamma.grad = beta.grad = None
        losses.append(total)
    return losses, error, kept[0]["bytes"]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("tokens", 4096), ("d-in", 1536), ("d-out", 384), ("steps", 10), ("replicas", 2)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    losses, error, kept = train(a.tokens, a.d_in, a.d_out, a.steps, a.replicas)
    print("loss", " ".join("%.4f" % v for v in losses))
    print("averaged gradient after the codec: relative error %.3g" % error)
    print("kept between the passes: %d bytes per replica, %.2f of the BF16 input's" % (
        kept, kept / (2.0 * a.tokens * a.d_in)))


if __name__ == "__main__":
    main()
