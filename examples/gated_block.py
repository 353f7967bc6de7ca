"""Training steps of a gated feed-forward block whose kept activations wait in 8 bits, with GIFT behind it.

y = x + drop(W (silu(Wg n) * (Wu n)) + b), n = norm(x), for R data-parallel replicas modelled on one GPU:

  forward    gift_layernorm_forward and gift_gated_forward keep n and h = silu(g) u as 8-bit checkpoints, the latter g and u
             besides; gift_linear_forward ends with dropout and the residual stream;
  backward   gift_dropout_backward draws the same bits again, gift_weight_grad takes the three weight gradients from
             the checkpoints, gift_gated_backward and gift_input_grad carry the gradient to the norm;
  codec      the second product's gradient (the method's fragile layer) goes through GIFT: K-FAC factor from replica
             0's h, whitened, packed to E4M3, averaged and mapped back (Algorithm 1).

    python examples/gated_block.py [--tokens 2048] [--d 512] [--f 1536] [--steps 5]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from fac_whitening_gb300 import gift as G  # noqa: E402

FMT, EPS, FN = "e4m3", 1e-5, "silu"


def bytes_of(n):
    return torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")


class GatedBlock(torch.autograd.Function):
    """The block in BF16 with FP32 weights' gradients.  `site` tells this dropout from the model's others; rng holds the
    seed and the step on the device; kept["h"] gets h's checkpoint, kept["status"] what only the device sees."""

    @staticmethod
    def forward(c, x, gamma, beta, Wg, Wu, W, b, ctx, p, rng, site, kept):
        T, d = x.shape
        f, dev, bf16, st = Wg.shape[0], x.device, torch.bfloat16, kept["status"]
        Wg, Wu, W = Wg.to(bf16), Wu.to(bf16), W.to(bf16)
        new = lambda n: torch.empty(T, n, dtype=bf16, device=dev)  # noqa: E731
        keep = lambda n: tuple(torch.empty(k, dtype=torch.uint8, device=dev) for k in G.gift_act_sizes(FMT, T, n))  # noqa: E731,E501
        ws = lambda op, o, i: bytes_of(G.gift_act_workspace_bytes(ctx, op, bf16, T, o, i))  # noqa: E731
        n, h, gate, up, y, rstd = new(d), new(f), new(f), new(f), new(d), torch.empty(T, device=dev)
        n_kept, h_kept = keep(d), keep(f)
        G.gift_layernorm_forward(ctx, x, gamma, beta, EPS, n, rstd=rstd, fmt=FMT, codes=n_kept[0], scales=n_kept[1],
                                 status=st)
        G.gift_gated_forward(ctx, n, Wg, Wu, FN, h, gate=gate, up=up, fmt=FMT, codes=h_kept[0], scales=h_kept[1],
                             ws=ws("gated_forward", f, d), status=st)
        G.gift_linear_forward(ctx, h, W, y, bias=b, residual=x, p=p, rng=rng, site=site,
                              ws=ws("linear_forward", d, f), status=st)
        c.save_for_backward(*n_kept, *h_kept, rstd, gate, up, gamma, beta, Wg, Wu, W, rng)
        c.ctx, c.p, c.site, c.status, c.ws = ctx, p, site, st, ws
        kept["h"] = h_kept
        return y

    @staticmethod
    def backward(c, dy):
        nc, ns, hc, hs, rstd, gate, up, gamma, beta, Wg, Wu, W, rng = c.saved_tensors
        dy = dy.contiguous()
        (T, d), f, ctx, ws = dy.shape, Wg.shape[0], c.ctx, c.ws
        k = dict(status=c.status)
        f32 = lambda *s: torch.empty(*s, device=dy.device)  # noqa: E731
        dz, dn, dx, dg, du = (torch.empty_like(t) for t in (dy, dy, dy, gate, up))
        dW, dWg, dWu, db, dgamma, dbeta = f32(d, f), f32(f, d), f32(f, d), f32(d), f32(d), f32(d)
        G.gift_dropout_backward(ctx, dy, dz, c.p, rng, c.site, db, ws=ws("dropout_backward", d, d))
        G.gift_weight_grad(ctx, dz, hc, hs, FMT, dW, ws=ws("weight_grad", d, f), **k)
        G.gift_gated_backward(ctx, dz, W, gate, up, FN, dg, du, ws=ws("gated_backward", d, f), **k)
        for delta, out in ((dg, dWg), (du, dWu)):
            G.gift_weight_grad(ctx, delta, nc, ns, FMT, out, gamma=gamma, beta=beta, ws=ws("weight_grad", f, d), **k)
        G.gift_input_grad(ctx, dg, Wg, dn, delta2=du, W2=Wu, ws=ws("input_grad", f, d), **k)
        G.gift_layernorm_backward(ctx, dn, nc, gamma, rstd, dx, dgamma, dbeta, scales=ns, fmt=FMT,
                                  ws=ws("layernorm_backward", d, d), **k)
        return dx + dy, dgamma, dbeta, dWg, dWu, dW, db, None, None, None, None, None


def average_through_codec(ctx, grads, h_kept, T, status):
    """The replicas' gradients of the second product, whitened with the factor of replica 0's h (from its checkpoint),
    packed to E4M3, averaged and mapped back."""
    d, f = grads[0].shape
    dev = grads[0].device
    h = torch.empty(T, f, dtype=torch.bfloat16, device=dev)
    G.gift_act_decode(ctx, *h_kept, FMT, h, status=status)
    fac = G.Factor.empty("lowrank", d, f, planes=True)
    need = lambda op, *a: bytes_of(G.gift_workspace_bytes(ctx, op, "lowrank", FMT, "tensor", d, f, *a))  # noqa: E731
    G.gift_factor_update(ctx, fac, h, seed=1, status=status, ws=need("factor_update", T))
    codes = [torch.empty(d, f, dtype=torch.uint8, device=dev) for _ in grads]
    scales = [torch.empty(1, device=dev) for _ in grads]
    G.gift_encode_replicas(ctx, fac, grads, FMT, "tensor", codes, scales, status=status, ws=need("encode"))
    out = torch.empty(d, f, device=dev)
    G.gift_reduce_decode(ctx, fac, codes, scales, FMT, "tensor", d, f, out, status=status, ws=need("reduce_decode"))
    return out


def parameters(d, f, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    params = [torch.ones(d, device="cuda"), torch.zeros(d, device="cuda"), r(f, d) / d ** 0.5, r(f, d) / d ** 0.5,
              r(d, f) / f ** 0.5, torch.zeros(d, device="cuda")]
    return [p.requires_grad_() for p in params], r


def train(tokens=2048, d=512, f=1536, steps=5, replicas=2, p=0.1, lr=0.05, seed=0):
    """Runs the steps; returns the losses and the codec's relative error."""
    ctx = G.Context(torch.cuda.current_device())
    params, r = parameters(d, f, seed)
    xs = [r(tokens, d).to(torch.bfloat16) for _ in range(replicas)]
    goals = [torch.tanh(x.float() @ r(d, d) / d ** 0.5) for x in xs]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    rngs = [torch.tensor([seed + 1 + i, 0], dtype=torch.int64, device="cuda") for i in range(replicas)]
    losses, error = [], 0.0
    for _ in range(steps):
        sums, gW, total, kept = [0.0] * len(params), [], 0.0, [{"status": status} for _ in xs]
        for x, goal, rng, k in zip(xs, goals, rngs, kept):
            y = GatedBlock.apply(x, *params, ctx, p, rng, 0, k)
            loss = (y.float() - goal).square().mean()
            grads = torch.autograd.grad(loss, params)
            gW.append(grads[4])
            sums = [s + g / replicas for s, g in zip(sums, grads)]
            total += loss.item() / replicas
            rng[1] += 1   # the next step's bits
        avg = average_through_codec(ctx, gW, kept[0]["h"], tokens, status)
        if int(status.item()):
            raise G.GiftError(int(status.item()), "a training step")
        error = ((avg - sums[4]).norm() / sums[4].norm()).item()
        sums[4] = avg
        with torch.no_grad():
            for q, g in zip(params, sums):
                q -= lr * d * g
        losses.append(total)
    return losses, error


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("tokens", 2048), ("d", 512), ("f", 1536), ("steps", 5), ("replicas", 2)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    losses, error = train(a.tokens, a.d, a.f, a.steps, a.replicas)
    print("loss", " ".join("%.4f" % v for v in losses))
    print("averaged gradient of the second product after the codec: relative error %.3g" % error)


if __name__ == "__main__":
    main()
