"""Cases of the activation-checkpoint operators: layer norm forward and backward, the 8-bit
activation checkpoint (encode and decode), and the weight gradient taken from a checkpoint.

Every operator has a plain form here (elementary torch operations in FP32, one rounding at the
end) and is reached through fac_whitening_gb300.gift when `own` is set.

An 8-bit checkpoint of x (T tokens x d) is one E4M3 or E5M2 code per element and one
power-of-two scale 2^k per token and 128 consecutive columns, kept as the byte k + 127; k is the
smallest exponent with amax <= FMAX 2^k, held within [-110, 127 - EMAX].  Its values are exact in
BF16.
"""
import math

import torch

own = False

GROUP = 128
EPS = 1e-5
FORMATS = {   # largest value's exponent, its mantissa bits, torch's type
    "e4m3": (8, 3, torch.float8_e4m3fn),
    "e5m2": (15, 2, torch.float8_e5m2),
}
K_MIN = -110
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---- cases --------------------------------------------------------------------------------
def listed():
    return [
        # a small layer's step: latency is all there is (the tiny workload's 512 tokens x 256)
        {"name": "norm_forward_tiny", "op": "norm_forward", "T": 512, "d": 256, "dt": "f32", "fmt": "none"},
        # the 600M-like model's norm before a linear layer, keeping the 8-bit checkpoint of its output's
        # normalised rows, and reading the checkpoint back as a backward pass does
        {"name": "norm_forward_saved_600m", "op": "norm_forward", "T": 16384, "d": 1536, "dt": "bf16", "fmt": "e4m3"},
        # a small layer's backward pass from the kept input
        {"name": "norm_backward_tiny", "op": "norm_backward", "T": 512, "d": 256, "dt": "f32", "fmt": "none"},
        # the stress layers' width over a long batch, from the kept BF16 input
        {"name": "norm_backward_wide", "op": "norm_backward", "T": 32768, "d": 4096, "dt": "bf16", "fmt": "none"},
        # the 600M-like norm's backward pass from the 8-bit checkpoint
        {"name": "norm_backward_saved_600m", "op": "norm_backward", "T": 16384, "d": 1536, "dt": "bf16", "fmt": "e4m3"},
        # a ragged batch of an odd width, E5M2 checkpoint, FP32 gradients
        {"name": "norm_backward_saved_odd", "op": "norm_backward", "T": 5003, "d": 1361, "dt": "f32", "fmt": "e5m2"},
        # a small layer's checkpoint, written and read back
        {"name": "checkpoint_tiny", "op": "checkpoint", "T": 512, "d": 256, "dt": "f32", "fmt": "e4m3"},
        # the input of the 600M-like model's second MLP product, written and read back
        {"name": "checkpoint_600m", "op": "checkpoint", "T": 16384, "d": 6144, "dt": "bf16", "fmt": "e4m3"},
        # a small layer's weight gradient from FP32 output gradients
        {"name": "weight_grad_tiny", "op": "weight_grad", "T": 512, "d": 256, "d_out": 64, "dt": "f32", "fmt": "e4m3",
         "affine": False},
        # the 600M-like second MLP product (1536 x 6144 over 16384 tokens): the gradient the codec encodes
        {"name": "weight_grad_600m", "op": "weight_grad", "T": 16384, "d": 6144, "d_out": 1536, "dt": "bf16",
         "fmt": "e4m3", "affine": False},
        # a ragged batch with odd layer sizes behind a norm (its gain and offset folded in), E5M2
        {"name": "weight_grad_affine_odd", "op": "weight_grad", "T": 5003, "d": 2731, "d_out": 1021, "dt": "bf16",
         "fmt": "e5m2", "affine": True},
        # the stress layer: 4096 x 16384 over 32768 tokens
        {"name": "weight_grad_stress", "op": "weight_grad", "T": 32768, "d": 16384, "d_out": 4096, "dt": "bf16",
         "fmt": "e4m3", "affine": False},
    ]


def _log(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.4 and n >= 64:   # layer sizes are mostly multiples of 64, batches mostly are not
        n -= n % 64
    return max(lo, min(hi, n))


def draw(rng):
    op = rng.choice(["norm_forward", "norm_backward", "checkpoint", "weight_grad"])
    dt = rng.choice(["f32", "bf16", "bf16"])
    fmt = rng.choice(["e4m3", "e4m3", "e5m2"])
    T, d = _log(rng, 1, 32768), _log(rng, 8, 16384)
    if op == "weight_grad":
        return {"op": op, "T": T, "d": d, "d_out": _log(rng, 8, 4096), "dt": dt, "fmt": fmt,
                "affine": rng.random() < 0.5}
    T = max(1, min(T, (1 << 27) // d))
    if op != "checkpoint" and rng.random() < 0.5:
        fmt = "none"
    return {"op": op, "T": T, "d": d, "dt": dt, "fmt": fmt}


# ---- the checkpoint's plain form -------------------------------------------------------------
def _pow2(k):
    """2^k as FP32 for integer k in [-126, 127], from its bit pattern."""
    return ((k + 127) << 23).to(torch.int32).view(torch.float32)


def _encode(x, fmt):
    """Codes (float8, T x d) and scale exponents (int32, T x groups) of x in FP32."""
    emax, _, f8 = FORMATS[fmt]
    T, d = x.shape
    g = torch.nn.functional.pad(x, (0, -d % GROUP)).view(T, -1, GROUP)
    m, e = torch.frexp(g.abs().amax(-1))   # amax = m 2^e, m in [1/2, 1); FMAX = 0.875 2^(emax + 1)
    k = torch.where(m > 0.875, e - emax, e - emax - 1).to(torch.int32).clamp(K_MIN, 127 - emax)
    top = 1.75 * 2.0 ** emax
    q = (g * _pow2(-k)[..., None]).clamp(-top, top).to(f8).view(T, -1)[:, :d]
    return q.contiguous(), k


def _decode(q, k):
    """The values of codes q (float8) with scale exponents k, in FP32 (exact)."""
    T, d = q.shape
    s = _pow2(k)[..., None].expand(-1, -1, GROUP).reshape(T, -1)[:, :d]
    return q.float() * s


# ---- inputs ----------------------------------------------------------------------------------
def _residual(T, d, gen, dev):
    """Residual-stream rows: channels of unequal size and offset, a few large ones, tokens of unequal norm."""
    r = lambda *s: torch.randn(*s, device=dev, generator=gen)  # noqa: E731
    chan = torch.exp(0.5 * r(d))
    chan[torch.randint(d, (max(1, d // 256),), device=dev, generator=gen)] *= 20.0
    x = r(T, d)
    x.mul_(chan).add_(0.3 * r(d)).mul_(torch.exp(0.4 * r(T, 1)))
    return x


def _activations(T, d, gen, dev):
    """Inputs of the second MLP product: GELU of rows whose channels fall off as a power law."""
    r = lambda *s: torch.randn(*s, device=dev, generator=gen)  # noqa: E731
    size = torch.arange(1, d + 1, device=dev, dtype=torch.float32).pow(-0.3)[torch.randperm(d, device=dev, generator=gen)]
    u = r(T, d)
    u.mul_(2.0 * size).add_(0.1 * r(d))
    return u.mul_(torch.special.ndtr(u))


def _gradients(T, d, gen, dev):
    """Output gradients: small, with tokens that weigh more than others."""
    g = torch.randn(T, d, device=dev, generator=gen)
    return g.mul_(1e-3 * torch.exp(0.7 * torch.randn(T, 1, device=dev, generator=gen)))


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    T, d, dt, fmt, op = case["T"], case["d"], TYPES[case["dt"]], case["fmt"], case["op"]
    s = {"op": op, "fmt": fmt, "dt": dt}
    if op.startswith("norm"):
        x = _residual(T, d, gen, dev).to(dt)
        s["gamma"] = 1.0 + 0.2 * torch.randn(d, device=dev, generator=gen)
        s["beta"] = 0.1 * torch.randn(d, device=dev, generator=gen)
        if op == "norm_forward":
            s["x"] = x
        else:
            s["dy"] = _gradients(T, d, gen, dev).to(dt)
            xf = x.float()
            var, mean = torch.var_mean(xf, dim=1, correction=0)
            rstd = torch.rsqrt(var + EPS)
            s["rstd"] = rstd
            if fmt == "none":
                s["x"], s["mean"] = x, mean
            else:
                q, k = _encode((xf - mean[:, None]) * rstd[:, None], fmt)
                s["codes"], s["scales"] = q.view(torch.uint8), (k + 127).to(torch.uint8)
    elif op == "checkpoint":
        s["x"] = _activations(T, d, gen, dev).to(dt)
    else:
        q, k = _encode(_activations(T, d, gen, dev).to(torch.bfloat16).float(), fmt)
        s["codes"], s["scales"] = q.view(torch.uint8), (k + 127).to(torch.uint8)
        s["delta"] = _gradients(T, case["d_out"], gen, dev).to(dt)
        s["gamma"] = s["beta"] = None
        if case["affine"]:
            s["gamma"] = 1.0 + 0.2 * torch.randn(d, device=dev, generator=gen)
            s["beta"] = 0.1 * torch.randn(d, device=dev, generator=gen)
    if own:
        _keep(case, s)
    return s


def _keep(case, s):
    """What a training program holds for the calls: the context, a workspace, its output buffers."""
    from fac_whitening_gb300 import gift as G
    dev = torch.device("cuda")
    T, d, dt, fmt, op = case["T"], case["d"], s["dt"], case["fmt"], case["op"]
    s["ctx"] = ctx = G.Context(torch.cuda.current_device())
    s["status"] = torch.zeros(1, dtype=torch.int32, device=dev)
    f32 = lambda *n: torch.empty(*n, dtype=torch.float32, device=dev)  # noqa: E731
    if fmt != "none" and "codes" not in s:
        cb, sb = G.gift_act_sizes(fmt, T, d)
        s["out_codes"] = torch.empty(cb, dtype=torch.uint8, device=dev)
        s["out_scales"] = torch.empty(sb, dtype=torch.uint8, device=dev)
        s["values"] = torch.empty(T, d, dtype=torch.bfloat16 if op == "norm_forward" else dt, device=dev)
    need = 0
    if op == "norm_forward":
        s["y"], s["mean"], s["rstd"] = torch.empty(T, d, dtype=dt, device=dev), f32(T), f32(T)
    elif op == "norm_backward":
        s["dx"], s["dgamma"], s["dbeta"] = torch.empty(T, d, dtype=dt, device=dev), f32(d), f32(d)
        need = G.gift_act_workspace_bytes(ctx, "layernorm_backward", dt, T, d, d)
    elif op == "weight_grad":
        s["dW"], s["db"] = f32(case["d_out"], d), f32(case["d_out"])
        need = G.gift_act_workspace_bytes(ctx, "weight_grad", dt, T, case["d_out"], d)
    s["ws"] = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)


# ---- one pass ----------------------------------------------------------------------------------
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from fac_whitening_gb300 import gift as G
    op, ctx, st, fmt = s["op"], s["ctx"], s["status"], s["fmt"]
    if op == "norm_forward":
        if fmt == "none":
            G.gift_layernorm_forward(ctx, s["x"], s["gamma"], s["beta"], EPS, s["y"], mean=s["mean"], rstd=s["rstd"],
                                     status=st)
            return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
        G.gift_layernorm_forward(ctx, s["x"], s["gamma"], s["beta"], EPS, s["y"], rstd=s["rstd"], fmt=fmt,
                                 codes=s["out_codes"], scales=s["out_scales"], status=st)
        G.gift_act_decode(ctx, s["out_codes"], s["out_scales"], fmt, s["values"], status=st)
        return {"y": s["y"], "rstd": s["rstd"], "saved": s["values"]}
    if op == "norm_backward":
        if fmt == "none":
            G.gift_layernorm_backward(ctx, s["dy"], s["x"], s["gamma"], s["rstd"], s["dx"], s["dgamma"], s["dbeta"],
                                      mean=s["mean"], ws=s["ws"], status=st)
        else:
            G.gift_layernorm_backward(ctx, s["dy"], s["codes"], s["gamma"], s["rstd"], s["dx"], s["dgamma"],
                                      s["dbeta"], fmt=fmt, scales=s["scales"], ws=s["ws"], status=st)
        return {"dx": s["dx"], "dgamma": s["dgamma"], "dbeta": s["dbeta"]}
    if op == "checkpoint":
        G.gift_act_encode(ctx, s["x"], fmt, s["out_codes"], s["out_scales"], status=st)
        G.gift_act_decode(ctx, s["out_codes"], s["out_scales"], fmt, s["values"], status=st)
        return {"values": s["values"]}
    G.gift_weight_grad(ctx, s["delta"], s["codes"], s["scales"], fmt, s["dW"], db=s["db"], gamma=s["gamma"],
                       beta=s["beta"], ws=s["ws"], status=st)
    return {"dW": s["dW"], "db": s["db"]}


def _saved(s):
    """The checkpoint a backward pass starts from, as FP32 values."""
    return _decode(s["codes"].view(FORMATS[s["fmt"]][2]), s["scales"].to(torch.int32) - 127)


def _run_plain(s):
    op, dt = s["op"], s["dt"]
    if op == "norm_forward":
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        c = x - mean
        rstd = torch.rsqrt((c * c).mean(1, keepdim=True) + EPS)
        n = c * rstd
        y = (n * s["gamma"] + s["beta"]).to(dt)
        if s["fmt"] == "none":
            return {"y": y, "mean": mean[:, 0], "rstd": rstd[:, 0]}
        return {"y": y, "rstd": rstd[:, 0], "saved": _decode(*_encode(n, s["fmt"])).to(torch.bfloat16)}
    if op == "norm_backward":
        dy = s["dy"].float()
        rstd = s["rstd"][:, None]
        n = (s["x"].float() - s["mean"][:, None]) * rstd if s["fmt"] == "none" else _saved(s)
        g = dy * s["gamma"]
        dx = rstd * (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True))
        return {"dx": dx.to(dt), "dgamma": (dy * n).sum(0), "dbeta": dy.sum(0)}
    if op == "checkpoint":
        return {"values": _decode(*_encode(s["x"].float(), s["fmt"])).to(dt)}
    delta = s["delta"].float()
    dW = delta.t() @ _saved(s)
    db = delta.sum(0)
    if s["gamma"] is not None:
        dW = dW * s["gamma"] + db[:, None] * s["beta"]
    return {"dW": dW, "db": db}


# ---- from the definition, in 64 bits -------------------------------------------------------------
def _round64(v, fmt):
    """v (float64) rounded to the checkpoint's values: nearest, ties to even, per group of 128 columns."""
    emax, bits, _ = FORMATS[fmt]
    out = torch.empty_like(v)
    for c in range(0, v.shape[1], GROUP):
        g = v[:, c:c + GROUP]
        top = g.abs().amax(1, keepdim=True)
        k = torch.ceil(torch.log2(torch.clamp(top, min=1e-300) / (1.75 * 2.0 ** emax)) - 1e-12).clamp(K_MIN, 127 - emax)
        two_k = torch.exp2(k)
        u = g / two_k
        lowest = 2 - 2 ** (3 if fmt == "e4m3" else 4)   # exponent of the smallest normal code
        e = torch.floor(torch.log2(torch.clamp(u.abs(), min=1e-300))).clamp(min=lowest)
        step = torch.exp2(e - bits)
        r = torch.round(u / step) * step
        out[:, c:c + GROUP] = r.clamp(-1.75 * 2.0 ** emax, 1.75 * 2.0 ** emax) * two_k
    return out


def _value64(codes, scales, fmt):
    """Codes (bytes) and scale bytes as float64 values, from the formats' bit fields."""
    bits = FORMATS[fmt][1]
    bias = 7 if fmt == "e4m3" else 15
    i = torch.arange(256, device=codes.device)
    e, m = (i & 127) >> bits, (i & ((1 << bits) - 1)).double() / (1 << bits)
    table = torch.where(e == 0, m * 2.0 ** (1 - bias), (1 + m) * torch.exp2((e - bias).double()))
    table = torch.where(i >= 128, -table, table)
    s = torch.exp2(scales.double() - 127).repeat_interleave(GROUP, dim=1)[:, :codes.shape[1]]
    return table[codes.long()] * s


@torch.no_grad()
def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    op, fmt = s["op"], s["fmt"]
    if op == "norm_forward":
        x = s["x"].double()
        mean = x.sum(1) / x.shape[1]
        dev = x - mean[:, None]
        rstd = 1.0 / torch.sqrt(dev.square().sum(1) / x.shape[1] + EPS)
        n = dev * rstd[:, None]
        y = n * s["gamma"].double() + s["beta"].double()
        if fmt == "none":
            return {"y": y, "mean": mean, "rstd": rstd}
        return {"y": y, "rstd": rstd, "saved": _round64(n, fmt)}
    if op == "norm_backward":
        dy, rstd, d = s["dy"].double(), s["rstd"].double()[:, None], case["d"]
        if fmt == "none":
            n = (s["x"].double() - s["mean"].double()[:, None]) * rstd
        else:
            n = _value64(s["codes"], s["scales"], fmt)
        h = dy * s["gamma"].double()
        a, b = h.sum(1, keepdim=True) / d, (h * n).sum(1, keepdim=True) / d
        return {"dx": rstd * (h - a - n * b), "dgamma": (dy * n).sum(0), "dbeta": dy.sum(0)}
    if op == "checkpoint":
        return {"values": _round64(s["x"].double(), fmt)}
    dW = torch.zeros(case["d_out"], case["d"], dtype=torch.float64, device="cuda")
    db = torch.zeros(case["d_out"], dtype=torch.float64, device="cuda")
    for t in range(0, case["T"], 4096):
        r = slice(t, t + 4096)
        dl = s["delta"][r].double()
        dW += torch.einsum("to,ti->oi", dl, _value64(s["codes"][r], s["scales"][r], fmt))
        db += dl.sum(0)
    if s["gamma"] is not None:
        dW = dW * s["gamma"].double() + torch.outer(db, s["beta"].double())
    return {"dW": dW, "db": db}


# ---- what a pass cannot do without ------------------------------------------------------------------
def work(case):
    T, d, op = case["T"], case["d"], case["op"]
    e = 4 if case["dt"] == "f32" else 2
    code = T * d + T * -(-d // GROUP)   # codes and scale bytes of a checkpoint
    if op == "norm_forward":
        if case["fmt"] == "none":
            return {"bytes": 2 * T * d * e + 8 * T + 8 * d, "flops": 8 * T * d}
        # forward (x in; y, rstd and the checkpoint out), then the checkpoint in and its BF16 values out
        return {"bytes": 2 * T * d * e + 4 * T + 8 * d + 2 * code + 2 * T * d, "flops": 11 * T * d}
    if op == "norm_backward":
        kept = T * d * e + 8 * T if case["fmt"] == "none" else code + 4 * T
        return {"bytes": 2 * T * d * e + kept + 12 * d, "flops": 14 * T * d}
    if op == "checkpoint":
        return {"bytes": 2 * T * d * e + 2 * code, "flops": 4 * T * d}
    o = case["d_out"]
    return {"bytes": T * o * e + code + 4 * o * d + 4 * o + (8 * d if case["affine"] else 0), "flops": 2 * T * o * d}
