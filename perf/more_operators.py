"""Cases of the feed-forward operators: the gated block's forward and backward pass, the linear layer with
dropout and residual behind it, the input gradient, and dropout by itself.

Every operator has a plain form here (elementary torch operations in FP32, one rounding at the
end) and is reached through fac_whitening_gb300.gift when `own` is set.

  gated_forward   g = x Wg^T + bg, u = x Wu^T + bu, h = a(g) u; g and u are kept for the backward pass, h also as an
                  8-bit checkpoint for the weight gradient of the layer that reads it
  gated_backward  dh = dy W, dg = dh u a'(g), du = dh a(g)
  input_grad      dx = delta W, or delta W + delta2 W2 for the block's two projections
  linear          y = residual + drop(x W^T + bias)
  dropout         forward y = residual + drop(x + bias), then backward dx = drop(dy), dbias = sum_t dx

drop() is decided by a counter-based generator: Philox4x32-10 with the 64-bit seed as key and the counter
(column / 8, row, site, step) gives 128 bits for eight columns of a row, 16 for each (the lower half of a word first).
A value is dropped where its 16 bits are below P = round(65536 p) and otherwise scaled by 65536 / (65536 - P).

The 8-bit checkpoint has one E4M3 or E5M2 code per element and one power-of-two scale 2^k per token and 128
consecutive columns; k is the smallest exponent with amax <= FMAX 2^k, held within [-110, 127 - EMAX].
"""
import math

import torch

own = False

GROUP = 128
FORMATS = {   # largest value's exponent, its mantissa bits, torch's type
    "e4m3": (8, 3, torch.float8_e4m3fn),
    "e5m2": (15, 2, torch.float8_e5m2),
}
K_MIN = -110
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
MOST = 1 << 41   # tokens x width x hidden width of the largest case


# ---- cases --------------------------------------------------------------------------------
def listed():
    return [
        # a small block's step: latency counts (the tiny workload's 512 tokens x 256, four times as wide inside)
        {"name": "gated_forward_tiny", "op": "gated_forward", "T": 512, "d": 256, "f": 1024, "dt": "f32",
         "fn": "silu", "bias": True, "fmt": "e4m3"},
        # the 600M-like model's block over its 16384 tokens
        {"name": "gated_forward_600m", "op": "gated_forward", "T": 16384, "d": 1536, "f": 6144, "dt": "bf16",
         "fn": "silu", "bias": False, "fmt": "e4m3"},
        # the stress layers' block (4096 x 16384) over 32768 tokens
        {"name": "gated_forward_stress", "op": "gated_forward", "T": 32768, "d": 4096, "f": 16384, "dt": "bf16",
         "fn": "silu", "bias": False, "fmt": "e4m3"},
        # a small block's backward pass
        {"name": "gated_backward_tiny", "op": "gated_backward", "T": 512, "d": 256, "f": 1024, "dt": "f32",
         "fn": "silu"},
        # the 600M-like block's backward pass through its second product
        {"name": "gated_backward_600m", "op": "gated_backward", "T": 16384, "d": 1536, "f": 6144, "dt": "bf16",
         "fn": "silu"},
        # a ragged batch with odd layer sizes, GELU's tanh form
        {"name": "gated_backward_odd", "op": "gated_backward", "T": 5003, "d": 1361, "f": 2731, "dt": "bf16",
         "fn": "gelu_tanh"},
        # the gradient that the 600M-like block hands to the norm in front of it, from both projections
        {"name": "input_grad_600m", "op": "input_grad", "T": 16384, "d": 1536, "f": 6144, "dt": "bf16", "two": True},
        # one layer's input gradient, a ragged FP32 batch with odd sizes
        {"name": "input_grad_odd", "op": "input_grad", "T": 1003, "d": 1361, "f": 1021, "dt": "f32", "two": False},
        # the 600M-like block's second product on the last few tokens of a batch: the weights are all there is
        {"name": "linear_few_tokens", "op": "linear", "T": 24, "d": 1536, "f": 6144, "dt": "bf16", "p": 0.1},
        # the 600M-like block's second product, with dropout and the residual stream
        {"name": "linear_600m", "op": "linear", "T": 16384, "d": 1536, "f": 6144, "dt": "bf16", "p": 0.1},
        # dropout of the 600M-like residual stream, both directions
        {"name": "dropout_600m", "op": "dropout", "T": 16384, "d": 1536, "dt": "bf16", "p": 0.1},
        # a ragged FP32 batch of an odd width
        {"name": "dropout_odd", "op": "dropout", "T": 5003, "d": 1361, "dt": "f32", "p": 0.25},
    ]


def _log(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.4 and n >= 64:   # layer sizes are mostly multiples of 64, batches mostly are not
        n -= n % 64
    return max(lo, min(hi, n))


def draw(rng):
    op = rng.choice(["gated_forward", "gated_backward", "input_grad", "linear", "dropout"])
    dt = rng.choice(["f32", "bf16", "bf16"])
    T, d, f = _log(rng, 1, 32768), _log(rng, 8, 4096), _log(rng, 8, 16384)
    case = {"op": op, "T": T, "d": d, "dt": dt}
    if op == "dropout":
        return case | {"p": rng.choice([0.0, 0.1, 0.25, 0.5])}
    if dt == "f32":   # FP32 products are checked on small layers and few tokens
        case["T"] = max(1, min(T, (MOST >> 6) // (d * f)))
    case["f"] = f
    if op.startswith("gated"):
        case["fn"] = rng.choice(["silu", "silu", "gelu", "gelu_tanh"])
    if op == "gated_forward":
        case |= {"bias": rng.random() < 0.5, "fmt": rng.choice(["none", "e4m3", "e4m3", "e5m2"])}
    elif op == "input_grad":
        case["two"] = rng.random() < 0.5
    elif op == "linear":
        case["p"] = rng.choice([0.0, 0.1, 0.25])
    return case


# ---- the checkpoint's plain form -------------------------------------------------------------
def _pow2(k):
    """2^k as FP32 for integer k in [-126, 127], from its bit pattern."""
    return ((k + 127) << 23).to(torch.int32).view(torch.float32)


def _through_checkpoint(x, fmt):
    """The values that the 8-bit checkpoint of x (FP32) stands for."""
    emax, _, f8 = FORMATS[fmt]
    T, d = x.shape
    g = torch.nn.functional.pad(x, (0, -d % GROUP)).view(T, -1, GROUP)
    m, e = torch.frexp(g.abs().amax(-1))   # amax = m 2^e, m in [1/2, 1); FMAX = 0.875 2^(emax + 1)
    k = torch.where(m > 0.875, e - emax, e - emax - 1).to(torch.int32).clamp(K_MIN, 127 - emax)
    top = 1.75 * 2.0 ** emax
    q = (g * _pow2(-k)[..., None]).clamp(-top, top).to(f8)
    return (q.float() * _pow2(k)[..., None]).view(T, -1)[:, :d]


# ---- dropout's plain form ----------------------------------------------------------------------
def _drop_below(p):
    return int(math.floor(65536.0 * p + 0.5))


def _kept(T, d, rng, site):
    """The 16 bits of every element, from Philox4x32-10 in 64-bit integers."""
    low = 0xFFFFFFFF
    seed, step = rng[0], rng[1]
    n = -(-d // 8)
    c = [torch.arange(n, device=rng.device).expand(T, n), torch.arange(T, device=rng.device)[:, None].expand(T, n),
         torch.full((), site, device=rng.device, dtype=torch.int64), step & low]
    k0, k1 = seed & low, (seed >> 32) & low
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57   # wrap around: the 64 bits of the product
        c = [((b >> 32) & low) ^ c[1] ^ k0, b & low, ((a >> 32) & low) ^ c[3] ^ k1, a & low]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    halves = [h for w in c for h in (w & 0xFFFF, w >> 16)]
    return torch.stack(halves, -1).view(T, 8 * n)[:, :d]


def _drop(v, p, rng, site):
    """v (FP32) with dropped values 0 and the others scaled."""
    P = _drop_below(p)
    if P == 0:
        return v
    return torch.where(_kept(*v.shape, rng, site) >= P, v * (65536.0 / (65536 - P)), torch.zeros((), device=v.device))


# ---- the gate's plain form -----------------------------------------------------------------------
def _phi(g):
    return 0.5 * torch.erfc(g * -math.sqrt(0.5))


def _tanh_inner(g):
    """z and dz/dg with GELU's tanh form g / (1 + exp(-z))."""
    c = 2.0 * math.sqrt(2.0 / math.pi)
    return c * (g + 0.044715 * g * g * g), c * (1.0 + 3.0 * 0.044715 * g * g)


def _gate(g, fn):
    if fn == "gelu":
        return g * _phi(g)
    return g / (1.0 + torch.exp(-(g if fn == "silu" else _tanh_inner(g)[0])))


def _gate_slope(g, fn):
    if fn == "gelu":
        return _phi(g) + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))
    z, dz = (g, 1.0) if fn == "silu" else _tanh_inner(g)
    s = 1.0 / (1.0 + torch.exp(-z))
    return s + g * dz * s * (1.0 / (1.0 + torch.exp(z)))


# ---- inputs ----------------------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    r = lambda *s: torch.randn(*s, device=dev, generator=gen)  # noqa: E731
    T, d, dt, op = case["T"], case["d"], TYPES[case["dt"]], case["op"]
    f = case.get("f", 0)
    s = {"op": op, "dt": dt, "fn": case.get("fn"), "p": case.get("p", 0.0), "fmt": case.get("fmt", "none")}
    # gradients: small, with tokens that weigh more than others
    gradients = lambda n: (r(T, n) * (1e-3 * torch.exp(0.7 * r(T, 1)))).to(dt)  # noqa: E731
    weights = lambda o, i: (r(o, i) / math.sqrt(i)).to(dt)  # noqa: E731
    if op == "gated_forward":   # a norm's output: channels with a gain of their own, a few large ones
        gain = 1.0 + 0.2 * r(d)
        gain[torch.randint(d, (max(1, d // 256),), device=dev, generator=gen)] *= 4.0
        s["x"] = r(T, d).mul_(gain).add_(0.1 * r(d)).to(dt)
        s["Wg"], s["Wu"] = weights(f, d), weights(f, d)
        s["bg"] = 0.1 * r(f) if case["bias"] else None
        s["bu"] = 0.1 * r(f) if case["bias"] else None
    elif op == "gated_backward":
        s["dy"], s["W"] = gradients(d), weights(d, f)
        s["gate"], s["up"] = r(T, f).mul_(1.2).add_(0.1 * r(f)).to(dt), r(T, f).to(dt)
    elif op == "input_grad":
        s["delta"], s["W"] = gradients(f), weights(f, d)
        s["delta2"], s["W2"] = (gradients(f), weights(f, d)) if case["two"] else (None, None)
    elif op == "linear":   # a gate's output: heavy at zero, channels of unequal size
        u = r(T, f).mul_(torch.exp(0.5 * r(f)))
        s["x"] = (u * torch.sigmoid(u) * r(T, f)).to(dt)
        s["W"], s["bias"], s["residual"] = weights(d, f), 0.1 * r(d), r(T, d).to(dt)
    else:
        s["x"], s["residual"], s["dy"] = r(T, d).to(dt), r(T, d).to(dt), gradients(d)
        s["bias"] = 0.1 * r(d)
    if op in ("linear", "dropout"):   # the seed and the step, where a captured step reads them
        s["rng"] = torch.randint(0, 1 << 62, (2,), device=dev, generator=gen)
        s["rng"][1] &= 0xFFFFF
        s["site"] = 7
    if own:
        _keep(case, s)
    return s


def _keep(case, s):
    """What a training program holds for the calls: the context, a workspace, its output buffers."""
    from fac_whitening_gb300 import gift as G
    dev = torch.device("cuda")
    T, d, dt, op = case["T"], case["d"], s["dt"], case["op"]
    f = case.get("f", 0)
    s["ctx"] = ctx = G.Context(torch.cuda.current_device())
    s["status"] = torch.zeros(1, dtype=torch.int32, device=dev)
    new = lambda *n: torch.empty(*n, dtype=dt, device=dev)  # noqa: E731
    if op == "gated_forward":
        s["h"], s["gate"], s["up"] = new(T, f), new(T, f), new(T, f)
        if s["fmt"] != "none":
            cb, sb = G.gift_act_sizes(s["fmt"], T, f)
            s["codes"] = torch.empty(cb, dtype=torch.uint8, device=dev)
            s["scales"] = torch.empty(sb, dtype=torch.uint8, device=dev)
            s["values"] = torch.empty(T, f, dtype=torch.bfloat16, device=dev)
        need = G.gift_act_workspace_bytes(ctx, "gated_forward", dt, T, f, d)
    elif op == "gated_backward":
        s["dgate"], s["dup"] = new(T, f), new(T, f)
        need = G.gift_act_workspace_bytes(ctx, "gated_backward", dt, T, d, f)
    elif op == "input_grad":
        s["dx"] = new(T, d)
        need = G.gift_act_workspace_bytes(ctx, "input_grad", dt, T, f, d)
    elif op == "linear":
        s["y"] = new(T, d)
        need = G.gift_act_workspace_bytes(ctx, "linear_forward", dt, T, d, f)
    else:
        s["y"], s["dx"], s["dbias"] = new(T, d), new(T, d), torch.empty(d, device=dev)
        need = G.gift_act_workspace_bytes(ctx, "dropout_backward", dt, T, d, d)
    s["ws"] = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)


# ---- one pass ----------------------------------------------------------------------------------
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from fac_whitening_gb300 import gift as G
    op, ctx, st, ws = s["op"], s["ctx"], s["status"], s["ws"]
    if op == "gated_forward":
        out = {"h": s["h"], "gate": s["gate"], "up": s["up"]}
        if s["fmt"] == "none":
            G.gift_gated_forward(ctx, s["x"], s["Wg"], s["Wu"], s["fn"], s["h"], gate=s["gate"], up=s["up"],
                                 bg=s["bg"], bu=s["bu"], ws=ws, status=st)
            return out
        G.gift_gated_forward(ctx, s["x"], s["Wg"], s["Wu"], s["fn"], s["h"], gate=s["gate"], up=s["up"], bg=s["bg"],
                             bu=s["bu"], fmt=s["fmt"], codes=s["codes"], scales=s["scales"], ws=ws, status=st)
        G.gift_act_decode(ctx, s["codes"], s["scales"], s["fmt"], s["values"], status=st)
        return out | {"saved": s["values"]}
    if op == "gated_backward":
        G.gift_gated_backward(ctx, s["dy"], s["W"], s["gate"], s["up"], s["fn"], s["dgate"], s["dup"], ws=ws,
                              status=st)
        return {"dgate": s["dgate"], "dup": s["dup"]}
    if op == "input_grad":
        G.gift_input_grad(ctx, s["delta"], s["W"], s["dx"], delta2=s["delta2"], W2=s["W2"], ws=ws, status=st)
        return {"dx": s["dx"]}
    if op == "linear":
        G.gift_linear_forward(ctx, s["x"], s["W"], s["y"], bias=s["bias"], residual=s["residual"], p=s["p"],
                              rng=s["rng"], site=s["site"], ws=ws, status=st)
        return {"y": s["y"]}
    G.gift_dropout_forward(ctx, s["x"], s["y"], s["p"], s["rng"], site=s["site"], bias=s["bias"],
                           residual=s["residual"])
    G.gift_dropout_backward(ctx, s["dy"], s["dx"], s["p"], s["rng"], site=s["site"], dbias=s["dbias"], ws=ws)
    return {"y": s["y"], "dx": s["dx"], "dbias": s["dbias"]}


def _run_plain(s):
    op, dt = s["op"], s["dt"]
    if op == "gated_forward":
        x = s["x"].float()
        g, u = x @ s["Wg"].float().t(), x @ s["Wu"].float().t()
        if s["bg"] is not None:
            g, u = g + s["bg"], u + s["bu"]
        h = _gate(g, s["fn"]) * u
        out = {"h": h.to(dt), "gate": g.to(dt), "up": u.to(dt)}
        if s["fmt"] != "none":
            out["saved"] = _through_checkpoint(h, s["fmt"]).to(torch.bfloat16)
        return out
    if op == "gated_backward":
        dh = s["dy"].float() @ s["W"].float()
        g = s["gate"].float()
        return {"dgate": (dh * s["up"].float() * _gate_slope(g, s["fn"])).to(dt),
                "dup": (dh * _gate(g, s["fn"])).to(dt)}
    if op == "input_grad":
        dx = s["delta"].float() @ s["W"].float()
        if s["delta2"] is not None:
            dx = dx + s["delta2"].float() @ s["W2"].float()
        return {"dx": dx.to(dt)}
    if op == "linear":
        v = s["x"].float() @ s["W"].float().t() + s["bias"]
        return {"y": (s["residual"].float() + _drop(v, s["p"], s["rng"], s["site"])).to(dt)}
    v = s["x"].float() + s["bias"]
    y = s["residual"].float() + _drop(v, s["p"], s["rng"], s["site"])
    dx = _drop(s["dy"].float(), s["p"], s["rng"], s["site"])
    return {"y": y.to(dt), "dx": dx.to(dt), "dbias": dx.sum(0)}


# ---- from the definition, in 64 bits -------------------------------------------------------------
def _round64(v, fmt):
    """v (float64) rounded to the checkpoint's values: nearest, ties to even, per group of 128 columns."""
    emax, bits, _ = FORMATS[fmt]
    top, lowest = 1.75 * 2.0 ** emax, 2 - 2 ** (3 if fmt == "e4m3" else 4)
    out = torch.empty_like(v)
    for c in range(0, v.shape[1], GROUP):
        g = v[:, c:c + GROUP]
        amax = g.abs().amax(1, keepdim=True)
        two_k = torch.exp2(torch.ceil(torch.log2(torch.clamp(amax, min=1e-300) / top) - 1e-12).clamp(K_MIN, 127 - emax))
        u = g / two_k
        e = torch.floor(torch.log2(torch.clamp(u.abs(), min=1e-300))).clamp(min=lowest)   # of the smallest normal code
        step = torch.exp2(e - bits)
        out[:, c:c + GROUP] = (torch.round(u / step) * step).clamp(-top, top) * two_k
    return out


def _factor64(T, d, p, rng, site):
    """0 or the scale for every element: Philox4x32-10 with its products taken by 16-bit halves."""
    P = _drop_below(p)
    dev = rng.device
    if P == 0:
        return torch.ones(T, d, dtype=torch.float64, device=dev)
    seed, step = int(rng[0]), int(rng[1])

    def wide(m, v):   # (upper, lower) 32 bits of m v
        ll, lh = (m & 0xFFFF) * (v & 0xFFFF), (m & 0xFFFF) * (v >> 16)
        hl, hh = (m >> 16) * (v & 0xFFFF), (m >> 16) * (v >> 16)
        mid = (ll >> 16) + (lh & 0xFFFF) + (hl & 0xFFFF)
        return hh + (lh >> 16) + (hl >> 16) + (mid >> 16), (ll & 0xFFFF) | ((mid & 0xFFFF) << 16)

    groups = (d + 7) // 8
    at = torch.arange(T * groups, device=dev)
    x0, x1 = at % groups, at // groups
    x2, x3 = torch.full_like(at, site), torch.full_like(at, step % 2 ** 32)
    for i in range(10):
        k0, k1 = (seed + i * 0x9E3779B9) % 2 ** 32, (seed // 2 ** 32 + i * 0xBB67AE85) % 2 ** 32
        h0, l0 = wide(0xD2511F53, x0)
        h1, l1 = wide(0xCD9E8D57, x2)
        x0, x1, x2, x3 = h1 ^ x1 ^ k0, l1, h0 ^ x3 ^ k1, l0
    bits = torch.empty(T, groups, 8, dtype=torch.int64, device=dev)
    for j, w in enumerate((x0, x1, x2, x3)):
        bits[:, :, 2 * j] = (w % 65536).view(T, groups)
        bits[:, :, 2 * j + 1] = (w // 65536).view(T, groups)
    keep = bits.view(T, 8 * groups)[:, :d] >= P
    return keep.double() * (1.0 / (1.0 - P / 65536.0))


def _a64(g, fn):
    """a(g) and a'(g) in 64 bits."""
    if fn == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * torch.sigmoid(-g))
    if fn == "gelu":
        phi = torch.special.ndtr(g)
        return g * phi, phi + g * torch.exp(-g.square() / 2) / math.sqrt(2 * math.pi)
    t = torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))
    dt = (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 0.134145 * g.square())
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * dt


@torch.no_grad()
def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    op = case["op"]
    if op == "dropout":
        m = _factor64(case["T"], case["d"], s["p"], s["rng"], s["site"])
        dx = s["dy"].double() * m
        return {"y": (s["x"].double() + s["bias"].double()) * m + s["residual"].double(), "dx": dx, "dbias": dx.sum(0)}
    if op == "gated_forward":
        T, f = case["T"], case["f"]
        wg, wu = s["Wg"].double(), s["Wu"].double()
        kinds = ["h", "gate", "up"] + (["saved"] if s["fmt"] != "none" else [])
        out = {k: torch.empty(T, f, dtype=torch.float64, device="cuda") for k in kinds}
        for t in range(0, T, 4096):
            x = s["x"][t:t + 4096].double()
            g, u = torch.einsum("td,fd->tf", x, wg), torch.einsum("td,fd->tf", x, wu)
            if s["bg"] is not None:
                g, u = g + s["bg"].double(), u + s["bu"].double()
            h = _a64(g, s["fn"])[0] * u
            for k, v in (("h", h), ("gate", g), ("up", u)):
                out[k][t:t + 4096] = v
            if "saved" in out:
                out["saved"][t:t + 4096] = _round64(h, s["fmt"])
        return out
    if op == "gated_backward":
        dh = torch.einsum("to,of->tf", s["dy"].double(), s["W"].double())
        a, slope = _a64(s["gate"].double(), s["fn"])
        return {"dgate": dh * s["up"].double() * slope, "dup": dh * a}
    if op == "input_grad":
        dx = torch.einsum("to,oi->ti", s["delta"].double(), s["W"].double())
        if s["delta2"] is not None:
            dx += torch.einsum("to,oi->ti", s["delta2"].double(), s["W2"].double())
        return {"dx": dx}
    v = torch.einsum("ti,oi->to", s["x"].double(), s["W"].double()) + s["bias"].double()
    return {"y": s["residual"].double() + v * _factor64(case["T"], case["d"], s["p"], s["rng"], s["site"])}


# ---- what a pass cannot do without ------------------------------------------------------------------
def work(case):
    T, d, op = case["T"], case["d"], case["op"]
    f = case.get("f", 0)
    e = 4 if case["dt"] == "f32" else 2
    if op == "gated_forward":
        n = T * d * e + 2 * f * d * e + 3 * T * f * e + (8 * f if case["bias"] else 0)
        if case["fmt"] != "none":   # the checkpoint out, then in, and its BF16 values out
            n += 2 * (T * f + T * -(-f // GROUP)) + 2 * T * f
        return {"bytes": n, "flops": 4 * T * d * f}
    if op == "gated_backward":
        return {"bytes": T * d * e + d * f * e + 4 * T * f * e, "flops": 2 * T * d * f}
    if op == "input_grad":
        k = 2 if case["two"] else 1
        return {"bytes": k * (T * f + f * d) * e + T * d * e, "flops": 2 * k * T * d * f}
    if op == "linear":
        return {"bytes": T * f * e + d * f * e + 2 * T * d * e + 4 * d, "flops": 2 * T * d * f}
    return {"bytes": 5 * T * d * e + 8 * d, "flops": 6 * T * d}
