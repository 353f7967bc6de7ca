"""GPU parity of the feed-forward block's calls (gated products, linear layer with dropout, input gradient, dropout)
with their 64-bit statements.

Tolerances: mlp_ref.product bounds the tensor cores' sums, mlp_ref.gate_error the gate's arithmetic; an output adds
half its spacing.  Whole-number operands whose sums FP32 holds are compared bit for bit, dropped elements too.
"""
import numpy as np
import pytest
import torch

import act_ref as A
import mlp_ref as R
from fac_whitening_gb300 import gift as G
from gpu_util import DEV, ctx, status

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
FNS = ["silu", "gelu", "gelu_tanh"]


def host(t):
    return t.detach().double().cpu().numpy()


def put(x, dt="f32", off=False):
    """x on the device in type dt; off: one element past an allocation's start."""
    if x is None:
        return None
    t = torch.as_tensor(np.ascontiguousarray(x)).to(DEV, DT[dt])
    if not off:
        return t
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
    flat[1:].copy_(t.reshape(-1))
    return flat[1:].view(t.shape)


class Out:
    """An output of n elements between two guards that nothing may write."""
    GUARD = 4096

    def __init__(self, shape, dt, off=False):
        n = int(np.prod(shape))
        self.flat = torch.full((2 * self.GUARD + n + 1,), 77, dtype=dt, device=DEV)
        self.at, self.n = self.GUARD + (1 if off else 0), n
        self.t = self.flat[self.at:self.at + n].view(shape)

    def checked(self):
        assert (self.flat[:self.at] == 77).all() and (self.flat[self.at + self.n:] == 77).all()
        return self.t


def rounded(x, dt):
    """x as the type holds it, in 64 bits."""
    return torch.as_tensor(np.ascontiguousarray(x)).to(DT[dt]).double().numpy()


def normal(rng, *shape, dt="f32"):
    return rounded(rng.standard_normal(shape), dt)


def workspace(op, dt, T, d_out, d_in, c=None):
    n = G.gift_act_workspace_bytes(c or ctx(), op, DT[dt], T, d_out, d_in)
    return torch.full((max(n, 1),), 0xFF, dtype=torch.uint8, device=DEV)   # NaN wherever it is read unwritten


def rng_of(seed, step):
    return torch.tensor([seed, step], dtype=torch.int64, device=DEV)


def gated_forward(x, Wg, Wu, fn, dt, bg=None, bu=None, fmt=None, kept=True, off=False, c=None):
    T, d = x.shape
    f = Wg.shape[0]
    h = Out((T, f), DT[dt], off)
    g, u = (Out((T, f), DT[dt], off), Out((T, f), DT[dt], off)) if kept else (None, None)
    codes = scales = None
    if fmt:
        cb, sb = G.gift_act_sizes(fmt, T, f)
        codes, scales = Out((cb,), torch.uint8, off), Out((sb,), torch.uint8, off)
    st = status()
    G.gift_gated_forward(c or ctx(), put(x, dt, off), put(Wg, dt, off), put(Wu, dt, off), fn, h.t,
                         gate=g and g.t, up=u and u.t, bg=put(bg), bu=put(bu), fmt=fmt or "e4m3",
                         codes=codes and codes.t, scales=scales and scales.t,
                         ws=workspace("gated_forward", dt, T, f, d, c), status=st)
    out = {"h": host(h.checked()), "status": int(st.item())}
    if kept:
        out["gate"], out["up"] = host(g.checked()), host(u.checked())
    if fmt:
        out["codes"] = codes.checked().cpu().numpy().reshape(T, f)
        out["scales"] = scales.checked().cpu().numpy().reshape(T, -1)
    return out


def linear(x, W, dt, bias=None, residual=None, p=0.0, rng=None, site=0, off=False, inplace=False, c=None):
    T, d_in = x.shape
    d_out = W.shape[0]
    y, st = Out((T, d_out), DT[dt], off), status()
    res = put(residual, dt, off)
    if inplace:
        y.t.copy_(res)
        res = y.t
    G.gift_linear_forward(c or ctx(), put(x, dt, off), put(W, dt, off), y.t, bias=put(bias), residual=res, p=p,
                          rng=rng, site=site, ws=workspace("linear_forward", dt, T, d_out, d_in, c), status=st)
    assert int(st.item()) == 0
    return host(y.checked())


def input_grad(delta, W, dt, delta2=None, W2=None, off=False, c=None):
    T, d_out = delta.shape
    d_in = W.shape[1]
    dx, st = Out((T, d_in), DT[dt], off), status()
    G.gift_input_grad(c or ctx(), put(delta, dt, off), put(W, dt, off), dx.t, delta2=put(delta2, dt, off),
                      W2=put(W2, dt, off), ws=workspace("input_grad", dt, T, d_out, d_in, c), status=st)
    assert int(st.item()) == 0
    return host(dx.checked())


def gated_backward(dy, W, gate, up, fn, dt, off=False, inplace=False, c=None):
    T, d_out = dy.shape
    f = W.shape[1]
    dg, du, st = Out((T, f), DT[dt], off), Out((T, f), DT[dt], off), status()
    g, u = put(gate, dt, off), put(up, dt, off)
    if inplace:
        dg.t.copy_(g)
        du.t.copy_(u)
        g, u = dg.t, du.t
    G.gift_gated_backward(c or ctx(), put(dy, dt, off), put(W, dt, off), g, u, fn, dg.t, du.t,
                          ws=workspace("gated_backward", dt, T, d_out, f, c), status=st)
    assert int(st.item()) == 0
    return host(dg.checked()), host(du.checked())


def whole(rng, dt, rows, k, top=None):
    """Whole numbers; FP32's take three BF16 terms."""
    return rng.integers(-(top or 3), (top or 3) + 1, (rows, k)).astype(np.float64)


# One token to more than a tile, odd and even, k of one block and of several segments, columns of one group and of several
# tiles, and of tiles of each width (64, 128, 192, 256).
SHAPES = [(1, 1, 1), (1, 8, 16), (2, 64, 128), (3, 129, 257), (33, 72, 144), (130, 513, 96), (257, 40, 136),
          (300, 1100, 528), (5, 2500, 300), (1, 1536, 1024), (300, 72, 64), (300, 100, 192), (600, 130, 384),
          (700, 257, 250)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("off", [False, True], ids=["aligned", "unaligned"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_products_of_whole_numbers_are_exact(shape, dt, off):
    T, k, n = shape
    rng = np.random.default_rng(T + 7 * k + 31 * n)
    # FP32: values of up to 18 bits (three terms) against -1, 0, 1 in few of the k places, sums below 2^24
    big = (1 << 17) + 1
    if dt == "f32":
        x = rng.integers(-big, big + 1, (T, k)).astype(np.float64)
        x[:, 60:] = rng.integers(-3, 4, x[:, 60:].shape)
    else:
        x = whole(rng, dt, T, k, 8)
    W, W2 = whole(rng, dt, n, k, 1), whole(rng, dt, n, k, 1)
    assert (np.abs(x) @ np.abs(W.T)).max() < 2 ** 24
    y = linear(x, W, dt, off=off)
    assert np.array_equal(y, rounded(x @ W.T, dt))
    out = gated_forward(x, W, W2, "silu", dt, off=off)
    assert out["status"] == 0
    assert np.array_equal(out["gate"], rounded(x @ W.T, dt)) and np.array_equal(out["up"], rounded(x @ W2.T, dt))
    V, V2 = np.ascontiguousarray(W.T), np.ascontiguousarray(W2.T)
    assert np.array_equal(input_grad(x, V, dt, off=off), rounded(x @ V, dt))
    half = np.floor(x / 2)
    assert np.array_equal(input_grad(x, V, dt, half, V2, off=off), rounded(x @ V + half @ V2, dt))
    # gate 0 at a'(0) = 1/2 and a(0) = 0
    dg, du = gated_backward(x, V, np.zeros((T, n)), np.full((T, n), 2.0), "silu", dt, off=off)
    assert np.array_equal(dg, rounded(x @ V, dt)) and not du.any()


@pytest.mark.parametrize("fn", FNS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("off", [False, True], ids=["aligned", "unaligned"])
@pytest.mark.parametrize("shape,fmt,bias", [((1, 1, 1), "e4m3", True), ((3, 129, 257), "e5m2", False),
                                            ((130, 200, 272), "e4m3", True), ((259, 33, 128), None, True),
                                            ((64, 700, 16), "e5m2", True)], ids=str)
def test_gated_forward(shape, fmt, bias, dt, off, fn):
    T, d, f = shape
    rng = np.random.default_rng(T + d + f)
    x, Wg, Wu = normal(rng, T, d, dt=dt), normal(rng, f, d, dt=dt) / 8, normal(rng, f, d, dt=dt) / 8
    x[0] *= 4.0
    bg, bu = (rounded(rng.standard_normal(f), "f32"), rounded(rng.standard_normal(f), "f32")) if bias else (None, None)
    out = gated_forward(x, Wg, Wu, fn, dt, bg, bu, fmt, off=off)
    assert out["status"] == 0
    (g, eg), (u, eu) = R.product(x, Wg.T, dt), R.product(x, Wu.T, dt)
    if bias:
        g, u = g + bg, u + bu
        eg, eu = eg + R.U32 * np.abs(g), eu + R.U32 * np.abs(u)
    assert (np.abs(out["gate"] - g) <= eg + R.half_step(g, dt) * 1.01).all()
    assert (np.abs(out["up"] - u) <= eu + R.half_step(u, dt) * 1.01).all()
    a, _ = R.gate(g, fn)
    h = a * u
    # |a'| <= 1.13
    eh = 1.13 * eg * (np.abs(u) + eu) + np.abs(a) * eu + (R.gate_error(g, fn) + 2 * R.U32) * np.abs(h)
    assert (np.abs(out["h"] - h) <= eh + 1.01 * R.half_step(h, dt) + 1e-37).all()
    if not fmt:
        return
    if dt == "f32":   # of the h that is returned
        codes, scales = A.encode(out["h"], fmt)
        assert np.array_equal(out["scales"], scales) and np.array_equal(out["codes"], codes)
        return
    v, s = A.decode(out["codes"], out["scales"], fmt), out["scales"].astype(np.float64) - 127
    top = A.magnitudes(fmt)[-1]
    for i in range(s.shape[1]):   # the smallest scale that holds the group, up to h's own error
        c = slice(128 * i, 128 * (i + 1))
        lo, hi = (np.abs(h[:, c]) - eh[:, c]).max(1), (np.abs(h[:, c]) + eh[:, c]).max(1)
        assert (lo <= top * 2.0 ** s[:, i]).all() and ((hi > top * 2.0 ** (s[:, i] - 1)) | (s[:, i] == -110)).all()
    steps = 2.0 ** np.repeat(s, 128, axis=1)[:, :f] * A.magnitudes(fmt)[1]
    half = {"e4m3": 2.0 ** -4, "e5m2": 2.0 ** -3}[fmt]
    assert (np.abs(v - h) <= 1.01 * eh + np.maximum(1.01 * half * np.abs(h), steps / 2)).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("off", [False, True], ids=["aligned", "unaligned"])
def test_gated_forward_without_what_is_optional(dt, off):
    rng = np.random.default_rng(8)
    x, Wg, Wu = normal(rng, 140, 200, dt=dt), normal(rng, 272, 200, dt=dt) / 8, normal(rng, 272, 200, dt=dt) / 8
    full = gated_forward(x, Wg, Wu, "silu", dt, fmt="e4m3", off=off)
    kept = gated_forward(x, Wg, Wu, "silu", dt, fmt="e4m3", kept=False, off=off)
    for k in ("h", "codes", "scales"):
        assert np.array_equal(full[k], kept[k]), k
    # without the checkpoint BF16 sums are folded less often: h within its rounding and that of the sums
    plain = gated_forward(x, Wg, Wu, "silu", dt, kept=False, off=off)
    (g, eg), (u, eu) = R.product(x, Wg.T, dt), R.product(x, Wu.T, dt)
    a, _ = R.gate(g, "silu")
    e = 1.13 * eg * (np.abs(u) + eu) + np.abs(a) * eu + (R.gate_error(g, "silu") + 2 * R.U32) * np.abs(a * u)
    assert (np.abs(plain["h"] - full["h"]) <= 2 * e + 2.02 * R.half_step(full["h"], dt)).all()
    # one bias alone
    b = rounded(rng.standard_normal(272), "f32")
    only = gated_forward(x, Wg, Wu, "silu", dt, bg=b, off=off)
    both = gated_forward(x, Wg, Wu, "silu", dt, bg=b, bu=np.zeros(272), off=off)
    for k in ("h", "gate", "up"):
        assert np.array_equal(only[k], both[k]), k


@pytest.mark.parametrize("fn", FNS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("off", [False, True], ids=["aligned", "unaligned"])
@pytest.mark.parametrize("inplace", [False, True], ids=["", "inplace"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (3, 129, 257), (130, 200, 272), (259, 33, 128), (64, 700, 16)], ids=str)
def test_gated_backward(shape, dt, off, inplace, fn):
    T, d, f = shape
    rng = np.random.default_rng(T + d + f)
    dy, W = normal(rng, T, d, dt=dt), normal(rng, d, f, dt=dt)
    gate, up = normal(rng, T, f, dt=dt) * 2, normal(rng, T, f, dt=dt)
    gate[0, :min(f, 8)] = rounded([0.0, -0.0, 30.0, -30.0, 100.0, -100.0, 1e-30, -8.0], dt)[:min(f, 8)]
    dg, du = gated_backward(dy, W, gate, up, fn, dt, off, inplace)
    dh, e = R.product(dy, W, dt)
    a, slope = R.gate(gate, fn)
    ge = R.gate_error(gate, fn)
    want = dh * up * slope
    # a' = s + g z' s (1 - s): its terms are at most 1 and 2 + |g|, and cancel
    es = ge * (np.abs(slope) + 2.0 * np.abs(a) + 1.0) * 1.5
    assert (np.abs(dg - want) <= np.abs(up) * (e * (np.abs(slope) + es) + np.abs(dh) * es) +
            4 * R.U32 * np.abs(want) + 1.01 * R.half_step(want, dt) + 1e-37).all()
    want = dh * a
    assert (np.abs(du - want) <= e * np.abs(a) * 1.01 + (ge + 2 * R.U32) * np.abs(want) +
            1.01 * R.half_step(want, dt) + 1e-37).all()


@pytest.mark.parametrize("p", [0.0, 0.1, 0.5])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("off", [False, True], ids=["aligned", "unaligned"])
@pytest.mark.parametrize("extras", ["none", "bias", "residual", "both", "inplace"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (3, 129, 257), (140, 200, 272), (5, 4000, 48)], ids=str)
def test_linear(shape, dt, off, extras, p):
    T, k, n = shape
    rng = np.random.default_rng(T + k + n)
    x, W = normal(rng, T, k, dt=dt), normal(rng, n, k, dt=dt)
    bias = rounded(rng.standard_normal(n), "f32") if extras in ("bias", "both") else None
    res = normal(rng, T, n, dt=dt) if extras in ("residual", "both", "inplace") else None
    seed, step, site = 0x123456789ABCDEF, 0x1_0000_0007, 3
    y = linear(x, W, dt, bias, res, p, rng_of(seed, step), site, off, extras == "inplace")
    v, e = R.product(x, W.T, dt)
    if bias is not None:
        v, e = v + bias, e + R.U32 * np.abs(v + bias)
    want = R.drop(v, p, seed, step, site)
    e = R.drop(e, p, seed, step, site) + 3 * R.U32 * np.abs(want)
    if p:
        dropped = ~R.keep(T, n, p, seed, step, site)
        assert np.array_equal(y[dropped], (np.zeros_like(v) if res is None else res)[dropped])
    if res is not None:
        want = want + res
    assert (np.abs(y - want) <= e + 2 * R.U32 * np.abs(want) + 1.01 * R.half_step(want, dt)).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("off", [False, True], ids=["aligned", "unaligned"])
@pytest.mark.parametrize("two", [False, True], ids=["one", "two"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (3, 129, 257), (140, 200, 272), (5, 4000, 48), (300, 70, 65)], ids=str)
def test_input_grad(shape, dt, off, two):
    T, k, n = shape
    rng = np.random.default_rng(T + k + n)
    a, W = normal(rng, T, k, dt=dt), normal(rng, k, n, dt=dt)
    a2, W2 = (normal(rng, T, k, dt=dt), normal(rng, k, n, dt=dt)) if two else (None, None)
    dx = input_grad(a, W, dt, a2, W2, off)
    want, e = R.product(np.hstack([a, a2]) if two else a, np.vstack([W, W2]) if two else W, dt)
    assert (np.abs(dx - want) <= e + 1.01 * R.half_step(want, dt)).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("off", [False, True], ids=["aligned", "unaligned"])
@pytest.mark.parametrize("p", [0.0, 1e-5, 0.1, 0.9, 65535 / 65536])
@pytest.mark.parametrize("shape", [(1, 1), (1, 16), (3, 129), (9, 512), (65, 1361), (300, 640), (5000, 24)], ids=str)
def test_dropout(shape, p, off, dt):
    T, d = shape
    rng = np.random.default_rng(T + d)
    x, res, dy = (normal(rng, T, d, dt=dt) for _ in range(3))
    bias = rounded(rng.standard_normal(d), "f32")
    seed, step, site = 0x7FEDCBA987654321, 41, 0xFFFFFFFF
    r = rng_of(seed, step)
    y, dx, db = Out((T, d), DT[dt], off), Out((T, d), DT[dt], off), Out((d,), torch.float32)
    G.gift_dropout_forward(ctx(), put(x, dt, off), y.t, p, r, site, put(bias), put(res, dt, off))
    G.gift_dropout_backward(ctx(), put(dy, dt, off), dx.t, p, r, site, db.t,
                            ws=workspace("dropout_backward", dt, T, d, d))
    v = R.drop(x + bias, p, seed, step, site)
    want = v + res
    assert (np.abs(host(y.checked()) - want) <= 3 * R.U32 * np.abs(v) + R.U32 * np.abs(want) +
            1.01 * R.half_step(want, dt)).all()
    want = R.drop(dy, p, seed, step, site)
    assert (np.abs(host(dx.checked()) - want) <= R.U32 * np.abs(want) + 1.01 * R.half_step(want, dt)).all()
    assert np.array_equal(host(dx.t) == 0, want == 0)
    assert (np.abs(host(db.checked()) - want.sum(0)) <= (T + 1) * R.U32 * np.abs(want).sum(0)).all()
    y2, dx2 = Out((T, d), DT[dt], off), Out((T, d), DT[dt], off)   # without the extras, in place
    y2.t.copy_(put(x, dt))
    dx2.t.copy_(put(dy, dt))
    G.gift_dropout_forward(ctx(), y2.t, y2.t, p, r, site)
    G.gift_dropout_backward(ctx(), dx2.t, dx2.t, p, r, site)
    want = R.drop(x, p, seed, step, site)
    assert (np.abs(host(y2.checked()) - want) <= R.U32 * np.abs(want) + 1.01 * R.half_step(want, dt)).all()
    y2.t.copy_(put(res, dt))   # in the residual's place
    G.gift_dropout_forward(ctx(), put(x, dt, off), y2.t, p, r, site, put(bias), y2.t)
    assert torch.equal(y2.checked(), y.t)
    assert torch.equal(dx2.checked(), dx.t)
