"""GPU parity of the 8-bit activation checkpoint, the layer norm and the weight gradient with
their 64-bit statements.

Tolerances.  u = 2^-24.  A sum of N FP32 terms in any order is off by at most N u sum|terms|
(plus the rounding of each term); a BF16 result, 8 significant bits, adds half
its spacing: at most 2^-8 of the value.  Where
the tensor cores sum, a step truncates instead of rounding (twice u).  Codes, scale bytes and
decoded values are compared bit for bit.
"""
import numpy as np
import pytest
import torch

import act_ref as R
from fac_whitening_gb300 import gift as G
from gpu_util import DEV, ctx, status

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def dev(x, dt=torch.float32):
    return None if x is None else torch.as_tensor(np.ascontiguousarray(x)).to(DEV, dt)


def host(t):
    return t.detach().double().cpu().numpy()


def unaligned(t):
    """The same dense tensor one element past an allocation's start."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    flat[1:].copy_(t.reshape(-1))
    return flat[1:].view(t.shape)


def empty(shape, dt, off):
    t = torch.empty(*shape, dtype=dt, device=DEV)
    return unaligned(t) if off else t


def rows(T, d, dt, seed, offset=0.0):
    """Activation-like rows rounded to dt: unequal channels, some tokens much larger."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, d)) * np.exp(rng.standard_normal(d)) * np.exp(rng.standard_normal((T, 1))) + offset
    return torch.as_tensor(x).to(DT[dt])


def act_encode(x, fmt, off=False):
    T, d = x.shape
    cb, sb = G.gift_act_sizes(fmt, T, d)
    codes, scales, st = empty((cb,), torch.uint8, off), empty((sb,), torch.uint8, off), status()
    G.gift_act_encode(ctx(), x, fmt, codes, scales, status=st)
    return codes, scales, int(st.item())


SHAPES = [(1, 1), (1, 128), (1, 127), (3, 129), (5, 16), (7, 1000), (33, 256), (64, 8), (2, 6144), (1, 16384), (300, 333)]


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("off", [False, True], ids=["aligned", "unaligned"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_checkpoint_bits(shape, dt, fmt, off):
    T, d = shape
    x = rows(T, d, dt, 10 * T + d)
    x[0, 0] = -0.0
    if T > 2:
        x[1] = 0.0
        x[2] *= 1e-37
    xd = x.to(DEV)
    codes, scales, st = act_encode(unaligned(xd) if off else xd, fmt, off)
    want_c, want_s = R.encode(x.double().numpy(), fmt)
    assert st == 0
    assert np.array_equal(scales.cpu().numpy().reshape(want_s.shape), want_s)
    assert np.array_equal(codes.cpu().numpy().reshape(T, d), want_c)
    want = R.decode(want_c, want_s, fmt)
    for out_dt in ("f32", "bf16"):
        out, st = empty((T, d), DT[out_dt], off), status()
        G.gift_act_decode(ctx(), codes, scales, fmt, out, status=st)
        assert int(st.item()) == 0
        got = host(out)
        assert np.array_equal(got, want) and np.array_equal(np.signbit(got), np.signbit(want))


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_checkpoint_extremes_and_ties(fmt):
    emax = R.EMAX[fmt]
    mags = R.magnitudes(fmt)
    mids = (mags[:-1] + mags[1:]) / 2
    x = np.zeros((6, 384), dtype=np.float32)
    x[0, :] = 3.4e38
    x[1, :] = -3.4028234e38
    x[2, :] = 1e-45
    x[3, :len(mids)] = mids          # every tie of the format, with the scale pinned to 1
    x[3, 128:128 + len(mids)] = -mids
    x[3, [127, 255]] = mags[-1]
    x[4, 0], x[4, 128], x[4, 256] = mags[-1], np.nextafter(np.float32(mags[-1]), np.float32(np.inf)), 2.0 ** emax
    x[5, ::2] = 2.0 ** -126
    codes, scales, st = act_encode(dev(x), fmt)
    want_c, want_s = R.encode(x, fmt)
    assert st == 0
    assert np.array_equal(scales.cpu().numpy().reshape(want_s.shape), want_s)
    assert np.array_equal(codes.cpu().numpy().reshape(x.shape), want_c)
    assert want_s[4, 0] == 127 and want_s[4, 1] == 128
    out = torch.empty(6, 384, device=DEV)
    G.gift_act_decode(ctx(), codes, scales, fmt, out)
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_every_code_and_scale_decodes_exactly(fmt):
    kmax = 127 - R.EMAX[fmt]
    last = len(R.magnitudes(fmt))
    codes = np.array([c for c in range(256) if (c & 127) < last], dtype=np.uint8)
    s = np.arange(17, kmax + 128, dtype=np.uint8)
    c2 = np.zeros((len(s), 256), dtype=np.uint8)
    c2[:, :len(codes)] = codes
    s2 = np.repeat(s[:, None], 2, axis=1)
    want = R.decode(c2, s2, fmt)
    for dt in ("f32", "bf16"):
        out = torch.empty(len(s), 256, dtype=DT[dt], device=DEV)
        G.gift_act_decode(ctx(), dev(c2, torch.uint8), dev(s2, torch.uint8), fmt, out)
        assert np.array_equal(host(out), want)


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_nonfinite_groups_are_marked(bad, dt):
    x = rows(4, 300, dt, 3)
    x[1, 130] = bad
    codes, scales, st = act_encode(x.to(DEV), "e4m3")
    assert st == G.ERR_NONFINITE
    s = scales.cpu().numpy().reshape(4, 3)
    assert s[1, 1] == 255 and (s == 255).sum() == 1
    out, st = torch.empty(4, 300, dtype=DT[dt], device=DEV), status()
    G.gift_act_decode(ctx(), codes, scales, "e4m3", out, status=st)
    assert int(st.item()) == G.ERR_NONFINITE
    nan = torch.isnan(out).cpu().numpy()
    assert nan[1, 128:256].all() and nan.sum() == 128


# ---- layer norm ------------------------------------------------------------------------------
def norm_inputs(T, d, dt, seed, affine=True, offset=0.0):
    rng = np.random.default_rng(seed)
    x = rows(T, d, dt, seed, offset)
    gamma = (1 + 0.3 * rng.standard_normal(d)).astype(np.float32) if affine else None
    beta = (0.5 * rng.standard_normal(d)).astype(np.float32) if affine else None
    return x, gamma, beta


def forward(x, gamma, beta, eps, fmt=None, off=False):
    T, d = x.shape
    y, mean, rstd, st = empty((T, d), x.dtype, off), empty((T,), torch.float32, off), empty((T,), torch.float32, off), status()
    codes = scales = None
    if fmt:
        cb, sb = G.gift_act_sizes(fmt, T, d)
        codes, scales = empty((cb,), torch.uint8, off), empty((sb,), torch.uint8, off)
    G.gift_layernorm_forward(ctx(), x, dev(gamma), dev(beta), eps, y, mean=mean, rstd=rstd, fmt=fmt or "e4m3",
                             codes=codes, scales=scales, status=st)
    return y, mean, rstd, codes, scales, int(st.item())


NORM_SHAPES = [(1, 1), (1, 2), (3, 7), (1, 16384), (5, 128), (17, 1361), (512, 256), (9, 1536), (4, 6144), (3, 8200),
               (2, 40000), (130, 33)]


@pytest.mark.parametrize("off", [False, True], ids=["aligned", "unaligned"])
@pytest.mark.parametrize("affine", [True, False], ids=["affine", "plain"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", NORM_SHAPES, ids=str)
def test_norm_forward(shape, dt, affine, off):
    T, d = shape
    x, gamma, beta = norm_inputs(T, d, dt, T + d, affine, offset=0.7)
    xd = x.to(DEV)
    y, mean, rstd, _, _, st = forward(unaligned(xd) if off else xd, gamma, beta, 1e-5, off=off)
    assert st == 0
    xs = x.double().numpy()
    wy, wn, wm, wr = R.norm_forward(xs, gamma, beta, 1e-5)
    N = d + 8   # terms of a row's sums, and the operations around them
    tol_m = N * R.U32 * np.abs(xs).mean(axis=1)
    assert np.all(np.abs(host(mean) - wm) <= tol_m + 1e-30)
    # rstd moves by half the relative error of the variance: its own sum, and 2 mean error deviations
    assert np.all(np.abs(host(rstd) - wr) <= wr * (N * R.U32 + tol_m * wr + 4 * R.U32))
    g = 1.0 if gamma is None else np.abs(gamma)
    tol = g * (np.abs(wn) * (N * R.U32 + (tol_m * wr)[:, None]) + (tol_m * wr)[:, None] + 4 * R.U32 * np.abs(wn))
    tol = tol + 4 * R.U32 * (np.abs(wy) + (0 if beta is None else np.abs(beta))) + 1e-30
    if dt == "bf16":
        tol = tol + R.U16 * (np.abs(wy) + tol)
    assert np.all(np.abs(host(y) - wy) <= tol)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("off", [False, True], ids=["aligned", "unaligned"])
@pytest.mark.parametrize("shape", NORM_SHAPES, ids=str)
def test_norm_forward_checkpoint_is_the_encode_of_n(shape, fmt, off):
    # without gain and offset y is n itself, so codes and scales are gift_act_encode's of y, bit for bit
    T, d = shape
    x = rows(T, d, "f32", 5 * T + d).to(DEV)
    y, _, _, codes, scales, st = forward(unaligned(x) if off else x, None, None, 1e-5, fmt, off)
    assert st == 0
    want_c, want_s = R.encode(host(y), fmt)
    assert np.array_equal(scales.cpu().numpy().reshape(want_s.shape), want_s)
    assert np.array_equal(codes.cpu().numpy().reshape(T, d), want_c)
    # BF16 rows: the same checkpoint rule on the unrounded n, so within one rounding of it
    xb, gamma, beta = norm_inputs(T, d, "bf16", 5 * T + d)
    _, _, _, codes, scales, st = forward(xb.to(DEV), gamma, beta, 1e-5, fmt, off)
    _, wn, _, _ = R.norm_forward(xb.double().numpy(), gamma, beta, 1e-5)
    v = R.decode(codes.cpu().numpy().reshape(T, d), scales.cpu().numpy().reshape(T, -1), fmt)
    half = 2.0 ** (-4 if fmt == "e4m3" else -3)   # half a code step, relative to the value
    amax = np.repeat(np.maximum.reduceat(np.abs(wn), range(0, d, 128), axis=1), 128, axis=1)[:, :d]
    lowest = 2.0 ** (-17 if fmt == "e4m3" else -31)   # half the smallest step, relative to the group's amax
    assert st == 0 and np.all(np.abs(v - wn) <= half * np.abs(wn) + lowest * amax + (d + 16) * 4 * R.U32)


# aligned rows by every number of pieces per lane and of warps per row, whole and partial last pieces, and
# more rows than are resident at once
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(5000, 528), (3001, 1040), (2600, 1536), (700, 2064), (641, 3600), (400, 4112),
                                   (200, 8208), (320, 10000), (170, 16384), (160, 16400)], ids=str)
def test_norm_forward_of_many_aligned_rows(shape, dt):
    test_norm_forward(shape, dt, True, False)
    if dt == "bf16":
        test_norm_forward_checkpoint_is_the_encode_of_n(shape, "e4m3", False)


def test_norm_forward_constant_and_nonfinite_rows():
    x = rows(6, 200, "f32", 9)
    x[1] = 3.25
    x[2] = 0.0
    x[3, 17] = np.nan
    x[4, 5] = np.inf
    y, mean, rstd, codes, scales, st = forward(x.to(DEV), None, None, 1e-5, "e4m3")
    assert st == G.ERR_NONFINITE
    assert torch.equal(y[1:3], torch.zeros(2, 200, device=DEV))
    assert abs(rstd[1].item() * 1e-5 ** 0.5 - 1) < 1e-6 and mean[1].item() == 3.25
    s = scales.cpu().numpy().reshape(6, 2)
    assert (s[3] == 255).all() and (s[4] == 255).any() and (s[[0, 1, 2, 5]] != 255).all()
    good = R.norm_forward(x[[0, 5]].double().numpy(), None, None, 1e-5)[0]
    assert np.allclose(host(y)[[0, 5]], good, rtol=1e-4, atol=1e-5)


def test_norm_forward_large_offset():
    # deviations, not a difference of squares: an offset of 1000 deviations keeps 4 digits of them
    T, d = 8, 3000
    x = torch.as_tensor(np.random.default_rng(4).standard_normal((T, d)) + 1000.0).float()
    y = forward(x.to(DEV), None, None, 1e-5)[0]
    want = R.norm_forward(x.double().numpy(), None, None, 1e-5)[0]
    assert np.abs(host(y) - want).max() <= (d + 8) * R.U32 * 1000.0 * 1.2


def backward(dy, saved, gamma, rstd, mean=None, scales=None, fmt="e4m3", sums=(True, True), off=False):
    T, d = dy.shape
    dx, st = empty((T, d), dy.dtype, off), status()
    dg = empty((d,), torch.float32, off) if sums[0] else None
    db = empty((d,), torch.float32, off) if sums[1] else None
    ws = empty((G.gift_act_workspace_bytes(ctx(), "layernorm_backward", dy.dtype, T, d, d),), torch.uint8, off)
    ws.fill_(0xFF)   # NaN bit patterns: nothing may be read before it is written
    G.gift_layernorm_backward(ctx(), dy, saved, dev(gamma), rstd, dx, dg, db, mean=mean, scales=scales, fmt=fmt,
                              ws=ws, status=st)
    return dx, dg, db, int(st.item())


def check_backward(T, d, dt, dy, n, n_err, gamma, rstd, got):
    """got against the formula at n (64-bit), n_err bounding what the kernel's n is off by."""
    dx, dg, db, st = got
    wx, wg, wb = R.norm_backward(dy, n, gamma, rstd)
    assert st == 0
    h = np.abs(dy) * (1.0 if gamma is None else np.abs(gamma))
    N = d + 8
    ma, mb = h.mean(axis=1, keepdims=True), (h * (np.abs(n) + n_err)).mean(axis=1, keepdims=True)
    tol = rstd[:, None] * (8 * R.U32 * (h + ma + np.abs(n) * mb) + N * R.U32 * (ma + np.abs(n) * mb) +
                           n_err * mb + np.abs(n) * (h * n_err).mean(axis=1, keepdims=True)) + 1e-30
    if dt == "bf16":
        tol = tol + R.U16 * (np.abs(wx) + tol)
    assert np.all(np.abs(host(dx) - wx) <= tol)
    if dg is not None:
        t = ((T + 4) * R.U32 * np.abs(dy * n) + np.abs(dy) * n_err).sum(axis=0)
        assert np.all(np.abs(host(dg) - wg) <= t + 1e-30)
    if db is not None:
        assert np.all(np.abs(host(db) - wb) <= T * R.U32 * np.abs(dy).sum(axis=0) + 1e-30)


BACK_SHAPES = NORM_SHAPES + [(700, 96), (2000, 40), (333, 4096)]


@pytest.mark.parametrize("off", [False, True], ids=["aligned", "unaligned"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", BACK_SHAPES, ids=str)
def test_norm_backward_from_input(shape, dt, off):
    T, d = shape
    x, gamma, _ = norm_inputs(T, d, dt, 3 * T + d, affine=(T + d) % 3 != 0)
    dy = rows(T, d, dt, 77 + T + d)
    xs = x.double().numpy()
    _, _, mean, rstd = R.norm_forward(xs, None, None, 1e-5)
    mean, rstd = mean.astype(np.float32), rstd.astype(np.float32)
    n = (xs - mean[:, None].astype(np.float64)) * rstd[:, None].astype(np.float64)
    put = unaligned if off else (lambda t: t)
    got = backward(put(dy.to(DEV)), put(x.to(DEV)), gamma, dev(rstd), mean=dev(mean), off=off)
    check_backward(T, d, dt, dy.double().numpy(), n, 3 * R.U32 * np.abs(n), gamma, rstd.astype(np.float64), got)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("off", [False, True], ids=["aligned", "unaligned"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", BACK_SHAPES, ids=str)
def test_norm_backward_from_checkpoint(shape, dt, fmt, off):
    T, d = shape
    x, gamma, _ = norm_inputs(T, d, dt, 3 * T + d, affine=(T + d) % 3 != 0)
    dy = rows(T, d, dt, 78 + T + d)
    _, n0, _, rstd = R.norm_forward(x.double().numpy(), None, None, 1e-5)
    rstd = rstd.astype(np.float32)
    codes, scales = R.encode(n0.astype(np.float32), fmt)
    n = R.decode(codes, scales, fmt)
    put = unaligned if off else (lambda t: t)
    got = backward(put(dy.to(DEV)), put(dev(codes, torch.uint8)), gamma, dev(rstd),
                   scales=put(dev(scales, torch.uint8)), fmt=fmt, off=off)
    check_backward(T, d, dt, dy.double().numpy(), n, 0.0, gamma, rstd.astype(np.float64), got)


@pytest.mark.parametrize("sums", [(False, False), (True, False), (False, True)], ids=str)
def test_norm_backward_optional_sums(sums):
    T, d = 70, 200
    x, gamma, _ = norm_inputs(T, d, "f32", 6)
    dy = rows(T, d, "f32", 7)
    _, _, mean, rstd = R.norm_forward(x.double().numpy(), None, None, 1e-5)
    args = (dy.to(DEV), x.to(DEV), gamma, dev(rstd))
    full, part = backward(*args, mean=dev(mean)), backward(*args, mean=dev(mean), sums=sums)
    for a, b, on in zip(full[:3], part[:3], (True,) + sums):
        assert (b is not None) == on and (b is None or torch.equal(a, b))


def test_norm_gradients_against_differences():
    # the whole chain on the GPU (forward's statistics into backward) against central differences of
    # the 64-bit forward: h^2 truncation and FP32 rounding of the gradient both stay below 1e-4
    T, d = 5, 60
    x, gamma, beta = norm_inputs(T, d, "f32", 21)
    w = rows(T, d, "f32", 22)
    _, mean, rstd, _, _, _ = forward(x.to(DEV), gamma, beta, 1e-5)
    dx, dg, db, _ = backward(w.to(DEV), x.to(DEV), gamma, rstd, mean=mean)
    rng = np.random.default_rng(5)
    xs, ws = x.double().numpy(), w.double().numpy()
    g64, b64 = gamma.astype(np.float64), beta.astype(np.float64)
    f = lambda x, g, b: float((ws * R.norm_forward(x, g, b, 1e-5)[0]).sum())  # noqa: E731
    for k, got in enumerate((dx, dg, db)):
        v = rng.standard_normal((T, d) if k == 0 else d)
        at = lambda e: f(xs + (e * v if k == 0 else 0), g64 + (e * v if k == 1 else 0), b64 + (e * v if k == 2 else 0))  # noqa: E731
        diff = (at(1e-4) - at(-1e-4)) / 2e-4
        scale = np.linalg.norm(host(got)) * np.linalg.norm(v)
        assert abs(diff - (host(got) * v).sum()) <= 1e-4 * scale


def test_norm_backward_nonfinite_is_reported_and_stays_in_its_row():
    T, d = 6, 300
    x, gamma, _ = norm_inputs(T, d, "f32", 8)
    dy = rows(T, d, "f32", 9)
    _, n0, _, rstd = R.norm_forward(x.double().numpy(), None, None, 1e-5)
    codes, scales = R.encode(n0.astype(np.float32), "e4m3")
    scales[2, 1] = 255
    dx, dg, db, st = backward(dy.to(DEV), dev(codes, torch.uint8), gamma, dev(rstd), scales=dev(scales, torch.uint8))
    assert st == G.ERR_NONFINITE
    ok = torch.isfinite(dx).all(dim=1).cpu().numpy()
    assert not ok[2] and ok[[0, 1, 3, 4, 5]].all() and torch.isfinite(db).all()
    bad = torch.isnan(dg).cpu().numpy()
    assert bad[128:256].all() and bad.sum() == 128


# ---- weight gradient -------------------------------------------------------------------------
def weight_grad(delta, codes, scales, fmt, d_in, gamma=None, beta=None, db=True, off=False):
    T, d_out = delta.shape
    dW, st = empty((d_out, d_in), torch.float32, off), status()
    bias = empty((d_out,), torch.float32, off) if db else None
    ws = empty((G.gift_act_workspace_bytes(ctx(), "weight_grad", delta.dtype, T, d_out, d_in),), torch.uint8, off)
    ws.fill_(0xFF)
    G.gift_weight_grad(ctx(), delta, codes, scales, fmt, dW, db=bias, gamma=dev(gamma), beta=dev(beta), ws=ws,
                       status=st)
    assert int(st.item()) == 0
    return dW, bias


WG_SHAPES = [(1, 1, 1), (1, 64, 256), (3, 5, 7), (63, 64, 128), (64, 128, 256), (65, 129, 257), (512, 64, 256),
             (300, 200, 384), (1000, 136, 1008), (257, 1021, 300), (129, 7, 2731), (2, 1536, 100), (4097, 256, 256),
             (640, 520, 912), (1, 3, 5000)]


@pytest.mark.parametrize("off", [False, True], ids=["aligned", "unaligned"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("shape", WG_SHAPES, ids=str)
def test_weight_grad_integers_are_exact(shape, fmt, dt, off):
    # small integers: every sum is exact in FP32 in any order, so dW and db must be the integers
    T, d_out, d_in = shape
    rng = np.random.default_rng(T + 3 * d_out + 7 * d_in)
    delta = rng.integers(-3, 4, (T, d_out)).astype(np.float64)
    v = rng.integers(-7, 8, (T, d_in)).astype(np.float64)
    codes, scales = R.encode(v, fmt)
    v = R.decode(codes, scales, fmt)
    want, wb = R.weight_grad(delta, v)
    put = unaligned if off else (lambda t: t)
    dW, db = weight_grad(put(dev(delta, DT[dt])), put(dev(codes, torch.uint8)), put(dev(scales, torch.uint8)), fmt,
                         d_in, off=off)
    assert np.array_equal(host(db), wb)
    assert np.array_equal(host(dW), want)


@pytest.mark.parametrize("affine", ["none", "gain", "both", "offset"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 64, 256), (65, 129, 257), (512, 64, 256), (1000, 136, 1008), (5003, 264, 528)],
                         ids=str)
def test_weight_grad_against_the_formula(shape, dt, affine):
    T, d_out, d_in = shape
    fmt = "e4m3" if d_in % 2 else "e5m2"
    rng = np.random.default_rng(T + d_out)
    delta = rows(T, d_out, dt, T + d_out)
    codes, scales = R.encode(rows(T, d_in, "f32", T + d_in).double().numpy(), fmt)
    v = R.decode(codes, scales, fmt)
    gamma = (1 + 0.3 * rng.standard_normal(d_in)).astype(np.float32) if affine in ("gain", "both") else None
    beta = (0.5 * rng.standard_normal(d_in)).astype(np.float32) if affine in ("offset", "both") else None
    ds = delta.double().numpy()
    want, wb = R.weight_grad(ds, v, gamma, beta)
    dW, db = weight_grad(delta.to(DEV), dev(codes, torch.uint8), dev(scales, torch.uint8), fmt, d_in, gamma, beta,
                         db=affine != "offset")
    size = np.abs(ds).T @ np.abs(v) * (1.0 if gamma is None else np.abs(gamma))
    if beta is not None:
        size = size + np.outer(np.abs(ds).sum(axis=0), np.abs(beta))
    assert np.all(np.abs(host(dW) - want) <= (T + 8) * 2 * R.U32 * size)
    # folded to nearest every 256 tokens, 16 truncating steps of at most 2u in a fold: 32 u, and the
    # folds' own rounding, of the whole
    assert np.linalg.norm(host(dW) - want) <= (32 + T / 256) * R.U32 * 1.3 * np.linalg.norm(want)
    if db is not None:
        assert np.all(np.abs(host(db) - wb) <= T * R.U32 * np.abs(ds).sum(axis=0))


def test_weight_grad_is_the_derivative_of_the_layer():
    # Y = v W^T, L = sum(delta Y): L is linear in W, so its difference along any direction is exact
    T, d_out, d_in = 70, 24, 144
    delta = rows(T, d_out, "bf16", 31)
    codes, scales = R.encode(rows(T, d_in, "f32", 32).double().numpy(), "e4m3")
    v, ds = R.decode(codes, scales, "e4m3"), delta.double().numpy()
    dW, _ = weight_grad(delta.to(DEV), dev(codes, torch.uint8), dev(scales, torch.uint8), "e4m3", d_in)
    dirn = np.random.default_rng(3).standard_normal((d_out, d_in))
    diff = (ds * (v @ dirn.T)).sum()
    assert abs(diff - (host(dW) * dirn).sum()) <= 1e-5 * np.linalg.norm(host(dW)) * np.linalg.norm(dirn)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(130, 40, 400), (300, 264, 528)], ids=str)
def test_weight_grad_marked_group_reaches_its_columns_only(shape, dt):
    T, d_out, d_in = shape
    delta = rows(T, d_out, dt, 5)
    codes, scales = R.encode(rows(T, d_in, "f32", 6).double().numpy(), "e4m3")
    scales[T - 2, 1] = 255
    dW, _ = weight_grad(delta.to(DEV), dev(codes, torch.uint8), dev(scales, torch.uint8), "e4m3", d_in)
    nan = torch.isnan(dW).cpu().numpy()
    assert nan[:, 128:256].all() and not nan[:, :128].any() and not nan[:, 256:].any()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_weight_grad_extreme_scales(dt):
    # checkpoint values at both ends of the scale range, gradients that bring the product back to one
    T, d_out, d_in = 96, 16, 256
    rng = np.random.default_rng(8)
    v = rng.choice([-1.0, 1.0, 0.5, 3.0], (T, d_in))
    v[:, :128] *= 2.0 ** 120
    v[:, 128:] *= 2.0 ** -100
    delta = rng.integers(-3, 4, (T, d_out)).astype(np.float64)
    codes, scales = R.encode(v, "e4m3")
    want, _ = R.weight_grad(delta, R.decode(codes, scales, "e4m3"))
    dW, _ = weight_grad(dev(delta, DT[dt]), dev(codes, torch.uint8), dev(scales, torch.uint8), "e4m3", d_in)
    assert np.array_equal(host(dW), want)


# db beside a full last tile and one with room, with tokens in one slice and in several, and where a tile
# more would cost another wave of tiles on 152 SMs
@pytest.mark.parametrize("affine", [False, True])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(300, 264, 512), (300, 264, 640), (9000, 100, 512), (9000, 100, 640),
                                   (1100, 1024, 4864)], ids=str)
def test_weight_grad_bias_gradient_of_every_tiling(shape, dt, affine):
    T, d_out, d_in = shape
    rng = np.random.default_rng(T + d_in)
    delta = rng.integers(-3, 4, (T, d_out)).astype(np.float64)
    codes, scales = R.encode(rng.integers(-7, 8, (T, d_in)).astype(np.float64), "e4m3")
    v = R.decode(codes, scales, "e4m3")
    gamma = rng.choice([-1.0, 0.5, 2.0], d_in).astype(np.float32) if affine else None
    beta = rng.integers(-4, 5, d_in).astype(np.float32) if affine else None
    want, wb = R.weight_grad(delta, v, gamma, beta)   # halves of integers below 2^23: exact in FP32
    d, c, s = dev(delta, DT[dt]), dev(codes, torch.uint8), dev(scales, torch.uint8)
    dW, db = weight_grad(d, c, s, "e4m3", d_in, gamma, beta)
    assert np.array_equal(host(dW), want) and np.array_equal(host(db), wb)
    dW, _ = weight_grad(d, c, s, "e4m3", d_in, gamma, beta, db=False)
    assert np.array_equal(host(dW), want)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_weight_grad_extreme_scales_of_a_wide_layer(dt, fmt):
    # the same through the tensor-core kernel, with single tokens at the ends of the range among others
    T, d_out, d_in = 300, 264, 528
    rng = np.random.default_rng(9)
    v = rng.choice([-1.0, 1.0, 0.5, 3.0], (T, d_in))
    delta = rng.integers(-3, 4, (T, d_out)).astype(np.float64)
    k = np.zeros(T, dtype=int)
    k[[3, 64, 200, 299]] = [100, -90, 60, -100]
    v, delta = np.ldexp(v, k[:, None]), np.ldexp(delta, -k[:, None])
    codes, scales = R.encode(v, fmt)
    want, _ = R.weight_grad(delta, R.decode(codes, scales, fmt))
    dW, _ = weight_grad(dev(delta, DT[dt]), dev(codes, torch.uint8), dev(scales, torch.uint8), fmt, d_in)
    assert np.array_equal(host(dW), want)


# ---- what every call holds to -----------------------------------------------------------------
def test_calls_repeat_bit_for_bit_and_keep_to_their_stream():
    T, d, d_out = 700, 520, 136
    x, gamma, beta = norm_inputs(T, d, "bf16", 41)
    dy, delta = rows(T, d, "bf16", 42), rows(T, d_out, "bf16", 43)
    side = torch.cuda.Stream()

    def step():
        y, mean, rstd, codes, scales, _ = forward(x.to(DEV), gamma, beta, 1e-5, "e4m3")
        dx, dg, db, _ = backward(dy.to(DEV), codes, gamma, rstd, scales=scales)
        dW, dB = weight_grad(delta.to(DEV), codes, scales, "e4m3", d, gamma, beta)
        return [y, mean, rstd, codes, scales, dx, dg, db, dW, dB]

    first = step()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        second = step()
    side.synchronize()
    for a, b in zip(first, second):
        assert torch.equal(a, b)


def test_calls_can_be_captured_and_replayed():
    T, d, d_out = 300, 384, 128
    x, gamma, beta = norm_inputs(T, d, "bf16", 51)
    xd, g, b = x.to(DEV), dev(gamma), dev(beta)
    delta = rows(T, d_out, "bf16", 52).to(DEV)
    cb, sb = G.gift_act_sizes("e4m3", T, d)
    codes, scales = empty((cb,), torch.uint8, False), empty((sb,), torch.uint8, False)
    y, rstd, dx = torch.empty_like(xd), empty((T,), torch.float32, False), torch.empty_like(xd)
    dg, db, dW = empty((d,), torch.float32, False), empty((d,), torch.float32, False), empty((d_out, d), torch.float32, False)
    w1 = empty((G.gift_act_workspace_bytes(ctx(), "layernorm_backward", torch.bfloat16, T, d, d),), torch.uint8, False)
    w2 = empty((G.gift_act_workspace_bytes(ctx(), "weight_grad", torch.bfloat16, T, d_out, d),), torch.uint8, False)

    def step():
        G.gift_layernorm_forward(ctx(), xd, g, b, 1e-5, y, rstd=rstd, codes=codes, scales=scales)
        G.gift_layernorm_backward(ctx(), y, codes, g, rstd, dx, dg, db, scales=scales, ws=w1)
        G.gift_weight_grad(ctx(), delta, codes, scales, "e4m3", dW, gamma=g, beta=b, ws=w2)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (y, codes, dx, dg, db, dW)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (y, codes, dx, dg, db, dW):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, (y, codes, dx, dg, db, dW)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("sms", [1, 7, 38])
def test_contexts_of_a_share_of_the_gpu(sms):
    c = G.Context(torch.cuda.current_device())
    G.gift_set_option(c, G.OPT_SMS, sms)
    T, d, d_out = 515, 272, 136
    delta = dev(np.random.default_rng(1).integers(-3, 4, (T, d_out)), torch.bfloat16)
    v = np.random.default_rng(2).integers(-7, 8, (T, d)).astype(np.float64)
    codes, scales = R.encode(v, "e4m3")
    dW, st = torch.empty(d_out, d, device=DEV), status()
    ws = torch.empty(G.gift_act_workspace_bytes(c, "weight_grad", torch.bfloat16, T, d_out, d), dtype=torch.uint8, device=DEV)
    G.gift_weight_grad(c, delta, dev(codes, torch.uint8), dev(scales, torch.uint8), "e4m3", dW, ws=ws, status=st)
    want, _ = R.weight_grad(host(delta), R.decode(codes, scales, "e4m3"))
    assert int(st.item()) == 0 and np.array_equal(host(dW), want)


def test_offsets_past_32_bits():
    # 4.6 G elements: the last rows lie beyond 2^32 elements
    T, d, d_out = 70000, 65536, 8
    gen = torch.Generator(device=DEV).manual_seed(1)
    x = torch.empty(T, d, dtype=torch.bfloat16, device=DEV)
    for t in range(0, T, 10000):
        x[t:t + 10000].normal_(generator=gen)
    codes, scales, st = act_encode(x, "e4m3")
    assert st == 0
    pick = [0, 32767, 32768, 65535, 65536, 69999]
    c2, s2 = codes.view(T, d), scales.view(T, d // 128)
    want_c, want_s = R.encode(host(x[pick]), "e4m3")
    assert np.array_equal(c2[pick].cpu().numpy(), want_c) and np.array_equal(s2[pick].cpu().numpy(), want_s)
    y, rstd = torch.empty_like(x), torch.empty(T, device=DEV)
    G.gift_act_decode(ctx(), codes, scales, "e4m3", y)
    assert np.array_equal(host(y[pick]), R.decode(want_c, want_s, "e4m3"))
    G.gift_layernorm_forward(ctx(), x, None, None, 1e-5, y, rstd=rstd, codes=codes, scales=scales)
    wy = R.norm_forward(host(x[pick]), None, None, 1e-5)[0]
    assert np.abs(host(y[pick]) - wy).max() <= R.U16 * 1.01 * np.abs(wy).max()
    delta = torch.randint(-3, 4, (T, d_out), generator=gen, device=DEV).to(torch.bfloat16)
    dW, db = weight_grad(delta, codes, scales, "e4m3", d)
    cols = [0, 127, 30000, 65535]
    v = R.decode(c2[:, cols].cpu().numpy(), np.zeros((T, 1), np.uint8) + 127, "e4m3") * \
        np.ldexp(1.0, s2[:, [c // 128 for c in cols]].cpu().numpy().astype(int) - 127)
    want, wb = R.weight_grad(host(delta), v)
    assert np.array_equal(host(db), wb)
    assert np.linalg.norm(host(dW)[:, cols] - want) <= (32 + T / 256) * R.U32 * 1.3 * np.linalg.norm(want)
    dx, ws = x, torch.empty(G.gift_act_workspace_bytes(ctx(), "layernorm_backward", torch.bfloat16, T, d, d),
                            dtype=torch.uint8, device=DEV)
    dg = torch.empty(d, device=DEV)
    G.gift_layernorm_backward(ctx(), y, codes, None, rstd, dx, dg, scales=scales, ws=ws)
    n = R.decode(c2[pick].cpu().numpy(), s2[pick].cpu().numpy(), "e4m3")
    wx = R.norm_backward(host(y[pick]), n, None, host(rstd[pick]))[0]
    assert np.abs(host(dx[pick]) - wx).max() <= R.U16 * 1.01 * np.abs(wx).max()


# ---- refusals ------------------------------------------------------------------------------------
def _refused(call):
    with pytest.raises(G.GiftError) as e:
        call()
    assert e.value.status == G.ERR_INVALID_ARG


def test_refusals():
    c, L = ctx(), G.lib()
    x = torch.zeros(4, 256, device=DEV)
    codes, scales = torch.zeros(4, 256, dtype=torch.uint8, device=DEV), torch.zeros(4, 2, dtype=torch.uint8, device=DEV)
    v, m = torch.zeros(256, device=DEV), torch.zeros(4, device=DEV)
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)
    y = torch.zeros_like(x)
    for fmt in ("f32", "nvfp4"):
        _refused(lambda: G.gift_act_sizes(fmt, 4, 256))
        _refused(lambda: G.gift_act_encode(c, x, fmt, codes, scales))
        _refused(lambda: G.gift_act_decode(c, codes, scales, fmt, y))
        _refused(lambda: G.gift_layernorm_forward(c, x, v, v, 1e-5, y, fmt=fmt, codes=codes, scales=scales))
        _refused(lambda: G.gift_layernorm_backward(c, x, codes, v, m, y, v, v, scales=scales, fmt=fmt, ws=ws))
        _refused(lambda: G.gift_weight_grad(c, x, codes, scales, fmt, torch.zeros(256, 256, device=DEV), ws=ws))
    for T, d in ((0, 256), (4, 0), (-1, 256), (2 ** 30 + 1, 1)):
        _refused(lambda: G.gift_act_sizes("e4m3", T, d))
        assert L.gift_act_encode(c.handle, 4096, 0, T, d, 1, 4096, 4096, None, None) == G.ERR_INVALID_ARG
        assert L.gift_act_decode(c.handle, 4096, 4096, 1, T, d, 4096, 0, None, None) == G.ERR_INVALID_ARG
        assert L.gift_layernorm_forward(c.handle, 4096, 0, T, d, None, None, 1e-5, 4096, None, None, 1, None, None,
                                        None, None) == G.ERR_INVALID_ARG
        assert L.gift_layernorm_backward(c.handle, 4096, 0, T, d, 4096, 1, 4096, 1, None, 4096, None, 4096, None,
                                         None, None, 0, None, None) == G.ERR_INVALID_ARG
        assert L.gift_weight_grad(c.handle, 4096, 0, 4096, 4096, 1, T, 4, d, None, None, 4096, None, 4096, 1 << 40,
                                  None, None) == G.ERR_INVALID_ARG
    assert L.gift_act_encode(c.handle, 4096, 2, 4, 256, 1, 4096, 4096, None, None) == G.ERR_INVALID_ARG   # a bad type
    for eps in (-1e-5, float("nan"), float("inf")):
        _refused(lambda: G.gift_layernorm_forward(c, x, v, v, eps, y))
    _refused(lambda: G.gift_layernorm_forward(c, x, v, v, 1e-5, y, codes=codes))
    _refused(lambda: G.gift_layernorm_forward(c, x, v, v, 1e-5, None))
    _refused(lambda: G.gift_layernorm_backward(c, x, x, v, m, y, v, v, ws=ws))              # x without its mean
    _refused(lambda: G.gift_layernorm_backward(c, x, x, v, None, y, v, v, mean=m, ws=ws))   # no rstd
    _refused(lambda: G.gift_layernorm_backward(c, x, x, v, m, y, v, v, mean=m))             # sums without a workspace
    _refused(lambda: G.gift_layernorm_backward(c, x, x, v, m, y, v, None, mean=m, ws=ws[:256]))
    dW = torch.zeros(256, 256, device=DEV)
    _refused(lambda: G.gift_weight_grad(c, x, codes, scales, "e4m3", dW))
    _refused(lambda: G.gift_weight_grad(c, x, codes, scales, "e4m3", dW, ws=ws[:64]))
    _refused(lambda: G.gift_act_workspace_bytes(c, "encode", torch.float32, 4, 8, 8))
    _refused(lambda: G.gift_act_workspace_bytes(c, "weight_grad", torch.float32, 4, 0, 8))
    torch.cuda.synchronize()


def test_binding_refuses_wrong_buffers():
    c = ctx()
    x = torch.zeros(4, 256, device=DEV)
    codes, scales = torch.zeros(4, 256, dtype=torch.uint8, device=DEV), torch.zeros(4, 2, dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError):
        G.gift_act_encode(c, x.half(), "e4m3", codes, scales)
    with pytest.raises(ValueError):
        G.gift_act_encode(c, x, "e4m3", codes, scales[:2])
    with pytest.raises(ValueError):
        G.gift_act_encode(c, x.t(), "e4m3", codes, scales.new_zeros(1024))
    with pytest.raises(ValueError):
        G.gift_act_encode(c, x.cpu(), "e4m3", codes, scales)
    with pytest.raises(ValueError):
        G.gift_layernorm_forward(c, x, torch.zeros(255, device=DEV), None, 1e-5, torch.zeros_like(x))
    with pytest.raises(ValueError):
        G.gift_layernorm_forward(c, x, None, None, 1e-5, x.bfloat16())
    with pytest.raises(ValueError):
        G.gift_weight_grad(c, x, codes, scales, "e4m3", torch.zeros(256, 300, device=DEV), ws=codes)
