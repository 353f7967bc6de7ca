"""How the feed-forward calls are used: graphs, streams, threads, shares of the GPU, refusals, values that are not finite,
tensors past 32-bit offsets, and a block's training step from end to end."""
import ctypes
import threading

import numpy as np
import pytest
import torch

import act_ref as A
import mlp_ref as R
from fac_whitening_gb300 import gift as G
from gpu_util import DEV, ctx, status
from test_gpu_mlp import (DT, gated_backward, gated_forward, host, input_grad, linear, normal, rng_of, rounded,
                          workspace)

pytestmark = pytest.mark.gpu


class Block:
    """One block's buffers and its calls, forward and backward, as a training program makes them."""

    def __init__(self, T, d, f, dt, p=0.25, seed=0, fn="silu", c=None):
        g = torch.Generator(device=DEV).manual_seed(seed)
        r = lambda *s: torch.randn(*s, device=DEV, generator=g)  # noqa: E731
        t = lambda *s: torch.empty(*s, dtype=DT[dt], device=DEV)  # noqa: E731
        e = lambda *s: torch.empty(*s, device=DEV)  # noqa: E731
        self.c, self.p, self.fn, self.site, self.st = c or ctx(), p, fn, 9, status()
        self.T, self.d, self.f, self.dt = T, d, f, dt
        self.x, self.dy = r(T, d).to(DT[dt]), r(T, d).to(DT[dt])
        self.gamma, self.beta = 1 + 0.1 * r(d), 0.1 * r(d)
        self.Wg, self.Wu, self.W = ((r(*s) / s[1] ** 0.5).to(DT[dt]) for s in ((f, d), (f, d), (d, f)))
        self.bg, self.bu, self.b = 0.1 * r(f), 0.1 * r(f), 0.1 * r(d)
        self.rng = rng_of(seed + 77, 3)
        kept = lambda n: tuple(torch.empty(k, dtype=torch.uint8, device=DEV) for k in G.gift_act_sizes("e4m3", T, n))  # noqa: E731,E501
        self.n_kept, self.h_kept, self.rstd = kept(d), kept(f), e(T)
        self.n, self.h, self.gate, self.up, self.y = t(T, d), t(T, f), t(T, f), t(T, f), t(T, d)
        self.dz, self.dg, self.du, self.dn, self.dx = t(T, d), t(T, f), t(T, f), t(T, d), t(T, d)
        self.dW, self.dWg, self.dWu, self.db, self.dbg, self.dbu = e(d, f), e(f, d), e(f, d), e(d), e(f), e(f)
        self.dgamma, self.dbeta = e(d), e(d)
        ops = (("gated_forward", f, d), ("linear_forward", d, f), ("dropout_backward", d, d), ("weight_grad", d, f),
               ("weight_grad", f, d), ("gated_backward", d, f), ("input_grad", f, d), ("layernorm_backward", d, d))
        self.ws = torch.empty(max(G.gift_act_workspace_bytes(self.c, o, DT[dt], T, a, b) for o, a, b in ops),
                              dtype=torch.uint8, device=DEV)

    def forward(self):
        c, k, s = self.c, dict(ws=self.ws, status=self.st), self.st
        G.gift_layernorm_forward(c, self.x, self.gamma, self.beta, 1e-5, self.n, rstd=self.rstd,
                                 codes=self.n_kept[0], scales=self.n_kept[1], status=s)
        G.gift_gated_forward(c, self.n, self.Wg, self.Wu, self.fn, self.h, gate=self.gate, up=self.up, bg=self.bg,
                             bu=self.bu, codes=self.h_kept[0], scales=self.h_kept[1], **k)
        G.gift_linear_forward(c, self.h, self.W, self.y, bias=self.b, residual=self.x, p=self.p, rng=self.rng,
                              site=self.site, **k)

    def backward(self):
        c, k = self.c, dict(ws=self.ws, status=self.st)
        G.gift_dropout_backward(c, self.dy, self.dz, self.p, self.rng, self.site, self.db, ws=self.ws)
        G.gift_weight_grad(c, self.dz, *self.h_kept, "e4m3", self.dW, **k)
        G.gift_gated_backward(c, self.dz, self.W, self.gate, self.up, self.fn, self.dg, self.du, **k)
        G.gift_weight_grad(c, self.dg, *self.n_kept, "e4m3", self.dWg, db=self.dbg, gamma=self.gamma, beta=self.beta, **k)
        G.gift_weight_grad(c, self.du, *self.n_kept, "e4m3", self.dWu, db=self.dbu, gamma=self.gamma, beta=self.beta, **k)
        G.gift_input_grad(c, self.dg, self.Wg, self.dn, delta2=self.du, W2=self.Wu, **k)
        G.gift_layernorm_backward(c, self.dn, self.n_kept[0], self.gamma, self.rstd, self.dx, self.dgamma, self.dbeta,
                                  scales=self.n_kept[1], **k)

    def results(self):
        return [self.y, self.dx, self.dW, self.dWg, self.dWu, self.db, self.dbg, self.dbu, self.dgamma, self.dbeta]

    def step(self):
        self.forward()
        self.backward()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 16, 48), (130, 96, 272), (67, 129, 257)], ids=str)
def test_a_training_step_follows_the_formulas(shape, dt):
    """Every result of the chain from the values its call was given."""
    T, d, f = shape
    b = Block(T, d, f, dt)
    b.step()
    assert int(b.st.item()) == 0
    x, n, h, gate, up, dz, dg, du, dn = (host(t) for t in (b.x, b.n, b.h, b.gate, b.up, b.dz, b.dg, b.du, b.dn))
    Wg, Wu, W = host(b.Wg), host(b.Wu), host(b.W)
    drop = lambda v: R.drop(v, b.p, 77, 3, b.site)  # noqa: E731
    half, u = R.half_step, R.U32
    g64, eg = R.product(n, Wg.T, dt)
    assert (np.abs(gate - g64 - host(b.bg)) <= eg + 1.01 * half(g64 + host(b.bg), dt) + 4 * u * np.abs(g64)).all()
    z64, ez = R.product(h, W.T, dt)
    want = x + drop(z64 + host(b.b))
    assert (np.abs(host(b.y) - want) <= 1.4 * ez + 8 * u * (np.abs(z64) + np.abs(want)) + 1.01 * half(want, dt)).all()
    want = drop(host(b.dy))
    assert (np.abs(dz - want) <= u * np.abs(want) + 1.01 * half(want, dt)).all()
    hv = A.decode(b.h_kept[0].cpu().numpy().reshape(T, f), b.h_kept[1].cpu().numpy().reshape(T, -1), "e4m3")
    nv = A.decode(b.n_kept[0].cpu().numpy().reshape(T, d), b.n_kept[1].cpu().numpy().reshape(T, -1), "e4m3")
    # the checkpoint's rounding: half a step of four significant bits, and the smallest codes' steps
    assert (np.abs(hv - h) <= 2.0 ** -4 * 1.01 * np.abs(h) + 1.01 * half(h, dt) +
            2.0 ** -16 * np.abs(h).max(1, keepdims=True)).all()
    dh, e = R.product(dz, W, dt)
    a, slope = R.gate(gate, b.fn)
    ge = R.gate_error(gate, b.fn)
    es = ge * (np.abs(slope) + 2.0 * np.abs(a) + 1.0) * 1.5
    want = dh * up * slope
    assert (np.abs(dg - want) <= np.abs(up) * (e * (np.abs(slope) + es) + np.abs(dh) * es) + 4 * u * np.abs(want) +
            1.01 * half(want, dt)).all()
    for got, delta, v, gb in ((b.dW, dz, hv, None), (b.dWg, dg, nv, 1), (b.dWu, du, nv, 1)):
        gam, bet = (None, None) if gb is None else (host(b.gamma), host(b.beta))
        want, _ = A.weight_grad(delta, v, gam, bet)
        size, _ = A.weight_grad(np.abs(delta), np.abs(v), None if gam is None else np.abs(gam),
                                None if bet is None else np.abs(bet))
        assert (np.abs(host(got) - want) <= (2 * T + 8) * u * size + 1e-37).all()
    want, e = R.product(np.hstack([dg, du]), np.vstack([Wg, Wu]), dt)
    assert (np.abs(dn - want) <= e + 1.01 * half(want, dt)).all()
    dx, dgamma, dbeta = A.norm_backward(dn, nv, host(b.gamma), host(b.rstd))
    scale = np.abs(host(b.rstd))[:, None] * np.abs(dn * host(b.gamma)).max(1, keepdims=True) * (1 + np.abs(nv))
    assert (np.abs(host(b.dx) - dx) <= (d + 16) * u * scale * 4 + 1.01 * half(dx, dt)).all()


def test_gradients_against_differences():
    """The loss sum(y dy) along random directions, FP32, whose differences are taken in 64 bits; the checkpoints (4
    significant bits) stand for n and h in the weight gradients only, so those are compared through the values kept."""
    T, d, f = 40, 48, 64
    b = Block(T, d, f, "f32", p=0.25)
    b.step()
    assert int(b.st.item()) == 0
    n, dy = host(b.n), host(b.dy)
    P = {k: host(getattr(b, k)) for k in ("Wg", "Wu", "W", "bg", "bu", "b")}

    def loss(n, q):
        g, u = n @ q["Wg"].T + q["bg"], n @ q["Wu"].T + q["bu"]
        h = R.gate(g, b.fn)[0] * u
        return (R.drop(h @ q["W"].T + q["b"], b.p, 77, 3, b.site) * dy).sum()

    rng = np.random.default_rng(1)
    eps = 1e-6
    grads = {"n": host(b.dn), "bg": host(b.dbg), "bu": host(b.dbu), "b": host(b.db)}
    for name, grad in grads.items():
        v = rng.standard_normal(grad.shape)
        if name == "n":
            diff = (loss(n + eps * v, P) - loss(n - eps * v, P)) / (2 * eps)
        else:
            up, down = dict(P, **{name: P[name] + eps * v}), dict(P, **{name: P[name] - eps * v})
            diff = (loss(n, up) - loss(n, down)) / (2 * eps)
        # FP32 sums of at most T f terms along the chain; the differences' own error is below 1e-8 of the loss's scale
        assert abs(diff - (grad * v).sum()) <= 2e-5 * np.abs(grad * v).sum(), name


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(130, 96, 272), (24, 1536, 200), (67, 129, 257)], ids=str)
def test_equal_calls_give_equal_bits_and_graphs_read_new_steps(shape, dt):
    b = Block(*shape, dt)
    b.step()
    first = [t.clone() for t in b.results()]
    b.step()
    assert all(torch.equal(x, y) for x, y in zip(first, b.results()))
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        b.step()
    for t in b.results():
        t.zero_()
    graph.replay()
    assert all(torch.equal(x, y) for x, y in zip(first, b.results()))
    b.rng[1] += 1   # the next step: other bits, from the same graph
    graph.replay()
    second = [t.clone() for t in b.results()]
    assert not torch.equal(first[0], second[0])
    b.step()
    assert all(torch.equal(x, y) for x, y in zip(second, b.results()))
    assert int(b.st.item()) == 0


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_a_workspace_may_start_anywhere(dt):
    b = Block(67, 129, 257, dt)
    b.step()
    want = [t.clone() for t in b.results()]
    flat = torch.full((b.ws.numel() + 8,), 0xFF, dtype=torch.uint8, device=DEV)
    b.ws = flat[3:3 + b.ws.numel()]
    b.step()
    assert all(torch.equal(x, y) for x, y in zip(want, b.results()))
    assert (flat[:3] == 0xFF).all() and (flat[3 + b.ws.numel():] == 0xFF).all()


def test_two_graphs_share_a_workspace_one_after_the_other():
    a, b = Block(130, 96, 272, "f32", seed=1), Block(67, 129, 257, "f32", seed=2)
    want = []
    for k in (a, b):
        k.step()
        want.append([t.clone() for t in k.results()])
    shared = a.ws if a.ws.numel() > b.ws.numel() else b.ws
    graphs = []
    torch.cuda.synchronize()
    for k in (a, b):
        k.ws = shared
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=torch.cuda.Stream()):
            k.step()
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    for k, w in zip((a, b), want):
        assert all(torch.equal(x, y) for x, y in zip(w, k.results()))


def test_streams_and_threads_side_by_side():
    blocks = [Block(130 + 31 * i, 96, 272, ("f32", "bf16")[i % 2], seed=i) for i in range(4)]
    want = []
    for b in blocks:
        b.step()
        want.append([t.clone() for t in b.results()])
    torch.cuda.synchronize()
    streams, errors = [torch.cuda.Stream() for _ in blocks], []

    def work(b, s):
        try:
            with torch.cuda.stream(s):
                for _ in range(10):
                    b.step()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=p) for p in zip(blocks, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for b, w in zip(blocks, want):
        assert int(b.st.item()) == 0 and all(torch.equal(x, y) for x, y in zip(w, b.results()))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("sms", [1, 2, 7, 40])
def test_on_a_share_of_the_gpu(sms, dt):
    """Whole numbers: every plan of tiles and slices gives the same exact products."""
    c = G.Context(torch.cuda.current_device())
    G.gift_set_option(c, G.OPT_SMS, sms)
    rng = np.random.default_rng(sms)
    for T, k, n in ((600, 130, 700), (3, 2000, 264), (1000, 64, 65)):
        x, W = rng.integers(-3, 4, (T, k)).astype(float), rng.integers(-1, 2, (n, k)).astype(float)
        V = np.ascontiguousarray(W.T)
        want = rounded(x @ V, dt)
        assert np.array_equal(linear(x, W, dt, c=c), want)
        assert np.array_equal(input_grad(x, V, dt, c=c), want)
        out = gated_forward(x, W, -W, "silu", dt, c=c)
        assert np.array_equal(out["gate"], want) and np.array_equal(out["up"], -want)
        dg, _ = gated_backward(x, V, np.zeros((T, n)), np.full((T, n), 2.0), "silu", dt, c=c)
        assert np.array_equal(dg, want)


@pytest.mark.parametrize("off", [False, True], ids=["aligned", "unaligned"])
def test_what_is_not_finite_stays_in_its_row(off):
    rng = np.random.default_rng(5)
    T, k, n = 300, 200, 272
    x, W = normal(rng, T, k, dt="bf16"), normal(rng, n, k, dt="bf16") / 8
    clean = gated_forward(x, W, W, "gelu", "bf16", fmt="e4m3", off=off)
    bad = x.copy()
    bad[7, 3], bad[200, 0], bad[299, 199] = np.nan, np.inf, -np.inf
    out = gated_forward(bad, W, W, "gelu", "bf16", fmt="e4m3", off=off)
    assert clean["status"] == 0 and out["status"] == G.ERR_NONFINITE
    rows = np.isin(np.arange(T), [7, 200, 299])
    for key in ("h", "gate", "up", "codes", "scales"):
        assert np.array_equal(out[key][~rows], clean[key][~rows]), key
    assert np.isnan(out["gate"][7]).all() and not np.isfinite(out["gate"][[200, 299]]).any()
    assert (out["scales"][rows] == 255).all()
    # dropped elements are the residual, whatever was dropped
    res = normal(rng, T, n, dt="bf16")
    y = linear(bad, W, "bf16", residual=res, p=0.5, rng=rng_of(1, 2), site=3, off=off)
    dropped = ~R.keep(T, n, 0.5, 1, 2, 3)
    assert np.array_equal(y[dropped], res[dropped])
    assert not np.isfinite(y[rows][~dropped[rows]]).any()
    nan = torch.full((4, 64), float("nan"), device=DEV)
    y = torch.empty_like(nan)
    G.gift_dropout_forward(ctx(), nan, y, 0.5, rng_of(1, 2), 3)
    keep = R.keep(4, 64, 0.5, 1, 2, 3)
    assert np.array_equal(np.isnan(host(y)), keep) and (host(y)[~keep] == 0).all()


def test_fp32_extremes():
    """FP32's largest values and powers of two far apart: exact as long as the sums are."""
    big = float(np.finfo(np.float32).max)
    x = np.zeros((4, 64))
    x[0, 0], x[1, 1], x[2, 2], x[3, 3] = big, -big, 2.0 ** 100, 1.5 * 2.0 ** -60
    W = np.zeros((16, 64))
    W[0, :4] = [1.0, 1.0, 2.0 ** -90, 2.0 ** 50]
    W[1, :4] = [-0.5, 0.5, 2.0 ** 20, 1.0]
    assert np.array_equal(linear(x, W, "f32"), x @ W.T)
    assert np.array_equal(input_grad(x, np.ascontiguousarray(W.T), "f32"), x @ W.T)


@pytest.mark.parametrize("off", [False, True], ids=["aligned", "unaligned"])
def test_offsets_past_32_bits(off):
    """Outputs of more than 2^32 elements: the last rows."""
    T, N, K = (1 << 17) + 70, (1 << 15) + 16, 16
    x, W = torch.ones(T, K, dtype=torch.bfloat16, device=DEV), torch.ones(N, K, dtype=torch.bfloat16, device=DEV)
    x[-1] = 3
    n = T * N + 1
    flat = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    y = (flat[1:] if off else flat[:-1]).view(T, N)
    st = status()
    G.gift_linear_forward(ctx(), x, W, y, ws=workspace("linear_forward", "bf16", T, N, K), status=st)
    assert int(st.item()) == 0
    assert (y[:2] == 16).all() and (y[-300:-1] == 16).all() and (y[-1] == 48).all()
    rng = rng_of(3, 4)
    G.gift_dropout_forward(ctx(), y, y, 0.5, rng, 1)   # in place
    rows = np.arange(T - 40, T)
    keep = R.keep(T, N, 0.5, 3, 4, 1, rows=rows)
    want = np.where(keep, 32.0, 0.0)
    want[-1] *= 3
    assert np.array_equal(host(y[-40:]), want)


def test_refusals():
    c = ctx()
    T, d, f = 8, 16, 32
    z = lambda *s: torch.zeros(*s, device=DEV)  # noqa: E731
    x, Wg, h, y, W, rng = z(T, d), z(f, d), z(T, f), z(T, d), z(d, f), rng_of(0, 0)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    lib, null, f32, e4m3 = G.lib(), None, 0, 1
    p = lambda t: ctypes.c_void_p(t.data_ptr()) if t is not None else None  # noqa: E731
    n = ws.numel()

    def fwd(x=x, Wg=Wg, Wu=Wg, T=T, d=d, f=f, dt=f32, fn=0, h=h, g=null, u=null, fmt=e4m3, co=null, sc=null, ws=ws, n=n):
        return lib.gift_gated_forward(c.handle, p(x), dt, T, d, p(Wg), p(Wu), f, null, null, fn, p(h), p(g), p(u), fmt,
                                      p(co), p(sc), p(ws), n, null, null)

    def bwd(dy=x, W=W, g=h, u=h, dg=h, du=h, T=T, d=d, f=f, dt=f32, fn=0, ws=ws, n=n):
        return lib.gift_gated_backward(c.handle, p(dy), dt, T, d, p(W), f, p(g), p(u), fn, p(dg), p(du), p(ws), n, null,
                                       null)

    def lin(x=h, W=W, y=y, T=T, k=f, o=d, dt=f32, q=0.0, r=rng, ws=ws, n=n):
        return lib.gift_linear_forward(c.handle, p(x), dt, T, k, p(W), o, null, null, q, p(r), 0, p(y), p(ws), n, null,
                                       null)

    def inp(a=x, W=W, a2=null, W2=null, dx=h, T=T, o=d, k=f, dt=f32, ws=ws, n=n):
        return lib.gift_input_grad(c.handle, p(a), p(W), p(a2), p(W2), dt, T, o, k, p(dx), p(ws), n, null, null)

    def dro(x=x, y=y, T=T, d=d, dt=f32, q=0.5, r=rng):
        return lib.gift_dropout_forward(c.handle, p(x), dt, T, d, null, null, q, p(r), 0, p(y), null)

    def drb(dy=x, dx=y, T=T, d=d, dt=f32, q=0.5, r=rng, db=null, ws=null, n=0):
        return lib.gift_dropout_backward(c.handle, p(dy), dt, T, d, q, p(r), 0, p(dx), p(db), p(ws), n, null)

    for call in (fwd, bwd, lin, inp, dro, drb):
        assert call() == G.OK
    assert lin(r=null) == G.OK and dro(q=0.0, r=null) == G.OK and dro(q=2.0 ** -18, r=null) == G.OK
    refused = [fwd(x=null), fwd(Wg=null), fwd(Wu=null), fwd(h=null), fwd(ws=null), fwd(T=0), fwd(d=0), fwd(f=0),
               fwd(dt=2), fwd(fn=3), fwd(fn=-1), fwd(g=h), fwd(u=h), fwd(co=ws), fwd(sc=ws), fwd(co=ws, sc=ws, fmt=0),
               fwd(co=ws, sc=ws, fmt=3), fwd(n=256), fwd(T=(1 << 30) + 1),
               bwd(dy=null), bwd(W=null), bwd(g=null), bwd(u=null), bwd(dg=null), bwd(du=null), bwd(ws=null), bwd(T=0),
               bwd(d=0), bwd(f=0), bwd(dt=-1), bwd(fn=3), bwd(n=0),
               lin(x=null), lin(W=null), lin(y=null), lin(ws=null), lin(T=0), lin(k=0), lin(o=0), lin(dt=5), lin(q=-0.1),
               lin(q=1.0), lin(q=float("nan")), lin(q=1 - 2.0 ** -18), lin(q=0.5, r=null), lin(n=1),
               lin(T=1 << 30, o=1 << 30),
               inp(a=null), inp(W=null), inp(a2=x), inp(W2=W), inp(dx=null), inp(ws=null), inp(T=-1), inp(o=0), inp(k=0),
               inp(dt=2), inp(n=1),
               dro(x=null), dro(y=null), dro(T=0), dro(d=0), dro(dt=2), dro(q=1.5), dro(q=-1.0), dro(r=null),
               drb(dy=null), drb(dx=null), drb(T=0), drb(d=0), drb(dt=2), drb(q=float("inf")), drb(r=null), drb(db=y),
               drb(db=y, ws=ws, n=1)]
    assert all(s == G.ERR_INVALID_ARG for s in refused), refused
    for op in ("gated_forward", "gated_backward", "linear_forward", "input_grad"):
        with pytest.raises(G.GiftError):
            G.gift_act_workspace_bytes(c, op, torch.float32, 8, 0, 8)
    assert G.gift_act_workspace_bytes(c, "dropout_backward", torch.float32, 8, 0, 8) > 0
    with pytest.raises(ValueError):
        G.gift_linear_forward(c, x.half(), W.half(), y.half(), ws=ws)
    with pytest.raises(ValueError):
        G.gift_input_grad(c, x, W[:, ::2], h, ws=ws)
    torch.cuda.synchronize()
