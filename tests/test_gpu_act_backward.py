"""Layer norm's backward pass by every plan, with more rows than are resident at once and more than one slice of
tokens: every number of pieces and of warps per row, both accesses, from the input and from the checkpoint; on
a share of the GPU; past 32-bit offsets; from several threads.  Tolerances as in test_gpu_act.py.
"""
import threading

import numpy as np
import pytest
import torch

import act_ref as R
from fac_whitening_gb300 import gift as G
from gpu_util import DEV, ctx, status
from test_gpu_act import DT, backward, check_backward, dev, forward, host, norm_inputs, rows, unaligned, weight_grad

pytestmark = pytest.mark.gpu

# pieces of 512 columns: 1, 2, 3 (15 warps a CTA), 5, 6, 7, 8, one row a CTA from 9 on, 16; two and four pieces a
# lane; rows that are read again.  Odd widths go by elements, 256 columns a warp up to 4096
PLANS = [(9000, 96), (5000, 528), (3000, 1536), (900, 2064), (800, 2576), (700, 3584), (640, 3600), (400, 4112),
         (330, 5120), (300, 6160), (250, 8192), (200, 8208), (320, 10000), (170, 16384), (170, 16400), (60, 32768),
         (40, 40000), (5000, 129), (3001, 1361), (900, 2731), (700, 4095), (400, 5003), (200, 9001), (160, 17001)]


def _case(T, d, dt, saved, off):
    x, gamma, _ = norm_inputs(T, d, dt, 3 * T + d)
    dy = rows(T, d, dt, 79 + T + d)
    xs = x.double().numpy()
    _, n, mean, rstd = R.norm_forward(xs, None, None, 1e-5)
    mean, rstd = mean.astype(np.float32), rstd.astype(np.float32)
    put = unaligned if off else (lambda t: t)
    if saved == "input":
        n = (xs - mean[:, None].astype(np.float64)) * rstd[:, None].astype(np.float64)
        args = dict(saved=put(x.to(DEV)), mean=dev(mean))
        n_err = 3 * R.U32 * np.abs(n)
    else:
        codes, scales = R.encode(n.astype(np.float32), saved)
        n, n_err = R.decode(codes, scales, saved), 0.0
        args = dict(saved=put(dev(codes, torch.uint8)), scales=put(dev(scales, torch.uint8)), fmt=saved)
    call = lambda: backward(put(dy.to(DEV)), gamma=gamma, rstd=dev(rstd), off=off, **args)  # noqa: E731
    return call, (T, d, dt, dy.double().numpy(), n, n_err, gamma, rstd.astype(np.float64))


@pytest.mark.parametrize("off", [False, True], ids=["aligned", "unaligned"])
@pytest.mark.parametrize("saved", ["input", "e4m3"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", PLANS, ids=str)
def test_norm_backward_of_many_rows(shape, dt, saved, off):
    call, want = _case(*shape, dt, saved, off)
    got = call()
    check_backward(*want, got)
    for a, b in zip(got[:3], call()[:3]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("sms", [1, 7, 38])
@pytest.mark.parametrize("shape", [(515, 272), (300, 8208), (50, 40000)], ids=str)
def test_norm_passes_of_a_share_of_the_gpu(shape, sms):
    c = G.Context(torch.cuda.current_device())
    G.gift_set_option(c, G.OPT_SMS, sms)
    T, d = shape
    x, gamma, beta = norm_inputs(T, d, "bf16", sms)
    dy, st = rows(T, d, "bf16", 5), status()
    xd, g = x.to(DEV), dev(gamma)
    y, dx = torch.empty_like(xd), torch.empty_like(xd)
    mean, rstd, dg, db = (torch.empty(n, device=DEV) for n in (T, T, d, d))
    G.gift_layernorm_forward(c, xd, g, dev(beta), 1e-5, y, mean=mean, rstd=rstd, status=st)
    assert torch.equal(y, forward(xd, gamma, beta, 1e-5)[0])   # a row's sums do not depend on the grid
    ws = torch.empty(G.gift_act_workspace_bytes(c, "layernorm_backward", torch.bfloat16, T, d, d), dtype=torch.uint8,
                     device=DEV)
    ws.fill_(0xFF)
    G.gift_layernorm_backward(c, dy.to(DEV), xd, g, rstd, dx, dg, db, mean=mean, ws=ws, status=st)
    n = (x.double().numpy() - host(mean)[:, None]) * host(rstd)[:, None]
    check_backward(T, d, "bf16", dy.double().numpy(), n, 3 * R.U32 * np.abs(n), gamma, host(rstd),
                   (dx, dg, db, int(st.item())))


@pytest.mark.parametrize("shape", [(2900000, 1536), (530000, 8208), (110000, 40000)], ids=str)
def test_norm_backward_past_32_bits(shape):
    # 4.4 G elements from a checkpoint of E4M3 codes with scales 2^-4..2^-1
    T, d = shape
    gen = torch.Generator(device=DEV).manual_seed(2)
    dy, codes = torch.empty(T, d, dtype=torch.bfloat16, device=DEV), torch.empty(T, d, dtype=torch.uint8, device=DEV)
    groups = -(-d // 128)
    scales = torch.randint(123, 127, (T, groups), generator=gen, device=DEV, dtype=torch.uint8)
    step = 1 + (1 << 27) // d
    for t in range(0, T, step):
        dy[t:t + step].normal_(generator=gen)
        part = torch.randint(0, 72, codes[t:t + step].shape, generator=gen, device=DEV, dtype=torch.uint8)   # up to 4
        codes[t:t + step] = part + 128 * (torch.rand(part.shape, generator=gen, device=DEV) < 0.5).to(torch.uint8)
    rstd = 0.5 + torch.rand(T, generator=gen, device=DEV)
    dx, dg, db, st = backward(dy, codes, None, rstd, scales=scales)
    assert st == 0
    pick = [0, 1, T // 2, T - 2, T - 1]
    value = lambda c, s: R.decode(c.cpu().numpy(), s.cpu().numpy(), "e4m3")  # noqa: E731
    n, h, r = value(codes[pick], scales[pick]), host(dy[pick]), host(rstd[pick])[:, None]
    wx = R.norm_backward(h, n, None, r[:, 0])[0]
    ma, mb = np.abs(h).mean(axis=1, keepdims=True), np.abs(h * n).mean(axis=1, keepdims=True)
    N = d + 8
    tol = r * (8 * R.U32 * (np.abs(h) + ma + np.abs(n) * mb) + N * R.U32 * (ma + np.abs(n) * mb))
    assert np.all(np.abs(host(dx[pick]) - wx) <= tol + R.U16 * (np.abs(wx) + tol))
    for c in (0, 127, d // 2, d - 1):
        col = value(codes[:, c:c + 1].contiguous(), scales[:, c // 128:c // 128 + 1].contiguous())[:, 0]
        g = host(dy[:, c].contiguous())
        # any order stays below (T + 4) u of the sum of sizes.  With random signs the m <= 5000 additions of a partial
        # sum err by u sqrt(m / 2) of the terms' root sum of squares, 3e-6; 1e-4 is far above it
        assert abs(dg[c].item() - (g * col).sum()) <= (T + 4) * R.U32 * np.abs(g * col).sum()
        assert abs(dg[c].item() - (g * col).sum()) <= 1e-4 * np.linalg.norm(g * col)
        assert abs(db[c].item() - g.sum()) <= 1e-4 * np.linalg.norm(g)


def test_calls_from_several_threads():
    # each thread its own stream and widths (CTAs of other sizes of the same kernels), on one context
    work = [[(300, 1536), (200, 4096), (90, 520)], [(200, 3584), (300, 1536), (64, 8208)], [(120, 2576), (333, 272), (90, 1361)],
            [(100, 2064), (50, 16400), (300, 1536)]]

    def passes(shapes):
        out = []
        for T, d in shapes:
            x, gamma, beta = norm_inputs(T, d, "bf16", T)
            y, mean, rstd, codes, scales, _ = forward(x.to(DEV), gamma, beta, 1e-5, "e4m3")
            dx, dg, db, st = backward(y, codes, gamma, rstd, scales=scales)
            delta = rows(T, 136, "bf16", d).to(DEV)
            dW, bias = weight_grad(delta, codes, scales, "e4m3", d, gamma, beta)
            assert st == 0
            out += [y, mean, rstd, codes, scales, dx, dg, db, dW, bias]
        torch.cuda.current_stream().synchronize()
        return out

    ctx()
    got, errors = [None] * len(work), []

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(3):
                    got[i] = passes(work[i])
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for i, shapes in enumerate(work):
        for a, b in zip(passes(shapes), got[i]):
            assert torch.equal(a, b)
