"""Plain 64-bit statements of the 8-bit activation checkpoint, the layer norm and the weight
gradient (numpy), for the tests."""
import numpy as np

GROUP = 128
EMAX = {"e4m3": 8, "e5m2": 15}
U32 = 2.0 ** -24   # unit roundoff of FP32
U16 = 2.0 ** -8    # unit roundoff of BF16 (8 significant bits)


def magnitudes(fmt):
    """The finite non-negative values of a format by code."""
    mbits, bias, last = (3, 7, 126) if fmt == "e4m3" else (2, 15, 123)
    out = []
    for c in range(last + 1):
        e, m = c >> mbits, (c & ((1 << mbits) - 1)) / (1 << mbits)
        out.append(m * 2.0 ** (1 - bias) if e == 0 else (1 + m) * 2.0 ** (e - bias))
    return np.array(out)


def scale_bytes(x, fmt):
    """k + 127 per token and group: the smallest k with amax <= FMAX 2^k, clamped; 255 for NaN/Inf."""
    T, d = x.shape
    out = np.zeros((T, -(-d // GROUP)), dtype=np.uint8)
    fmax, kmax = magnitudes(fmt)[-1], 127 - EMAX[fmt]
    pows = np.array([np.ldexp(fmax, k) for k in range(-110, kmax + 1)])
    for g in range(out.shape[1]):
        a = np.abs(x[:, g * GROUP:(g + 1) * GROUP]).max(axis=1)   # NaN propagates
        k = np.minimum(np.searchsorted(pows, a, side="left"), len(pows) - 1) - 110
        out[:, g] = np.where(np.isfinite(a), k + 127, 255)
    return out


def _per_element(scales, d):
    return np.repeat(scales.astype(np.int64) - 127, GROUP, axis=1)[:, :d]


def codes_of(x, scales, fmt):
    """Nearest code, ties to the even one, saturating; the sign of zero is kept."""
    mags = magnitudes(fmt)
    v = np.ldexp(np.abs(x), -_per_element(scales, x.shape[1]))
    hi = np.clip(np.searchsorted(mags, v, side="left"), 1, len(mags) - 1)
    lo = hi - 1
    below, above = v - mags[lo], mags[hi] - v
    c = np.where(below < above, lo, np.where(above < below, hi, np.where(lo % 2 == 0, lo, hi)))
    c = np.where(v > mags[-1], len(mags) - 1, c)
    return (c + 128 * np.signbit(x)).astype(np.uint8)


def encode(x, fmt):
    x = np.asarray(x, dtype=np.float64)
    s = scale_bytes(x, fmt)
    return codes_of(np.where(np.isfinite(x), x, 0.0), np.where(s == 255, 127, s), fmt), s


def decode(codes, scales, fmt):
    mags = magnitudes(fmt)
    table = np.full(256, np.nan)
    table[:len(mags)] = mags
    table[128:128 + len(mags)] = -mags
    v = np.ldexp(table[codes], _per_element(scales, codes.shape[1]))
    return np.where(_per_element(scales, codes.shape[1]) == 128, np.nan, v)


def norm_forward(x, gamma, beta, eps):
    """y, n, mean, rstd in 64 bits."""
    x = np.asarray(x, dtype=np.float64)
    mean = x.mean(axis=1)
    dev = x - mean[:, None]
    rstd = 1.0 / np.sqrt((dev * dev).mean(axis=1) + eps)
    n = dev * rstd[:, None]
    y = n * (1.0 if gamma is None else gamma) + (0.0 if beta is None else beta)
    return y, n, mean, rstd


def norm_backward(dy, n, gamma, rstd):
    """dx, dgamma, dbeta from the normalised rows n."""
    h = dy * (1.0 if gamma is None else gamma)
    a, b = h.mean(axis=1, keepdims=True), (h * n).mean(axis=1, keepdims=True)
    return rstd[:, None] * (h - a - n * b), (dy * n).sum(axis=0), dy.sum(axis=0)


def weight_grad(delta, v, gamma=None, beta=None):
    g, db = delta.T @ v, delta.sum(axis=0)
    if gamma is not None:
        g = g * gamma
    if beta is not None:
        g = g + np.outer(db, beta)
    return g, db
