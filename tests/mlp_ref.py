"""Plain 64-bit statements of the feed-forward operators (numpy), for the tests."""
import numpy as np
from scipy.special import erfc

U32 = 2.0 ** -24   # unit roundoff of FP32
U16 = 2.0 ** -8    # unit roundoff of BF16 (8 significant bits)


def gate(g, fn):
    """a(g) and a'(g)."""
    g = np.asarray(g, dtype=np.float64)
    if fn == "gelu":
        phi = 0.5 * erfc(-g / np.sqrt(2.0))
        return g * phi, phi + g * np.exp(-0.5 * g * g) / np.sqrt(2.0 * np.pi)
    if fn == "silu":
        z, dz = g, 1.0
    else:
        c = 2.0 * np.sqrt(2.0 / np.pi)
        z, dz = c * (g + 0.044715 * g ** 3), c * (1.0 + 3 * 0.044715 * g * g)
    e = np.exp(-np.abs(z))
    s, other = np.where(z >= 0, 1.0, e) / (1.0 + e), np.where(z >= 0, e, 1.0) / (1.0 + e)
    return g * s, s + g * dz * s * other


def gate_error(g, fn):
    """Relative error that FP32 arithmetic may leave in a and a' (each relative to |a| + |g a'| + the terms of a'): the
    exponential's argument carries a few roundings, so its error grows with the argument (at most 2 + 1.2 |z| units
    for the hardware's exponential, |z| units for the rounding of z's three products; erfc's with g^2)."""
    g = np.abs(np.asarray(g, dtype=np.float64))
    z = g if fn == "silu" else 1.6 * (g + 0.044715 * g ** 3) if fn == "gelu_tanh" else g * g
    return (16 + 8 * z) * 2 * U32


def philox(counter, key):
    """Philox4x32-10: counter of four arrays, key of two numbers; four arrays of 32-bit numbers."""
    m = np.uint64(0xFFFFFFFF)
    c = [np.asarray(x, dtype=np.uint64) for x in np.broadcast_arrays(*counter)]
    k = [int(key[0]), int(key[1])]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        hi_a, hi_b = a >> np.uint64(32), b >> np.uint64(32)
        c = [hi_b ^ c[1] ^ np.uint64(k[0]), b & m, hi_a ^ c[3] ^ np.uint64(k[1]), a & m]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def threshold(p):
    return int(np.floor(65536.0 * float(np.float32(p)) + 0.5))


def keep(T, d, p, seed, step, site, rows=None):
    """Truth values: the element is kept.  rows: which rows (all T by default)."""
    rows = np.arange(T) if rows is None else np.asarray(rows)
    groups = -(-d // 8)
    r = philox((np.arange(groups)[None, :], rows[:, None], np.uint64(site), np.uint64(step & 0xFFFFFFFF)),
               (seed & 0xFFFFFFFF, seed >> 32))
    bits = np.zeros((len(rows), groups, 8), dtype=np.int64)
    for j in range(4):
        bits[:, :, 2 * j] = (r[j] & np.uint64(0xFFFF)).astype(np.int64)
        bits[:, :, 2 * j + 1] = (r[j] >> np.uint64(16)).astype(np.int64)
    return bits.reshape(len(rows), 8 * groups)[:, :d] >= threshold(p)


def drop(v, p, seed, step, site):
    P = threshold(p)
    if P == 0:
        return v
    return np.where(keep(*v.shape, p, seed, step, site), v * (65536.0 / (65536 - P)), 0.0)


def product(a, b, dt):
    """a b (64 bits), and how far the tensor cores' FP32 sums may be off: an MMA adds 16 products and the accumulator,
    each truncated to the largest's last place (2 U32 of it), K / 16 times, and segments are added to nearest.  FP32
    operands make six times the steps, and the products that are left out are below 2^-23 of |a_k b_k|."""
    a, b = np.asarray(a, dtype=np.float64), np.asarray(b, dtype=np.float64)
    K = a.shape[1]
    size = np.abs(a) @ np.abs(b)
    if dt == "bf16":
        return a @ b, (2 * (17 * (-(-K // 16))) + K // 512 + 1) * U32 * size
    return a @ b, (12 * (17 * (-(-K // 16))) + K // 128 + 3) * U32 * size


def half_step(v, dt):
    return (U16 if dt == "bf16" else U32) * np.abs(v)
