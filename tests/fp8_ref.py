"""Plain 64-bit references of the 8-bit operators, in numpy, from the definitions."""
import numpy as np
import torch


def scale_cols(c):
    return -(-c // 512) * 4


def round_e4m3(v):
    """The nearest e4m3 value (3 bits below the leading one, spacing 2^-9 at least), ties to even."""
    v = np.asarray(v, np.float64)
    with np.errstate(all="ignore"):
        _, x = np.frexp(np.abs(v))
        step = np.ldexp(1.0, np.maximum(x - 1, -6) - 3)
        return np.where(np.isfinite(v), np.rint(v / step) * step, np.nan)


def scale_byte(amax):
    """b with b - 127 the least e such that amax <= 448 * 2^e, clamped to [0, 254]; 0 for 0; 255
    for an infinity or NaN."""
    amax = np.asarray(amax, np.float64)
    with np.errstate(all="ignore"):
        m, x = np.frexp(amax)  # amax = m 2^x, 0.5 <= m < 1; 448 = 0.875 * 2^9
        e = x - 9 + (m > 0.875)
    b = np.clip(e + 127, 0, 254)
    b = np.where(amax == 0, 0, b)
    return np.where(np.isfinite(amax), b, 255).astype(np.int64)


def scale_value(b):
    b = np.asarray(b, np.int64)
    return np.where(b == 255, np.nan, np.ldexp(1.0, np.where(b == 255, 0, b) - 127))


def amax_of(v, axis):
    """Largest |v|, with a NaN counting as the largest."""
    a = np.abs(v)
    return np.where(np.isnan(a).any(axis), np.inf, np.where(np.isnan(a), 0, a).max(axis))


def quantize(v):
    """Rows v [n, c] -> (e4m3 values [n, c], bytes [n, scale_cols(c)])."""
    v = np.asarray(v, np.float64)
    n, c = v.shape
    kb = -(-c // 128)
    w = np.zeros((n, kb * 128))
    w[:, :c] = v
    w = w.reshape(n, kb, 128)
    b = scale_byte(amax_of(w, 2))
    s = np.zeros((n, scale_cols(c)), np.int64)
    s[:, :kb] = b
    with np.errstate(all="ignore"):
        q = round_e4m3(w / scale_value(b)[:, :, None])
    return q.reshape(n, kb * 128)[:, :c], s


def quantize_weights(w):
    w = np.asarray(w, np.float64)
    E, n, c = w.shape
    nb, kb = -(-n // 128), -(-c // 128)
    p = np.zeros((E, nb * 128, kb * 128))
    p[:, :n, :c] = w
    p = p.reshape(E, nb, 128, kb, 128)
    b = scale_byte(amax_of(p.transpose(0, 1, 3, 2, 4).reshape(E, nb, kb, -1), 3))
    s = np.zeros((E, nb, scale_cols(c)), np.int64)
    s[:, :, :kb] = b
    with np.errstate(all="ignore"):
        q = round_e4m3(p / scale_value(b)[:, :, None, :, None])
    return q.reshape(E, nb * 128, kb * 128)[:, :n, :c], s


def dequantize(q, s):
    """Values [n, c] of e4m3 values and bytes [n, scale_cols(c)]."""
    return q * np.repeat(scale_value(s), 128, axis=-1)[..., : q.shape[-1]]


def dequantize_w(q, s):
    f = np.repeat(np.repeat(scale_value(s), 128, axis=1)[:, : q.shape[1]], 128, axis=2)[:, :, : q.shape[2]]
    return q * f


def to_torch(q, s):
    """(float8_e4m3fn, uint8) tensors of reference values and bytes."""
    return torch.from_numpy(q).to(torch.float32).to(torch.float8_e4m3fn), torch.from_numpy(s.astype(np.uint8))


def silu(a):
    with np.errstate(over="ignore"):
        return a / (1 + np.exp(-a))


def row_experts(counts, E):
    """Expert of each row: segments source-major, segment s holds rows of expert s % E."""
    counts = np.asarray(counts)
    return np.repeat(np.arange(len(counts)) % E, counts)


def matmul(a, w, experts):
    """a [n, K], w [E, N, K] in 64 bits -> (out [n, N], sum |a||w| [n, N])."""
    out, mag = np.zeros((a.shape[0], w.shape[1])), np.zeros((a.shape[0], w.shape[1]))
    for e in range(w.shape[0]):
        r = np.where(experts == e)[0]
        if len(r):
            out[r], mag[r] = a[r] @ w[e].T, np.abs(a[r]) @ np.abs(w[e]).T
    return out, mag
