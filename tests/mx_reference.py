"""Microscaled formats and the operators over them, plainly, in float64
(numpy).  Shares no code with the library: codes come from searching the
format's table of values, scales from frexp."""
import numpy as np

BLOCK, PAD = 32, 128


def padded(K):
    return (K + PAD - 1) // PAD * PAD


def _e4m3_table():
    """The 127 non-negative finite e4m3 values, by code."""
    v = []
    for code in range(127):
        e, m = code >> 3, code & 7
        v.append((m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(v)


E4M3 = _e4m3_table()
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def nearest(z, table):
    """Codes of the table values nearest to |z| (ties to the even code), saturating."""
    a = np.abs(z)
    hi = np.clip(np.searchsorted(table, a), 1, len(table) - 1)
    lo = hi - 1
    dl, dh = a - table[lo], table[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(up, hi, lo)


def scale_exponents(amax, fmt):
    """Exponent of every block's scale; amax finite, >= 0."""
    m, e = np.frexp(amax)  # amax = m 2^e, 1/2 <= m < 1
    fl = e - 1  # floor(log2 amax)
    if fmt == "e2m1":
        s = fl - 2
    else:
        s = fl - 8 + (m > 0.875)
    return np.maximum(np.where(amax > 0, s, -127), -127)


def quantize(x, fmt):
    """x [R, K] float64 -> (codes uint8 [R, Kp] unpacked with the sign in bit 7 (e4m3) or 3,
    scale bytes uint8 [R, Kp / 32])."""
    R, K = x.shape
    p = np.zeros((R, padded(K)))
    p[:, :K] = x
    b = p.reshape(R, -1, BLOCK)
    bad = ~np.isfinite(b).all(2)
    b = np.where(bad[:, :, None], 0.0, b)
    s = scale_exponents(np.abs(b).max(2), fmt)
    z = np.ldexp(b, -s[:, :, None])
    table, sign = (E4M3, 7) if fmt == "e4m3" else (E2M1, 3)
    codes = nearest(z, table) | (np.signbit(z).astype(np.int64) << sign)
    codes = np.where(bad[:, :, None], 0, codes)
    return codes.reshape(R, -1).astype(np.uint8), np.where(bad, 255, s + 127).astype(np.uint8)


def pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed):
    out = np.empty(packed.shape[:-1] + (packed.shape[-1] * 2,), np.uint8)
    out[..., 0::2] = packed & 15
    out[..., 1::2] = packed >> 4
    return out


def values(codes, scales, fmt):
    """float64 values of unpacked codes [..., Kp] and scale bytes [..., Kp / 32]."""
    if fmt == "e4m3":
        v = np.where(codes & 128, -1.0, 1.0) * np.append(E4M3, np.nan)[codes & 127]
    else:
        v = np.where(codes & 8, -1.0, 1.0) * E2M1[codes & 7]
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return v * np.repeat(s, BLOCK, -1)


def rms_norm(h, w, eps):
    return h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * w


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def erf(x):
    from scipy.special import erf as f
    return f(x)


def activation(p, act, N, inter, limit, alpha, beta):
    """act(p) of p [M, N1] and the gate / up halves (None for plain kinds)."""
    if act in ("silu_and_mul", "gelu_and_mul", "swiglu"):
        g, u = (p[:, 0::2], p[:, 1::2]) if inter else (p[:, :N], p[:, N:])
        if act == "silu_and_mul":
            return g * sigmoid(g) * u
        if act == "gelu_and_mul":
            return 0.5 * g * (1 + erf(g / np.sqrt(2))) * u
        if limit > 0:
            g, u = np.minimum(g, limit), np.clip(u, -limit, limit)
        return g * sigmoid(alpha * g) * (u + beta)
    if act == "relu":
        return np.maximum(p, 0)
    if act == "gelu":
        return 0.5 * p * (1 + erf(p / np.sqrt(2)))
    if act == "silu":
        return p * sigmoid(p)
    return p


def grouped(a, w, bias, seg_end):
    """Products of the rows of a (values) with their experts' w (values), and the sum of the
    terms' magnitudes (with the bias's)."""
    M, N1 = a.shape[0], w.shape[1]
    p, mag = np.zeros((M, N1)), np.zeros((M, N1))
    lo = 0
    for e, hi in enumerate(np.asarray(seg_end)):
        hi = int(min(max(hi, lo), M))
        if hi > lo:
            p[lo:hi] = a[lo:hi] @ w[e].T
            mag[lo:hi] = np.abs(a[lo:hi]) @ np.abs(w[e]).T
            if bias is not None:
                p[lo:hi] += bias[e]
                mag[lo:hi] += np.abs(bias[e])
        lo = hi
    return p, mag
