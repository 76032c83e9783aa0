"""fp64 oracle of the gated block's operators (root-mean-square norm, values in 8 bits, gated linear
recurrence, products with 4-bit weights), from their definitions, in numpy.  Test infrastructure
only: it shares no code with the CUDA path.  Sequences are time-major [K, B, D]; `ends` holds each
sequence's length.
"""
from __future__ import annotations

import numpy as np

from .trunk import sigmoid

BLOCK, PERIOD = 32, 8

# Every finite value of e4m3 that is not negative, by its code: exponent 0 is subnormal, code 127
# is NaN.
E4M3 = np.array([(c % 8) * 2.0 ** -9 if c < 8 else (1 + (c % 8) / 8) * 2.0 ** (c // 8 - 7)
                 for c in range(127)])


# ---- values in 8 bits ----

def e4m3_code(u):
    """The code nearest to a number, ties to the even code; |u| <= 448."""
    a = abs(float(u))
    hi = int(np.searchsorted(E4M3, a))
    lo = max(hi - 1, 0)
    hi = min(hi, 126)
    d_lo, d_hi = a - E4M3[lo], E4M3[hi] - a
    code = lo if d_lo < d_hi or (d_lo == d_hi and lo % 2 == 0) else hi
    return code | (128 if np.signbit(u) else 0)


def e4m3_value(code):
    v = np.nan if code % 128 == 127 else E4M3[code % 128]
    return -v if code >= 128 else v


def pack8(v):
    """(codes, scales) of a row: each block's scale is the smallest power of two, 2^-126 at least,
    that brings its largest magnitude to 448 or below."""
    v = np.asarray(v, dtype=np.float64)
    codes, scales = [], []
    for c in range(0, len(v), BLOCK):
        part = v[c:c + BLOCK]
        if not np.all(np.isfinite(part)):
            codes += [127] * len(part)
            scales.append(255)
            continue
        k = -126
        while np.max(np.abs(part)) > 448 * 2.0 ** k:
            k += 1
        codes += [e4m3_code(u * 2.0 ** -k) for u in part]
        scales.append(k + 127)
    return np.array(codes, dtype=np.uint8), np.array(scales, dtype=np.uint8)


def unpack8(codes, scales):
    return np.array([e4m3_value(int(c)) * (np.nan if scales[i // BLOCK] == 255
                                           else 2.0 ** (int(scales[i // BLOCK]) - 127))
                     for i, c in enumerate(codes)])


def held8(v):
    """What the rows of an array stand for in 8 bits."""
    v = np.asarray(v, dtype=np.float64)
    rows = v.reshape(-1, v.shape[-1])
    return np.stack([unpack8(*pack8(r)) for r in rows]).reshape(v.shape)


# ---- root-mean-square norm ----

def rmsnorm(s, w, eps):
    return s * w / np.sqrt((s * s).mean(axis=1, keepdims=True) + eps)


def rmsnorm_backward(dy, s, w, eps, stream=None, ds=0.0):
    """dx, dw, and y formed again.  `stream` takes the place of s behind the statistics."""
    rstd = 1.0 / np.sqrt((s * s).mean(axis=1, keepdims=True) + eps)
    hat = (s if stream is None else stream) * rstd
    g = dy * w
    dx = rstd * (g - hat * (g * hat).mean(axis=1, keepdims=True)) + ds
    return dx, (dy * hat).sum(axis=0), hat * w


# ---- gated linear recurrence ----

def silu(z):
    return 1.0 if z is None else z * sigmoid(z)


def gated(x, f, bias, z, h0, ends):
    """y, the last state, and the state before every step."""
    K, B, D = x.shape
    h, y, before = h0.copy(), np.zeros((K, B, D)), np.zeros((K, B, D))
    for b in range(B):
        for t in range(ends[b]):
            before[t, b] = h[b]
            g = sigmoid(f[t, b] + bias)
            h[b] = g * h[b] + sigmoid(-(f[t, b] + bias)) * x[t, b]
            y[t, b] = h[b] * silu(None if z is None else z[t, b])
    return y, h, before


def gated_backward(dy, x, f, bias, z, h0, ends, dh_last=None, kept=False):
    """The gradients as a dict, and y formed again.  `kept`: x, f and z as held in 8 bits, each
    period's h taken up again from the state that the recurrence on the unheld ones had."""
    K, B, D = x.shape
    before = gated(x, f, bias, z, h0, ends)[2]
    if kept:
        x, f, z = held8(x), held8(f), None if z is None else held8(z)
    y = np.zeros((K, B, D))
    out = {k: np.zeros((K, B, D)) for k in ("dx", "df", "dz")}
    out["dh0"] = np.zeros((B, D))
    for b in range(B):
        now = np.zeros((K, D))
        for t in range(ends[b]):
            start = before[t, b] if t % PERIOD == 0 or not kept else now[t - 1]
            before[t, b] = start
            g = sigmoid(f[t, b] + bias)
            now[t] = g * start + sigmoid(-(f[t, b] + bias)) * x[t, b]
            y[t, b] = now[t] * silu(None if z is None else z[t, b])
        c = np.zeros(D) if dh_last is None else dh_last[b].copy()
        for t in reversed(range(ends[b])):
            zt = None if z is None else z[t, b]
            g, i = sigmoid(f[t, b] + bias), sigmoid(-(f[t, b] + bias))
            dh = dy[t, b] * silu(zt) + c
            out["dx"][t, b] = dh * i
            out["df"][t, b] = dh * (before[t, b] - x[t, b]) * g * i
            if z is not None:
                s = sigmoid(zt)
                out["dz"][t, b] = dy[t, b] * now[t] * (s + zt * s * (1 - s))
            c = dh * g
        out["dh0"][b] = c
    out["dbias"] = out["df"].sum(axis=(0, 1))
    if z is None:
        del out["dz"]
    return out, y


# ---- 4-bit weights ----

def weights4(codes, scales, K, group):
    """W [N, K] of codes [N, ceil(K / 2)], two to a byte, and scales [N, ceil(K / group)]."""
    N = codes.shape[0]
    W = np.zeros((N, K))
    for k in range(K):
        W[:, k] = ((codes[:, k // 2].astype(int) >> (4 * (k % 2))) % 16 - 8) * scales[:, k // group]
    return W
