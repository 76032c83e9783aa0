"""fp64 oracle of the trunk operators (layer norm, counter-based dropout, causal convolution,
selective scan), from their definitions, in numpy.  Test infrastructure only: it shares no code
with the CUDA path.  Sequences are time-major [K, B, D]; `ends` holds each sequence's length.
"""
from __future__ import annotations

import numpy as np


def bf16(v):
    """Rounded to bf16, to nearest even, as float64."""
    m, e = np.frexp(np.asarray(v, dtype=np.float64))
    return np.ldexp(np.rint(m * 256.0), e - 8)


def sigmoid(v):
    return 0.5 * (1.0 + np.tanh(0.5 * v))


# ---- layer norm ----

def layernorm(x, w, b, eps):
    c = x - x.mean(axis=1, keepdims=True)
    rstd = 1.0 / np.sqrt((c * c).mean(axis=1, keepdims=True) + eps)
    return c * rstd * w + b


def layernorm_backward(dy, x, w, eps):
    c = x - x.mean(axis=1, keepdims=True)
    rstd = 1.0 / np.sqrt((c * c).mean(axis=1, keepdims=True) + eps)
    hat, g = c * rstd, dy * w
    dx = rstd * (g - g.mean(axis=1, keepdims=True) - hat * (g * hat).mean(axis=1, keepdims=True))
    return dx, (dy * hat).sum(axis=0), dy.sum(axis=0)


# ---- dropout ----

def philox4x32(counter, key, rounds=10):
    """Philox 4x32 (Salmon, Moraes, Dror, Shaw, 2011), one counter at a time in plain integers."""
    c, k = list(counter), list(key)
    for _ in range(rounds):
        p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(p1 >> 32) ^ c[1] ^ k[0], p1 & 0xFFFFFFFF, (p0 >> 32) ^ c[3] ^ k[1], p0 & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def dropout_mask(rows, n, p, seed, offset):
    """(kept, scale): element (row, 8 i + j) takes bits 16 j .. 16 j + 15 of the call with counter
    (i, row, offset low, offset high) and is kept where they are >= round(65536 p)."""
    cut = int(np.floor(np.float64(np.float32(p)) * 65536.0 + 0.5))
    kept = np.zeros((rows, n), dtype=bool)
    key = (seed & 0xFFFFFFFF, seed >> 32)
    for r in range(rows):
        for i in range(-(-n // 8)):
            words = philox4x32((i, r, offset & 0xFFFFFFFF, offset >> 32), key)
            for j in range(min(8, n - 8 * i)):
                kept[r, 8 * i + j] = (words[j // 2] >> (16 * (j % 2))) & 0xFFFF >= cut
    return kept, (65536.0 / (65536 - cut) if cut < 65536 else 0.0)


# ---- causal convolution ----

def conv(x, w, bias, x0, ends, silu=True):
    """u [K, B, D] and the last W - 1 inputs [B, W - 1, D] of each sequence."""
    K, B, D = x.shape
    W = w.shape[1]
    u, last = np.zeros((K, B, D)), np.zeros((B, W - 1, D))
    for b in range(B):
        line = np.concatenate([x0[b], x[:ends[b], b]])
        for t in range(ends[b]):
            p = bias + (w.T * line[t:t + W]).sum(axis=0)
            u[t, b] = p * sigmoid(p) if silu else p
        last[b] = line[ends[b]:ends[b] + W - 1]
    return u, last


def conv_backward(du, x, w, bias, x0, ends, silu=True):
    """dx, dx0, dw, dbias."""
    K, B, D = x.shape
    W = w.shape[1]
    dx, dx0 = np.zeros((K, B, D)), np.zeros((B, W - 1, D))
    dw, dbias = np.zeros((D, W)), np.zeros(D)
    for b in range(B):
        line = np.concatenate([x0[b], x[:ends[b], b]])
        dline = np.zeros_like(line)
        for t in range(ends[b]):
            g = du[t, b]
            if silu:
                p = bias + (w.T * line[t:t + W]).sum(axis=0)
                s = sigmoid(p)
                g = g * s * (1.0 + p * (1.0 - s))
            dline[t:t + W] += g * w.T
            dw += (g * line[t:t + W]).T
            dbias += g
        dx0[b], dx[:ends[b], b] = dline[:W - 1], dline[W - 1:]
    return dx, dx0, dw, dbias


# ---- selective scan ----

def _per_channel(m, D):
    """[.., G, N] -> [.., D, N]: a group's values at its channels."""
    return np.repeat(m, D // m.shape[-2], axis=-2)


def scan(i, ends, softplus=True):
    """i: x, dt [K, B, D], A [D, N], Bm, Cm [K, B, G, N], skip, dt_bias [D], z (or None), h0
    [B, D, N].  Returns y, the last state and, for scan_backward, every state before a step."""
    K, B, D = i["x"].shape
    raw = i["dt"] + i["dt_bias"]
    d = np.logaddexp(0.0, raw) if softplus else raw
    h, y, kept = i["h0"].astype(np.float64).copy(), np.zeros((K, B, D)), []
    for t in range(K):
        kept.append(h.copy())
        for b in range(B):
            if t >= ends[b]:
                continue
            a = np.exp(d[t, b][:, None] * i["A"])
            h[b] = a * h[b] + (d[t, b] * i["x"][t, b])[:, None] * _per_channel(i["Bm"][t, b], D)
            y[t, b] = (h[b] * _per_channel(i["Cm"][t, b], D)).sum(axis=1) + i["skip"] * i["x"][t, b]
            if i["z"] is not None:
                y[t, b] *= i["z"][t, b] * sigmoid(i["z"][t, b])
    return y, h, kept


def scan_backward(i, ends, dy, dh_last, softplus=True):
    K, B, D = i["x"].shape
    G, N = i["Bm"].shape[2:]
    _, _, kept = scan(i, ends, softplus)
    raw = i["dt"] + i["dt_bias"]
    d = np.logaddexp(0.0, raw) if softplus else raw
    out = {k: np.zeros((K, B, D)) for k in ("dx", "ddt", "dz")}
    out.update({k: np.zeros((K, B, G, N)) for k in ("dB", "dC")})
    out.update(dA=np.zeros((D, N)), dskip=np.zeros(D), ddt_bias=np.zeros(D))
    e = dh_last.astype(np.float64).copy()
    for t in reversed(range(K)):
        for b in range(B):
            if t >= ends[b]:
                continue
            x, dv = i["x"][t, b], d[t, b]
            Bn, Cn = _per_channel(i["Bm"][t, b], D), _per_channel(i["Cm"][t, b], D)
            a = np.exp(dv[:, None] * i["A"])
            q = a * kept[t][b]
            h = q + (dv * x)[:, None] * Bn
            r = dy[t, b]
            if i["z"] is not None:
                z, s = i["z"][t, b], sigmoid(i["z"][t, b])
                out["dz"][t, b] = r * ((h * Cn).sum(axis=1) + i["skip"] * x) * s * (1.0 + z * (1.0 - s))
                r = r * z * s
            f = e[b] + r[:, None] * Cn
            out["dC"][t, b] = (r[:, None] * h).reshape(G, D // G, N).sum(axis=1)
            out["dB"][t, b] = (f * (dv * x)[:, None]).reshape(G, D // G, N).sum(axis=1)
            out["dA"] += f * q * dv[:, None]
            dd = (f * (i["A"] * q + x[:, None] * Bn)).sum(axis=1)
            out["ddt"][t, b] = dd * (sigmoid(raw[t, b]) if softplus else 1.0)
            out["dx"][t, b] = dv * (f * Bn).sum(axis=1) + i["skip"] * r
            out["dskip"] += r * x
            e[b] = a * f
    out["ddt_bias"] = out["ddt"].sum(axis=(0, 1))
    out["dh0"] = e
    return out
