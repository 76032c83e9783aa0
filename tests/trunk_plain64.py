"""The trunk operators' definitions in float64 torch operations over whole batches, on any device,
for sizes at which the oracle's loops over sequences and rows would take too long.  Pinned to the
oracle by test_trunk_plain64.py; test infrastructure only.  Sequences are time-major [K, B, D];
`ends` holds each sequence's length, 0 .. K."""
from __future__ import annotations

import torch


def norm(x, w, b, eps=1e-5):
    c = x - x.mean(1, keepdim=True)
    return c * ((c * c).mean(1, keepdim=True) + eps).rsqrt() * w + b


def norm_backward(dy, x, w, eps=1e-5):
    """dx, dw, db."""
    c = x - x.mean(1, keepdim=True)
    rstd = ((c * c).mean(1, keepdim=True) + eps).rsqrt()
    hat, g = c * rstd, dy * w
    dx = rstd * (g - g.mean(1, keepdim=True) - hat * (g * hat).mean(1, keepdim=True))
    return dx, (dy * hat).sum(0), dy.sum(0)


def dropout_mask(rows, n, p, seed, offset, device="cpu"):
    """(kept, scale): Philox 4x32 with ten rounds in 64-bit integers, a call for eight columns."""
    low = 0xFFFFFFFF
    cut = int(torch.floor(torch.tensor(p, dtype=torch.float32).double() * 65536.0 + 0.5))

    def product(a, m):  # 32 x 32 bits: (high, low)
        lo, hi = a & 0xFFFF, a >> 16
        mid = hi * m + (lo * m >> 16)
        return mid >> 16 & low, ((mid & 0xFFFF) << 16) | (lo * m & 0xFFFF)

    groups = -(-n // 8)
    c = [torch.arange(groups, device=device).expand(rows, groups),
         torch.arange(rows, device=device)[:, None].expand(rows, groups),
         torch.full((rows, groups), offset & low, device=device),
         torch.full((rows, groups), offset >> 32, device=device)]
    k0, k1 = seed & low, seed >> 32
    for _ in range(10):
        (h0, l0), (h1, l1) = product(c[0], 0xD2511F53), product(c[2], 0xCD9E8D57)
        c = [h1 ^ c[1] ^ k0, l1, h0 ^ c[3] ^ k1, l0]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack(c, -1)
    pieces = torch.stack([words & 0xFFFF, words >> 16], -1).reshape(rows, groups * 8)[:, :n]
    return pieces >= cut, (65536.0 / (65536 - cut) if cut < 65536 else 0.0)


def _on(ends, K):
    """[K, B, 1] truth values: the step is before the sequence's end."""
    return (torch.arange(K, device=ends.device)[:, None] < ends)[..., None]


def conv(x, w, bias, x0, ends, silu=True, du=None):
    """u, last and, from du, dx, dx0, dw, dbias."""
    K, B, _ = x.shape
    W, on = w.shape[1], _on(ends, K)
    line = torch.cat([x0.transpose(0, 1), torch.where(on, x, 0.0)])
    p = bias + sum(line[j:j + K] * w[:, j] for j in range(W))
    s = torch.sigmoid(p)
    at = ends[:, None] + torch.arange(W - 1, device=x.device)
    out = dict(u=torch.where(on, p * s if silu else p, 0.0),
               last=line[at, torch.arange(B, device=x.device)[:, None]])
    if du is None:
        return out
    g = torch.where(on, du, 0.0)
    if silu:
        g = g * s * (1.0 + p * (1.0 - s))
    dline = torch.zeros_like(line)
    for j in range(W):
        dline[j:j + K] += g * w[:, j]
    out.update(dx=torch.where(on, dline[W - 1:], 0.0), dx0=dline[:W - 1].transpose(0, 1),
               dw=torch.stack([(g * line[j:j + K]).sum((0, 1)) for j in range(W)], 1),
               dbias=g.sum((0, 1)))
    return out


def scan(i, ends, softplus=True, backward=True):
    """i: x, dt, dy [K, B, D], A [D, N], Bm, Cm [K, B, G, N], skip, dt_bias [D], z (or None), h0
    and dh_last [B, D, N].  Returns y, h (the last state) and every gradient."""
    K, B, D = i["x"].shape
    G, N = i["Bm"].shape[2:]
    on = _on(ends, K)
    raw = i["dt"] + i["dt_bias"]
    d = torch.where(on, torch.logaddexp(raw, torch.zeros_like(raw)) if softplus else raw, 0.0)
    x = torch.where(on, i["x"], 0.0)
    z = i["z"]
    sz = None if z is None else torch.sigmoid(z)
    gate = 1.0 if z is None else z * sz

    def wide(m):  # [B, G, N] -> [B, D, N]
        return m.repeat_interleave(D // G, 1)

    h, kept, y = i["h0"], [], torch.zeros_like(x)
    for t in range(K):
        kept.append(h)
        new = torch.exp(d[t][..., None] * i["A"]) * h + (d[t] * x[t])[..., None] * wide(i["Bm"][t])
        h = torch.where(on[t][..., None], new, h)
        y[t] = (h * wide(i["Cm"][t])).sum(-1) + i["skip"] * x[t]
    y = torch.where(on, y, 0.0)
    out = dict(y=y * gate, h=h)
    if not backward:
        return out
    kept.append(h)
    dy = torch.where(on, i["dy"], 0.0)
    if z is not None:
        out["dz"] = dy * y * sz * (1.0 + z * (1.0 - sz))
    r = dy * gate
    out.update({k: torch.zeros_like(x) for k in ("dx", "ddt")})
    out.update({k: torch.zeros_like(i["Bm"]) for k in ("dB", "dC")})
    out.update(dA=torch.zeros_like(i["A"]), dD=(r * x).sum((0, 1)))
    e = i["dh_last"]
    for t in reversed(range(K)):
        live = on[t][..., None]
        f = torch.where(live, e + r[t][..., None] * wide(i["Cm"][t]), 0.0)
        a = torch.exp(d[t][..., None] * i["A"])
        q = a * kept[t]
        out["dC"][t] = torch.where(live, r[t][..., None] * kept[t + 1], 0.0).view(B, G, D // G, N).sum(2)
        out["dB"][t] = (f * (d[t] * x[t])[..., None]).view(B, G, D // G, N).sum(2)
        fq = f * q
        out["dA"] += (fq * d[t][..., None]).sum(0)
        fb = (f * wide(i["Bm"][t])).sum(-1)
        out["ddt"][t] = (fq * i["A"]).sum(-1) + x[t] * fb
        out["dx"][t] = d[t] * fb + i["skip"] * r[t]
        e = torch.where(live, a * f, e)
    if softplus:
        out["ddt"] *= torch.sigmoid(raw)
    out.update(ddt_bias=out["ddt"].sum((0, 1)), dh0=e)
    return out
