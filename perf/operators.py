"""What is measured of the trunk operators (layer norm, counter-based dropout, causal convolution,
selective scan): cases, inputs, a plain form in elementary torch operations, the framework's calls,
and a 64-bit form of the definitions.

Layouts follow the recurrent path: sequences are time-major [K][B][D], activations are fp32 or
bf16, parameters and states are fp32.

  norm      y = (x - mean) * rstd * w + b per row; backward: dx, dw, db.
  dropnorm  s = residual + mask * x / (1 - p), rounded to the activations' type; y = norm(s);
            backward from dy and the residual stream's own gradient ds: dx, dres, dw, db.
  conv      u_t = silu(bias + sum_j w[:, j] x_{t - (W-1) + j}) with a carried history of W-1
            inputs; backward: dx, dw, dbias, and the history's gradient.
  scan      d_t = softplus(dt_t + dt_bias);  h_t = exp(d_t A) h_{t-1} + d_t B_t x_t;
            y_t = (C_t . h_t + D x_t) silu(z_t); backward: every input's and parameter's gradient.
  token     one conv step and one scan step, for single tokens, each on inputs of its own.

A sequence of length L < K ends at L: later outputs and gradients are 0 and its state stays.
"""
import math

import numpy as np
import torch

own = False

F32, BF16 = "f32", "bf16"
EPS = 1e-5


# ---- cases ---------------------------------------------------------------------------------

def listed():
    return [
        # The smallest workload's rows (4 sequences x 8 steps, 32 channels): latency alone.
        dict(name="norm_f32_tiny", op="norm", rows=32, n=32, dtype=F32),
        # The stress workload's rows (2048 sequences x 128 steps, 256 channels): streaming.
        dict(name="norm_f32_stress", op="norm", rows=262144, n=256, dtype=F32),
        # Long rows of an odd width, so that no row but the first starts aligned.
        dict(name="norm_bf16_wide_odd", op="norm", rows=6007, n=2501, dtype=BF16),
        # A residual block of the 32 x 64 x 128 workload.
        dict(name="dropnorm_f32_pages", op="dropnorm", rows=2048, n=128, p=0.1, dtype=F32),
        # The same block at the stress workload's rows, activations in 16 bits.
        dict(name="dropnorm_bf16_stress", op="dropnorm", rows=262144, n=256, p=0.2, dtype=BF16),
        # The convolution in front of the scan, at the 32 x 64 workload.
        dict(name="conv_f32_pages", op="conv", B=32, K=64, D=256, W=4, ragged=False, dtype=F32),
        # A large batch of sequences of different lengths, an odd number of steps.
        dict(name="conv_bf16_ragged", op="conv", B=64, K=1023, D=1536, W=4, ragged=True, dtype=BF16),
        # Serving, a few sequences, one token each: latency.
        dict(name="token_f32_small", op="token", B=32, D=256, N=32, G=1, W=4, dtype=F32),
        # Serving, a full batch with a wide state: the state's traffic.
        dict(name="token_bf16_large", op="token", B=1024, D=2048, N=64, G=1, W=4, dtype=BF16),
        # Two long prompts of different lengths: few rows, a long axis.
        dict(name="scan_prompt_bf16_long", op="scan", train=False, B=2, K=8191, D=1024, N=16, G=1,
             ragged=True, dtype=BF16),
        # Training at the 32 x 64 workload, 32 states per channel.
        dict(name="scan_train_f32_pages", op="scan", train=True, B=32, K=64, D=256, N=32, G=1,
             ragged=False, dtype=F32),
        # Training on a large batch, B and C shared by groups of channels.
        dict(name="scan_train_bf16_large", op="scan", train=True, B=64, K=512, D=1024, N=16, G=2,
             ragged=False, dtype=BF16),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "dropnorm", "conv", "token", "prompt", "train"])
    dtype = rng.choice([F32, BF16])
    while True:
        if op in ("norm", "dropnorm"):
            c = dict(op=op, rows=_log_int(rng, 1, 262144), n=_log_int(rng, 8, 8192), dtype=dtype)
            if op == "dropnorm":
                c["p"] = rng.choice([0.05, 0.1, 0.25, 0.5])
            if 4096 <= c["rows"] * c["n"] <= 1 << 26 and c["n"] != 3072:
                return c
            continue
        D = rng.choice([1, 2, 4, 8]) * _log_int(rng, 16, 256)
        if D == 3072:
            continue
        if op == "conv":
            c = dict(op=op, B=_log_int(rng, 1, 256), K=_log_int(rng, 1, 2048), D=D,
                     W=rng.choice([2, 3, 4]), ragged=rng.random() < 0.5, dtype=dtype)
            if 4096 <= c["B"] * c["K"] * D <= 100_000_000:
                return c
            continue
        N, G = rng.choice([4, 8, 16, 16, 24, 32, 64]), rng.choice([1, 1, 2, 4])
        if D % G:
            continue
        if op == "token":
            c = dict(op=op, B=_log_int(rng, 1, 1024), D=D, N=N, G=G, W=rng.choice([2, 3, 4]),
                     dtype=dtype)
            if 4096 <= c["B"] * D * N <= 1 << 27:
                return c
            continue
        train = op == "train"
        c = dict(op="scan", train=train, B=_log_int(rng, 1, 64 if train else 8),
                 K=_log_int(rng, 16, 1024 if train else 8192), D=D, N=N, G=G,
                 ragged=rng.random() < 0.5, dtype=dtype)
        if 65536 <= c["B"] * c["K"] * D * N <= (1 << 29 if train else 1 << 28):
            return c


# ---- inputs --------------------------------------------------------------------------------

def _type(case):
    return torch.float32 if case["dtype"] == F32 else torch.bfloat16


def _inputs(case, seed):
    """The inputs of a case, on the GPU, from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    act = _type(case)

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda").mul_(std).add_(mean).to(dtype)

    def uniform(*shape, lo, hi):
        return torch.rand(*shape, generator=g, device="cuda").mul_(hi - lo).add_(lo)

    if case["op"] in ("norm", "dropnorm"):
        M, n = case["rows"], case["n"]
        t = dict(x=normal(M, n, std=1.5, mean=0.3, dtype=act), w=normal(n, std=0.2, mean=1.0),
                 b=normal(n, std=0.2), dy=normal(M, n, dtype=act))
        if case["op"] == "dropnorm":
            t["residual"] = normal(M, n, std=2.0, dtype=act)
            t["ds"] = normal(M, n, dtype=act)
            t["rng"] = torch.tensor([seed * 2654435761 % (1 << 62) + 12345, seed + (5 << 33)],
                                    dtype=torch.int64, device="cuda")
        return t
    B, D, W = case["B"], case["D"], case.get("W", 4)
    if case["op"] == "conv":
        K = case["K"]
        # x is the first half of the block's input projection; the second half is the gate z.
        t = dict(x=normal(K, B, 2 * D, dtype=act)[..., :D], w=uniform(D, W, lo=-0.5, hi=0.5),
                 bias=normal(D, std=0.1), x0=normal(B, W - 1, D, dtype=act),
                 dy=normal(K, B, D, dtype=act), lengths=None)
        if case["ragged"]:
            t["lengths"] = torch.randint(0, K + 1, (B,), generator=g, device="cuda",
                                         dtype=torch.int32)
        return t
    N, G = case["N"], case["G"]
    # Decay rates 1 .. N per channel, spread by a tenth; steps of 1e-3 to 1e-1 after softplus.
    A = -torch.arange(1, N + 1, device="cuda", dtype=torch.float32).repeat(D, 1)
    t = dict(A=A * uniform(D, N, lo=0.9, hi=1.1), D=normal(D, std=0.2, mean=1.0),
             dt_bias=torch.log(torch.expm1(torch.exp(uniform(D, lo=math.log(1e-3),
                                                             hi=math.log(1e-1))))))
    if case["op"] == "token":
        p = normal(B, 2 * G * N, dtype=act)
        t.update(x=normal(B, 2 * D, dtype=act)[:, :D], w=uniform(D, W, lo=-0.5, hi=0.5),
                 bias=normal(D, std=0.1), x0=normal(B, W - 1, D, dtype=act),
                 v=normal(B, D, dtype=act),  # what the scan reads: a rounding of u decides nothing
                 dt=normal(B, D, std=0.5, dtype=act), z=normal(B, D, dtype=act),
                 Bm=p[:, :G * N].unflatten(-1, (G, N)), Cm=p[:, G * N:].unflatten(-1, (G, N)),
                 h0=normal(B, D, N, std=0.1))
        return t
    K = case["K"]
    p = normal(K, B, 2 * G * N, dtype=act)  # B and C come out of one projection
    t.update(x=normal(K, B, D, dtype=act), dt=normal(K, B, D, std=0.5, dtype=act),
             z=normal(K, B, 2 * D, dtype=act)[..., D:],
             Bm=p[..., :G * N].unflatten(-1, (G, N)), Cm=p[..., G * N:].unflatten(-1, (G, N)),
             h0=normal(B, D, N, std=0.1), lengths=None)
    if case["ragged"]:
        t["lengths"] = torch.randint(0, K + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        t["lengths"][0] = K
    if case["train"]:
        t["dy"] = normal(K, B, D, dtype=act)
    return t


def prepare(case, seed):
    t = _inputs(case, seed)
    state = dict(case=case, t=t)
    if own:
        from recurrent_cfc_cell_gb300 import trunk

        act, op = _type(case), case["op"]
        if op == "norm":
            state["step"] = trunk.LayerNormStep(case["rows"], case["n"], dtype=act, eps=EPS).bind(
                x=t["x"], w=t["w"], b=t["b"], dy=t["dy"])
        elif op == "dropnorm":
            state["step"] = trunk.DropoutNormStep(case["rows"], case["n"], p=case["p"], dtype=act,
                                                  eps=EPS).bind(
                x=t["x"], residual=t["residual"], rng=t["rng"], w=t["w"], b=t["b"], dy=t["dy"],
                ds=t["ds"])
        elif op == "conv":
            state["step"] = trunk.ConvStep(case["K"], case["B"], case["D"], case["W"],
                                           dtype=act).bind(
                x=t["x"], w=t["w"], bias=t["bias"], x0=t["x0"], lengths=t["lengths"], dy=t["dy"])
        elif op == "token":
            state["conv"] = trunk.ConvToken(case["B"], case["D"], case["W"], dtype=act).bind(
                x=t["x"], w=t["w"], bias=t["bias"], state=t["x0"],
                new_state=torch.empty_like(t["x0"]))
            state["scan"] = trunk.ScanToken(case["B"], case["D"], case["N"], case["G"],
                                            dtype=act).bind(
                x=t["v"], dt=t["dt"], A=t["A"], Bm=t["Bm"], Cm=t["Cm"], D=t["D"],
                dt_bias=t["dt_bias"], z=t["z"], state=t["h0"],
                new_state=torch.empty_like(t["h0"]))
        else:
            state["step"] = trunk.ScanStep(case["K"], case["B"], case["D"], case["N"], case["G"],
                                           dtype=act, train=case["train"]).bind(
                x=t["x"], dt=t["dt"], A=t["A"], Bm=t["Bm"], Cm=t["Cm"], D=t["D"],
                dt_bias=t["dt_bias"], z=t["z"], h0=t["h0"], lengths=t["lengths"],
                dy=t.get("dy"))
    return state


# ---- one pass ------------------------------------------------------------------------------

def run(state):
    case, t = state["case"], state["t"]
    if own:
        if case["op"] == "token":
            u, conv_state = state["conv"].run()
            y, h = state["scan"].run()
            return dict(u=u, conv_state=conv_state, y=y, h=h)
        state["step"].run()
        return state["step"].outputs()
    if case["op"] == "norm":
        y, mean, rstd = _norm(t["x"].float(), t["w"], t["b"])
        dx, dw, db = _norm_backward(t["dy"].float(), t["x"].float(), t["w"], mean, rstd)
        act = _type(case)
        return dict(y=y.to(act), dx=dx.to(act), dw=dw, db=db)
    if case["op"] == "dropnorm":
        return _dropnorm(case, t)
    if case["op"] == "conv":
        return _conv(case, t)
    if case["op"] == "token":
        return _token(case, t)
    return _scan(case, t)


# ---- the plain forms -----------------------------------------------------------------------

def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _softplus(v):
    return torch.clamp(v, min=0.0) + torch.log1p(torch.exp(-torch.abs(v)))


def _norm(x, w, b):
    mean = x.mean(1, keepdim=True)
    c = x - mean
    rstd = torch.rsqrt((c * c).mean(1, keepdim=True) + EPS)
    return c * rstd * w + b, mean, rstd


def _norm_backward(dy, x, w, mean, rstd):
    xhat = (x - mean) * rstd
    g = dy * w
    dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    return dx, (dy * xhat).sum(0), dy.sum(0)


def _keep(rng, rows, n, p):
    """The dropout mask and its scale.  Eight columns share one call of the Philox 4x32 generator
    (ten rounds; Salmon, Moraes, Dror and Shaw, 2011): key = the seed, counter = (column / 8, row,
    offset's low and high half); column 8 i + j takes the j-th 16-bit piece of the result, lowest
    first, and is kept where that is at least round(65536 p)."""
    seed, offset = rng[0], rng[1]
    lo, hi = 0xFFFFFFFF, 32
    groups = (n + 7) // 8
    c0 = torch.arange(groups, device=rng.device).expand(rows, groups)
    c1 = torch.arange(rows, device=rng.device)[:, None].expand(rows, groups)
    c2 = (offset & lo).expand(rows, groups)
    c3 = ((offset >> hi) & lo).expand(rows, groups)
    k0, k1 = seed & lo, (seed >> hi) & lo

    def mul(a, m):  # 32 x 32 -> (high, low) in 64-bit signed integers
        high = ((a >> 16) * m + (((a & 0xFFFF) * m) >> 16)) >> 16
        low = ((((a >> 16) * m & 0xFFFF) << 16) + (a & 0xFFFF) * m) & lo
        return high, low

    for _ in range(10):
        h0, l0 = mul(c0, 0xD2511F53)
        h1, l1 = mul(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & lo, (k1 + 0xBB67AE85) & lo
    words = torch.stack([c0, c1, c2, c3], -1)
    pieces = torch.stack([words & 0xFFFF, words >> 16], -1).reshape(rows, groups * 8)[:, :n]
    cut = int(math.floor(p * 65536 + 0.5))
    return pieces >= cut, 65536.0 / (65536 - cut) if cut < 65536 else 0.0


def _dropnorm(case, t):
    act = _type(case)
    keep, scale = _keep(t["rng"], case["rows"], case["n"], case["p"])
    zero = torch.zeros((), device="cuda")
    s = (t["residual"].float() + torch.where(keep, t["x"].float() * scale, zero)).to(act)
    y, mean, rstd = _norm(s.float(), t["w"], t["b"])
    dx, dw, db = _norm_backward(t["dy"].float(), s.float(), t["w"], mean, rstd)
    dres = dx + t["ds"].float()
    return dict(s=s, y=y.to(act), dx=torch.where(keep, dres * scale, zero).to(act),
                dres=dres.to(act), dw=dw, db=db)


def _valid(lengths, K, B):
    """[K][B][1] truth values: step t of sequence b is before its end."""
    if lengths is None:
        return torch.ones(K, B, 1, dtype=torch.bool, device="cuda")
    return (torch.arange(K, device="cuda")[:, None] < lengths[None, :].long())[..., None]


def _conv(case, t):
    K, B, W, act = case["K"], case["B"], case["W"], _type(case)
    keep = _valid(t["lengths"], K, B)
    zero = torch.zeros((), device="cuda")
    xs = torch.cat([t["x0"].float().transpose(0, 1), t["x"].float()])  # [W - 1 + K][B][D]
    pre = t["bias"].expand(K, B, -1).clone()
    for j in range(W):
        pre += xs[j:j + K] * t["w"][:, j]
    sg = _sigmoid(pre)
    u = torch.where(keep, pre * sg, zero)
    # The last W - 1 inputs before each sequence's end, history included.
    end = torch.full((B,), K, device="cuda") if t["lengths"] is None else t["lengths"].long()
    at = end[:, None] + torch.arange(W - 1, device="cuda")[None, :]
    last = xs[at, torch.arange(B, device="cuda")[:, None]]
    g = torch.where(keep, t["dy"].float() * sg * (1.0 + pre * (1.0 - sg)), zero)
    dxs = torch.zeros_like(xs)
    dw = []
    for j in range(W):
        dxs[j:j + K] += g * t["w"][:, j]
        dw.append((g * xs[j:j + K]).sum((0, 1)))
    return dict(u=u.to(act), last=last.to(act), dx=dxs[W - 1:].to(act),
                dx0=dxs[:W - 1].transpose(0, 1).to(act), dw=torch.stack(dw, 1),
                dbias=g.sum((0, 1)))


def _token(case, t):
    act = _type(case)
    B, D, N, G = case["B"], case["D"], case["N"], case["G"]
    xs = torch.cat([t["x0"], t["x"][:, None]], 1)
    pre = t["bias"] + (xs.float() * t["w"].T).sum(1)
    u = (pre * _sigmoid(pre)).to(act)
    x = t["v"].float()
    d = _softplus(t["dt"].float() + t["dt_bias"])
    Bm = t["Bm"].float().repeat_interleave(D // G, 1)
    Cm = t["Cm"].float().repeat_interleave(D // G, 1)
    h = torch.exp(d[..., None] * t["A"]) * t["h0"] + (d * x)[..., None] * Bm
    z = t["z"].float()
    y = ((h * Cm).sum(-1) + t["D"] * x) * z * _sigmoid(z)
    return dict(u=u, conv_state=xs[:, 1:], y=y.to(act), h=h)


def _scan(case, t):
    """Steps are taken one after another, each one multiply-add over [B][D][N]; all that does not
    depend on the state is formed for a piece of steps at once."""
    K, B, D, N, G, act = case["K"], case["B"], case["D"], case["N"], case["G"], _type(case)
    E = D // G
    keep = _valid(t["lengths"], K, B)
    piece = max(1, min(K, (1 << 26) // (B * D * N)))
    raw = t["dt"].float() + t["dt_bias"]
    d = torch.where(keep, _softplus(raw), torch.zeros((), device="cuda"))
    x, z = t["x"].float(), t["z"].float()
    A = t["A"].view(G, E, N)
    sz = _sigmoid(z)

    def states(lo, hi, h):
        """exp(d A) and h_t for the steps lo .. hi - 1 from the state h before them."""
        dp = d[lo:hi].view(-1, B, G, E, 1)
        a = torch.exp(dp * A)
        hs = (dp * x[lo:hi].view(-1, B, G, E, 1)) * t["Bm"][lo:hi].float()[:, :, :, None, :]
        for k in range(hi - lo):
            h = hs[k].addcmul_(a[k], h)
        return a, hs

    y = torch.empty(K, B, D, device="cuda")  # before the gate
    starts, h = [], t["h0"].view(B, G, E, N)
    for lo in range(0, K, piece):
        starts.append(h)
        _, hs = states(lo, min(K, lo + piece), h)
        y[lo:lo + piece] = (hs * t["Cm"][lo:lo + piece].float()[:, :, :, None, :]).sum(-1).view(-1, B, D)
        h = hs[-1].clone()
    y = torch.where(keep, y + t["D"] * x, torch.zeros((), device="cuda"))
    out = dict(y=(y * z * sz).to(act), h=h.reshape(B, D, N))
    if not case["train"]:
        return out
    dy = torch.where(keep, t["dy"].float(), torch.zeros((), device="cuda"))
    out["dz"] = (dy * y * sz * (1.0 + z * (1.0 - sz))).to(act)
    g0 = dy * z * sz  # gradient of y before the gate
    dx, dd = torch.empty_like(x), torch.empty_like(x)
    dB, dC = torch.empty(K, B, G, N, device="cuda"), torch.empty(K, B, G, N, device="cuda")
    dA = torch.zeros(G, E, N, device="cuda")
    carry = torch.zeros(B, G, E, N, device="cuda")
    for lo in reversed(range(0, K, piece)):
        hi = min(K, lo + piece)
        before = starts.pop()
        a, hs = states(lo, hi, before)
        gp = g0[lo:hi].view(-1, B, G, E, 1)
        dC[lo:hi] = (hs * gp).sum(3)
        g = t["Cm"][lo:hi].float()[:, :, :, None, :] * gp  # becomes dL/dh_t
        for k in reversed(range(hi - lo)):
            g[k] += carry
            carry = a[k] * g[k]
        a[1:] *= hs[:-1]
        a[0] *= before
        a *= g  # dL/dh_t * exp(d A) h_{t-1}
        dp, xp = d[lo:hi].view(-1, B, G, E, 1), x[lo:hi].view(-1, B, G, E, 1)
        dA += (a * dp).sum((0, 1))
        gb = (g * t["Bm"][lo:hi].float()[:, :, :, None, :]).sum(-1, keepdim=True)
        dB[lo:hi] = (g * (dp * xp)).sum(3)
        dd[lo:hi] = ((a * A).sum(-1, keepdim=True) + xp * gb).view(-1, B, D)
        dx[lo:hi] = (dp * gb).view(-1, B, D)
    draw_ = torch.where(keep, dd * _sigmoid(raw), torch.zeros((), device="cuda"))
    out.update(dx=torch.where(keep, dx + t["D"] * g0, torch.zeros((), device="cuda")).to(act),
               ddt=draw_.to(act), dA=dA.view(D, N), dB=dB.to(act), dC=dC.to(act),
               dD=(g0 * x).sum((0, 1)), ddt_bias=draw_.sum((0, 1)), dh0=carry.reshape(B, D, N))
    return out


# ---- what a pass cannot do without ---------------------------------------------------------

def work(case):
    e = 4 if case["dtype"] == F32 else 2
    if case["op"] in ("norm", "dropnorm"):
        M, n = case["rows"], case["n"]
        if case["op"] == "norm":  # x, dy in; y, dx out; w, b, dw, db
            return dict(bytes=4 * M * n * e + 16 * n, flops=20 * M * n)
        # x, residual, dy, ds in; s, y, dx, dres out; the mask's integer work is not counted
        return dict(bytes=8 * M * n * e + 16 * n, flops=26 * M * n)
    if case["op"] == "conv":
        B, K, D, W = case["B"], case["K"], case["D"], case["W"]
        # x, dy in; u, dx out; the history and its gradient, in and out
        return dict(bytes=4 * K * B * D * e + 3 * B * (W - 1) * D * e + 8 * D * (W + 1),
                    flops=K * B * D * (6 * W + 25))
    B, D, N, G = case["B"], case["D"], case["N"], case["G"]
    if case["op"] == "token":
        W = case["W"]
        return dict(bytes=8 * B * D * N + B * D * e * (2 * (W - 1) + 6) + 2 * B * G * N * e
                    + 4 * D * (N + W + 3), flops=7 * B * D * N)
    K = case["K"]
    rows = K * B
    if not case["train"]:  # x, dt, z, B, C in; y out; the state in and out
        return dict(bytes=4 * rows * D * e + 2 * rows * G * N * e + 8 * B * D * N + 4 * D * (N + 2),
                    flops=7 * rows * D * N)
    # dy in, and dx, ddt, dz, dB, dC, dA, dD, ddt_bias, dh0 out beside the forward's
    return dict(bytes=8 * rows * D * e + 4 * rows * G * N * e + 12 * B * D * N + 8 * D * (N + 2),
                flops=24 * rows * D * N)


# ---- the definitions in 64 bits ------------------------------------------------------------

def _np(v):
    return None if v is None else v.double().cpu().numpy()


def _round_to(v, dtype):
    """float64 values rounded once to the activations' type (to nearest, ties to even)."""
    if dtype == F32:
        return v.astype(np.float32).astype(np.float64)
    m, e = np.frexp(v)  # 8 significant bits
    return np.ldexp(np.rint(m * 256.0), e - 8)


def _exact_mask(rng, rows, n, p):
    seed, offset = (int(v) % (1 << 64) for v in rng.cpu().tolist())
    low = np.uint64(0xFFFFFFFF)
    sh = np.uint64(32)
    ng = -(-n // 8)
    col, row = np.meshgrid(np.arange(ng, dtype=np.uint64), np.arange(rows, dtype=np.uint64))
    ctr = [col, row, np.full_like(col, offset & 0xFFFFFFFF), np.full_like(col, offset >> 32)]
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for r in range(10):
        pa, pb = ctr[0] * np.uint64(0xD2511F53), ctr[2] * np.uint64(0xCD9E8D57)
        ka = np.uint64((key[0] + r * 0x9E3779B9) & 0xFFFFFFFF)
        kb = np.uint64((key[1] + r * 0xBB67AE85) & 0xFFFFFFFF)
        ctr = [(pb >> sh) ^ ctr[1] ^ ka, pb & low, (pa >> sh) ^ ctr[3] ^ kb, pa & low]
    bits = np.stack(ctr, -1).astype("<u4").view("<u2").reshape(rows, ng * 8)[:, :n]
    cut = int(p * 65536 + 0.5)
    return bits >= cut, 65536.0 / (65536 - cut)


def _exact_norm(x, w, b, dy):
    mu = x.mean(axis=1, keepdims=True)
    inv = 1.0 / np.sqrt(x.var(axis=1, keepdims=True) + EPS)
    hat = (x - mu) * inv
    g = dy * w
    n = x.shape[1]
    dx = inv / n * (n * g - g.sum(1, keepdims=True) - hat * (g * hat).sum(1, keepdims=True))
    return hat * w + b, dx, np.einsum("ij,ij->j", dy, hat), dy.sum(0)


def exact(case, seed):
    op = case["op"]
    t = _inputs(case, seed)
    if op in ("norm", "dropnorm"):
        w, b, dy = _np(t["w"]), _np(t["b"]), _np(t["dy"])
        if op == "norm":
            y, dx, dw, db = _exact_norm(_np(t["x"]), w, b, dy)
            return dict(y=y, dx=dx, dw=dw, db=db)
        keep, scale = _exact_mask(t["rng"], case["rows"], case["n"], case["p"])
        s = _round_to(_np(t["residual"]) + keep * _np(t["x"]) * scale, case["dtype"])
        y, dx, dw, db = _exact_norm(s, w, b, dy)
        dres = dx + _np(t["ds"])
        return dict(s=s, y=y, dx=keep * dres * scale, dres=dres, dw=dw, db=db)
    B, D = case["B"], case["D"]
    if op == "conv":
        K, W = case["K"], case["W"]
        x, x0, w, dy = _np(t["x"]), _np(t["x0"]), _np(t["w"]), _np(t["dy"])
        ends = np.full(B, K) if t["lengths"] is None else t["lengths"].cpu().numpy()
        u, dx, last = np.zeros((K, B, D)), np.zeros((K, B, D)), np.zeros((B, W - 1, D))
        dx0, dw, dbias = np.zeros((B, W - 1, D)), np.zeros((D, W)), np.zeros(D)
        bias = _np(t["bias"])
        for i in range(B):
            L = int(ends[i])
            line = np.concatenate([x0[i], x[:L, i]], 0)  # line[W - 1 + t] = x_t
            last[i] = line[L:L + W - 1]
            if L == 0:
                continue
            pre = bias + sum(line[j:j + L] * w[:, j] for j in range(W))
            s = 0.5 * (1.0 + np.tanh(0.5 * pre))
            u[:L, i] = pre * s
            g = dy[:L, i] * (s + pre * s * (1.0 - s))
            dline = np.zeros_like(line)
            for j in range(W):
                dline[j:j + L] += g * w[:, j]
                dw[:, j] += np.einsum("td,td->d", g, line[j:j + L])
            dbias += g.sum(0)
            dx[:L, i], dx0[i] = dline[W - 1:], dline[:W - 1]
        return dict(u=u, last=last, dx=dx, dx0=dx0, dw=dw, dbias=dbias)
    N, G = case["N"], case["G"]
    group = np.arange(D) // (D // G)
    A, Dk, bias = _np(t["A"]), _np(t["D"]), _np(t["dt_bias"])

    def logistic(v):
        return 0.5 * (1.0 + np.tanh(0.5 * v))

    if op == "token":
        x0, x, w = _np(t["x0"]), _np(t["x"]), _np(t["w"])
        line = np.concatenate([x0, x[:, None]], 1)
        pre = _np(t["bias"]) + np.einsum("bjd,dj->bd", line, w)
        u = pre * logistic(pre)
        v = _np(t["v"])
        d = np.logaddexp(0.0, _np(t["dt"]) + bias)
        Bm, Cm, z = _np(t["Bm"])[:, group], _np(t["Cm"])[:, group], _np(t["z"])
        h = np.exp(d[..., None] * A) * _np(t["h0"]) + (d * v)[..., None] * Bm
        y = (np.einsum("bdn,bdn->bd", h, Cm) + Dk * v) * z * logistic(z)
        return dict(u=u, conv_state=line[:, 1:], y=y, h=h)
    K = case["K"]
    size = K * B * D * N
    if size > (60_000_000 if case["train"] else 300_000_000):
        return None
    ends = np.full(B, K) if t["lengths"] is None else t["lengths"].cpu().numpy()
    x, raw, z = _np(t["x"]), _np(t["dt"]) + bias, _np(t["z"])
    Bm, Cm = _np(t["Bm"]), _np(t["Cm"])
    d = np.logaddexp(0.0, raw)
    gate = z * logistic(z)
    h, y = _np(t["h0"]).copy(), np.zeros((K, B, D))
    kept = [h.copy()] if case["train"] else None
    for k in range(K):
        on = k < ends
        new = np.exp(d[k][..., None] * A) * h + (d[k] * x[k])[..., None] * Bm[k][:, group]
        h = new if on.all() else np.where(on[:, None, None], new, h)
        y[k] = on[:, None] * (np.einsum("bdn,bdn->bd", h, Cm[k][:, group]) + Dk * x[k])
        if kept is not None:
            kept.append(h)
    out = dict(y=y * gate, h=h)
    if not case["train"]:
        return out
    dy = _np(t["dy"]) * (np.arange(K)[:, None] < ends)[..., None]
    sz = logistic(z)
    dz = dy * y * (sz + z * sz * (1.0 - sz))
    dx, ddt, dA = np.zeros((K, B, D)), np.zeros((K, B, D)), np.zeros((D, N))
    dB, dC = np.zeros((K, B, G, N)), np.zeros((K, B, G, N))
    dD = np.zeros(D)
    r = np.zeros((B, D, N))  # dL/dh carried back
    for k in reversed(range(K)):
        on = (k < ends)[:, None, None]
        q = dy[k] * gate[k]
        full = r + q[..., None] * Cm[k][:, group]
        a = np.exp(d[k][..., None] * A)
        dC[k] = (q[..., None] * kept[k + 1]).reshape(B, G, D // G, N).sum(2) * on
        ga = full * a * kept[k] * on
        dA += (ga * d[k][..., None]).sum(0)
        fb = np.einsum("bdn,bdn->bd", full * on, Bm[k][:, group])
        dB[k] = (full * on * (d[k] * x[k])[..., None]).reshape(B, G, D // G, N).sum(2)
        ddt[k] = ((ga * A).sum(-1) + x[k] * fb) * logistic(raw[k])
        dx[k] = d[k] * fb + Dk * q
        dD += (q * x[k]).sum(0)
        r = np.where(on, a * full, r)
    out.update(dz=dz, dx=dx, ddt=ddt, dA=dA, dB=dB, dC=dC, dD=dD, ddt_bias=ddt.sum((0, 1)), dh0=r)
    return out
