"""What is measured of the gated block's operators (root-mean-square norm with the residual sum,
values in 8 bits, the gated linear recurrence, products with 4-bit weights): cases, inputs, a plain
form in elementary torch operations, the framework's calls, and a 64-bit form of the definitions.

Layouts follow the recurrent path: sequences are time-major [K][B][D], activations are fp32 or
bf16, parameters, statistics and states are fp32.

  norm      s = x + residual, rounded to the activations' type; y = s * rstd * w with
            rstd = (mean s^2 + eps)^-1/2; backward from dy and the stream's own gradient ds:
            dx (of both summands), dw.
  norm8     the same forward pass with y held in 8 bits, and the values that it then stands for.
  keepnorm  norm, with s kept in 8 bits (and rstd) for the backward pass, which also forms y again.
  gated     f_t = sigmoid(f_t + bias);  h_t = f_t h_{t-1} + (1 - f_t) x_t;
            y_t = h_t silu(z_t) (without z: h_t); backward: every input's gradient.  With `keep`
            the backward pass reads x, f and z as kept in 8 bits and takes h up again from the
            states of every 8th step; it also forms y again.
  gtoken    one step of the recurrence, for single tokens.
  q4        y = x W^T with W = (code - 8) * scale, codes of 4 bits, a scale for each `group`
            columns of a row.

8 bits: blocks of 32 columns of a row (the last may be shorter) share the smallest power of two 2^k,
k >= -126, with max |v| <= 448 * 2^k; a value is held as v / 2^k rounded to e4m3.

A sequence of length L < K ends at L: later outputs and gradients are 0 and its state stays.
"""
import math

import torch

own = False

F32, BF16 = "f32", "bf16"
EPS = 1e-5
BLOCK = 32   # columns that share a scale in 8 bits
PERIOD = 8   # steps between the states that the recurrence keeps


# ---- cases ---------------------------------------------------------------------------------

def listed():
    return [
        # The smallest workload's rows (4 sequences x 8 steps, 32 channels): latency alone.
        dict(name="norm_f32_tiny", op="norm", rows=32, n=32, dtype=F32),
        # The stress workload's rows (2048 sequences x 128 steps, 256 channels): streaming.
        dict(name="norm_bf16_stress", op="norm", rows=262144, n=256, dtype=BF16),
        # Wide rows of an odd width, so that no row but the first starts aligned.
        dict(name="norm_bf16_odd", op="norm", rows=9001, n=1537, dtype=BF16),
        # The norm in front of products on 8-bit rows, a prompt's worth of wide rows.
        dict(name="norm8_bf16_wide", op="norm8", rows=16384, n=2048, dtype=BF16),
        # Training at the stress workload's rows with the stream kept in 8 bits.
        dict(name="keepnorm_f32_stress", op="keepnorm", rows=262144, n=256, dtype=F32),
        # One long prompt: few channels, a long axis.
        dict(name="gated_prompt_bf16_long", op="gated", train=False, keep=False, B=1, K=32768,
             D=1024, z=True, ragged=False, dtype=BF16),
        # Training at the 32 x 64 workload, no output gate.
        dict(name="gated_train_f32_pages", op="gated", train=True, keep=False, B=32, K=64, D=256,
             z=False, ragged=False, dtype=F32),
        # Training on a large batch of sequences of different lengths, an odd number of steps.
        dict(name="gated_train_bf16_ragged", op="gated", train=True, keep=False, B=64, K=1023,
             D=1536, z=True, ragged=True, dtype=BF16),
        # Training on long sequences whose activations are kept in 8 bits.
        dict(name="gated_keep_bf16_long", op="gated", train=True, keep=True, B=16, K=2048, D=2048,
             z=True, ragged=False, dtype=BF16),
        # Serving, a full batch, one token each: the state's traffic.
        dict(name="gtoken_bf16_batch", op="gtoken", B=1024, D=2048, z=True, dtype=BF16),
        # Serving, one sequence: a wide projection's weights are read once for one token.
        dict(name="q4_bf16_one", op="q4", M=1, N=16384, K=4096, group=128, dtype=BF16),
        # Serving, a few sequences, a small projection of odd sizes.
        dict(name="q4_f32_few", op="q4", M=5, N=1537, K=1000, group=32, dtype=F32),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm8", "keepnorm", "prompt", "train", "keep", "gtoken", "q4"])
    dtype = rng.choice([F32, BF16])
    while True:
        if op in ("norm", "norm8", "keepnorm"):
            c = dict(op=op, rows=_log_int(rng, 1, 262144), n=_log_int(rng, 8, 8192), dtype=dtype)
            if 4096 <= c["rows"] * c["n"] <= 1 << 25:
                return c
            continue
        if op == "q4":
            c = dict(op=op, M=_log_int(rng, 1, 32), N=_log_int(rng, 64, 16384),
                     K=_log_int(rng, 64, 8192), group=rng.choice([32, 64, 128]), dtype=dtype)
            if 16384 <= c["N"] * c["K"] <= 1 << 26:
                return c
            continue
        D, z = rng.choice([1, 2, 4, 8]) * _log_int(rng, 16, 256), rng.random() < 0.7
        if op == "gtoken":
            c = dict(op=op, B=_log_int(rng, 1, 2048), D=D, z=z, dtype=dtype)
            if 4096 <= c["B"] * D <= 1 << 21:
                return c
            continue
        c = dict(op="gated", train=op != "prompt", keep=op == "keep",
                 B=_log_int(rng, 1, 8 if op == "prompt" else 256),
                 K=_log_int(rng, 16, 32768 if op == "prompt" else 4096), D=D, z=z,
                 ragged=rng.random() < 0.5, dtype=dtype)
        if 65536 <= c["B"] * c["K"] * D <= 60_000_000:
            return c


# ---- inputs --------------------------------------------------------------------------------

def _type(case):
    return torch.float32 if case["dtype"] == F32 else torch.bfloat16


def _inputs(case, seed):
    """The inputs of a case, on the GPU, from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    act, op = _type(case), case["op"]

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda").mul_(std).add_(mean).to(dtype)

    if op in ("norm", "norm8", "keepnorm"):
        M, n = case["rows"], case["n"]
        t = dict(x=normal(M, n, std=0.7, dtype=act), residual=normal(M, n, std=2.0, dtype=act),
                 w=normal(n, std=0.2, mean=1.0))
        if op != "norm8":
            t.update(dy=normal(M, n, dtype=act), ds=normal(M, n, dtype=act))
        return t
    if op == "q4":
        M, N, K, group = case["M"], case["N"], case["K"], case["group"]
        # Codes as a file of 4-bit weights holds them: column 2 i in the low half of byte i.
        t = dict(codes=torch.randint(0, 256, (N, (K + 1) // 2), generator=g, device="cuda",
                                     dtype=torch.uint8),
                 scales=(torch.rand(N, -(-K // group), generator=g, device="cuda") * 0.01
                         + 0.002).bfloat16(), x=normal(M, K, dtype=act))
        return t
    B, D = case["B"], case["D"]
    bias = torch.rand(D, generator=g, device="cuda") * 5.0  # memories of a few to 200 steps
    if op == "gtoken":
        xfz = normal(B, 3 * D, dtype=act)  # x, f and z come out of one projection
        return dict(x=xfz[:, :D], f=xfz[:, D:2 * D], z=xfz[:, 2 * D:] if case["z"] else None,
                    bias=bias, h0=normal(B, D, std=0.5))
    K = case["K"]
    xfz = normal(K, B, 3 * D, dtype=act)
    t = dict(x=xfz[..., :D], f=xfz[..., D:2 * D], z=xfz[..., 2 * D:] if case["z"] else None,
             bias=bias, h0=normal(B, D, std=0.5), lengths=None)
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
        if op in ("norm", "norm8", "keepnorm"):
            step = trunk.RMSNormStep(case["rows"], case["n"], dtype=act, eps=EPS,
                                     out8=op == "norm8", keep8=op == "keepnorm")
            state["step"] = step.bind(x=t["x"], w=t["w"], residual=t["residual"], dy=t.get("dy"),
                                      ds=t.get("ds"))
            if op == "norm8":
                state["values"] = trunk.Unpack8Step(case["rows"], case["n"], dtype=act).bind(
                    step.y8)
        elif op == "q4":
            weights = trunk.Weights4(t["codes"], t["scales"], case["K"], case["group"])
            state["step"] = trunk.MatvecStep(case["M"], weights, dtype=act).bind(t["x"])
        elif op == "gtoken":
            state["step"] = trunk.GatedToken(case["B"], case["D"], dtype=act).bind(
                x=t["x"], f=t["f"], bias=t["bias"], z=t["z"], state=t["h0"],
                new_state=torch.empty_like(t["h0"]))
        else:
            state["step"] = trunk.GatedStep(case["K"], case["B"], case["D"], dtype=act,
                                            train=case["train"], keep8=case["keep"]).bind(
                x=t["x"], f=t["f"], bias=t["bias"], z=t["z"], h0=t["h0"], lengths=t["lengths"],
                dy=t.get("dy"))
    return state


# ---- one pass ------------------------------------------------------------------------------

def run(state):
    case, t = state["case"], state["t"]
    op = case["op"]
    if own:
        if op == "gtoken":
            y, h = state["step"].run()
            return dict(y=y, h=h)
        state["step"].run()
        if op == "norm8":
            return dict(s=state["step"].s, y=state["values"].run())
        return state["step"].outputs()
    if op in ("norm", "norm8", "keepnorm"):
        return _norm(case, t)
    if op == "q4":
        return dict(y=(t["x"].float() @ _weights4(case, t).T).to(_type(case)))
    if op == "gtoken":
        v = t["f"].float() + t["bias"]
        h = _sigmoid(v) * t["h0"] + _sigmoid(-v) * t["x"].float()
        return dict(y=(h * _gate(t["z"])).to(_type(case)), h=h)
    return _gated(case, t)


# ---- the plain forms -----------------------------------------------------------------------

def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _gate(z):
    return 1.0 if z is None else z.float() * _sigmoid(z.float())


def _held8(v):
    """What fp32 values [..][n] stand for once they are held in 8 bits."""
    n = v.shape[-1]
    pad = -n % BLOCK
    if pad:
        v = torch.cat([v, torch.zeros(*v.shape[:-1], pad, device=v.device)], -1)
    blocks = v.unflatten(-1, (-1, BLOCK))
    m, e = torch.frexp(blocks.abs().amax(-1, keepdim=True))  # max |v| = m 2^e, m in [1/2, 1)
    k = torch.clamp(torch.where(m > 0.875, e - 8, e - 9), min=-126)  # 448 = 0.875 * 2^9
    up, down = ((k + 127) << 23).view(torch.float32), ((127 - k) << 23).view(torch.float32)
    held = (blocks * down).to(torch.float8_e4m3fn).float() * up
    return held.flatten(-2)[..., :n]


def _norm(case, t):
    act, w = _type(case), t["w"]
    s = (t["x"].float() + t["residual"].float()).to(act)
    v = s.float()
    rstd = torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)
    y = v * rstd * w
    if case["op"] == "norm8":
        return dict(s=s, y=_held8(y).to(act))
    out = dict(s=s, y=y.to(act))
    if case["op"] == "keepnorm":
        v = _held8(v)
        out["y_again"] = (v * rstd * w).to(act)
    hat = v * rstd
    dy = t["dy"].float()
    g = dy * w
    dx = rstd * (g - hat * (g * hat).mean(1, keepdim=True)) + t["ds"].float()
    out.update(dx=dx.to(act), dw=(dy * hat).sum(0))
    return out


def _weights4(case, t):
    N, K, group = case["N"], case["K"], case["group"]
    codes = torch.stack([t["codes"] & 15, t["codes"] >> 4], -1).view(N, -1)[:, :K]
    scales = t["scales"].float().repeat_interleave(group, 1)[:, :K]
    return (codes.float() - 8.0) * scales


def _recurrence(a, b, dim):
    """h_t = a_t h_{t-1} + b_t along a dimension, h_{-1} = 0, by doubling the steps that a term spans."""
    K, span = a.shape[dim], 1
    while span < K:
        ahead, rest = a.narrow(dim, 0, span), a.narrow(dim, span, K - span)
        b = torch.cat([b.narrow(dim, 0, span),
                       b.narrow(dim, span, K - span) + rest * b.narrow(dim, 0, K - span)], dim)
        a = torch.cat([ahead, rest * a.narrow(dim, 0, K - span)], dim)
        span *= 2
    return b


def _gated(case, t):
    K, B, D, act = case["K"], case["B"], case["D"], _type(case)
    on = torch.ones(K, B, 1, dtype=torch.bool, device="cuda")
    if t["lengths"] is not None:
        on = (torch.arange(K, device="cuda")[:, None] < t["lengths"][None, :].long())[..., None]
    zero, one = torch.zeros((), device="cuda"), torch.ones((), device="cuda")

    def gates(logits):
        v = logits + t["bias"]
        return torch.where(on, _sigmoid(v), one), torch.where(on, _sigmoid(-v), zero)

    x, h0 = t["x"].float(), t["h0"]
    f, i = gates(t["f"].float())
    b = i * x
    b[0] += f[0] * h0
    h = _recurrence(f, b, 0)
    out = dict(y=torch.where(on, h * _gate(t["z"]), zero).to(act), h=h[-1].clone())
    if not case["train"]:
        return out
    before = torch.cat([h0[None], h[:-1]])
    z = None if t["z"] is None else t["z"].float()
    if case["keep"]:
        x, z = _held8(x), None if z is None else _held8(z)
        f, i = gates(_held8(t["f"].float()))
        periods = -(-K // PERIOD)
        rest = periods * PERIOD - K
        b = torch.cat([i * x, torch.zeros(rest, B, D, device="cuda")])
        a = torch.cat([f, torch.ones(rest, B, D, device="cuda")])
        starts = before[::PERIOD]
        b[::PERIOD] += a[::PERIOD] * starts
        h = _recurrence(a.view(periods, PERIOD, B, D), b.view(periods, PERIOD, B, D), 1)
        before = torch.cat([starts[:, None], h[:, :-1]], 1).view(-1, B, D)[:K]
        h = h.view(-1, B, D)[:K]
        out["y_again"] = torch.where(on, h * _gate(z), zero).to(act)
    dy = torch.where(on, t["dy"].float(), zero)
    # dL/dh_t = dy_t gate_t + f_{t+1} dL/dh_{t+1}, from the last step to the first
    later = torch.cat([torch.ones(1, B, D, device="cuda"), f[1:].flip(0)])
    g = _recurrence(later, (dy * _gate(z)).flip(0), 0).flip(0)
    df = g * (before - x) * f * i
    if z is not None:
        sz = _sigmoid(z)
        out["dz"] = (dy * h * sz * (1.0 + z * (1.0 - sz))).to(act)
    out.update(dx=(g * i).to(act), df=df.to(act), dbias=df.sum((0, 1)), dh0=g[0] * f[0])
    return out


# ---- what a pass cannot do without ---------------------------------------------------------

def work(case):
    e = 4 if case["dtype"] == F32 else 2
    op, held = case["op"], 1 + 1 / BLOCK
    if op in ("norm", "norm8", "keepnorm"):
        M, n = case["rows"], case["n"]
        if op == "norm8":  # x, residual in; s and the values out, which are held in 8 bits
            return dict(bytes=M * n * (4 * e + held) + 4 * n, flops=8 * M * n)
        if op == "norm":  # x, residual, dy, ds in; s, y, dx out
            return dict(bytes=7 * M * n * e + 8 * n, flops=15 * M * n)
        # y again out as well; s kept, then read
        return dict(bytes=M * n * (8 * e + 2 * held) + 8 * n, flops=20 * M * n)
    if op == "q4":
        M, N, K = case["M"], case["N"], case["K"]
        return dict(bytes=N * ((K + 1) // 2) + 2 * N * -(-K // case["group"]) + M * (K + N) * e,
                    flops=2 * M * N * K)
    B, D, z = case["B"], case["D"], int(case["z"])
    if op == "gtoken":  # x, f, z and the state in; y and the state out
        return dict(bytes=B * D * (8 + (3 + z) * e) + 4 * D, flops=12 * B * D)
    steps = case["K"] * B * D
    if not case["train"]:
        return dict(bytes=steps * (3 + z) * e + 8 * B * D + 4 * D, flops=12 * steps)
    # and dy in; dx, df, dz out; the initial state's and the bias's gradients
    moved = steps * (6 + 2 * z) * e + 12 * B * D + 8 * D
    if case["keep"]:  # x, f and z kept, then read; y again out
        moved += steps * (2 * (2 + z) * held + e)
    return dict(bytes=moved, flops=35 * steps)


# ---- the definitions in 64 bits ------------------------------------------------------------

def _exact_type(v, dtype):
    """float64 values rounded once to the activations' type."""
    return v.to(torch.float32 if dtype == F32 else torch.bfloat16).double()


def _power(k):
    """2^k as float64, for whole k in -1022 .. 1023."""
    return (k.long() + 1023 << 52).view(torch.float64)


def _magnitude(v):
    """The largest whole k with 2^k <= v, for normal float64 values."""
    return (v.contiguous().view(torch.int64) >> 52) - 1023


def _exact_held8(v):
    """float64 values as they are held in 8 bits: three bits after the leading one, the smallest
    steps 2^-9, in units of the block's power of two."""
    held = torch.empty_like(v)
    for c in range(0, v.shape[-1], BLOCK):
        part = v[..., c:c + BLOCK]
        top = part.abs().max(-1, keepdim=True).values.clamp(min=2.0 ** -200)
        k = _magnitude(top) - 8  # top < 512 * 2^k
        k = torch.where(448.0 * _power(k) < top, k + 1, k)
        k = torch.where(448.0 * _power(k - 1) >= top, k - 1, k).clamp(min=-126)
        u = part * _power(-k)
        step = _power(_magnitude(u.abs().clamp(min=2.0 ** -6)) - 3)
        held[..., c:c + BLOCK] = torch.round(u / step) * step * _power(k)
    return held


def _logistic(v):
    return 0.5 + 0.5 * torch.tanh(0.5 * v)


def exact(case, seed):
    t = {k: v.double() if v is not None and v.is_floating_point() else v
         for k, v in _inputs(case, seed).items()}
    op, dtype = case["op"], case["dtype"]
    if op in ("norm", "norm8", "keepnorm"):
        n, w = case["n"], t["w"]
        s = _exact_type(t["x"] + t["residual"], dtype)
        scale = torch.sqrt(n / ((s * s).sum(1) + n * EPS))[:, None]
        y = s * scale * w
        if op == "norm8":
            return dict(s=s, y=_exact_held8(y))
        out = dict(s=s, y=y)
        if op == "keepnorm":
            s = _exact_held8(s)
            out["y_again"] = s * scale * w
        inner = torch.einsum("ij,ij,j->i", t["dy"], s, w)[:, None]
        out.update(dx=t["ds"] + scale * w * t["dy"] - scale ** 3 / n * inner * s,
                   dw=torch.einsum("ij,ij,ik->j", t["dy"], s, scale))
        return out
    if op == "q4":
        N, K, group, M = case["N"], case["K"], case["group"], case["M"]
        y = torch.zeros(M, N, dtype=torch.float64, device="cuda")
        for c in range(0, K, group):
            cols = torch.arange(c, min(K, c + group), device="cuda")
            code = (t["codes"][:, cols // 2].long() >> (4 * (cols % 2))) % 16 - 8
            y += (t["x"][:, cols] @ code.double().T) * t["scales"][:, c // group]
        return dict(y=y)
    bias, h = t["bias"], t["h0"]

    def swish(z):
        return 1.0 if z is None else z * _logistic(z)

    if op == "gtoken":
        f = _logistic(t["f"] + bias)
        h = f * h + (1.0 - f) * t["x"]
        return dict(y=h * swish(t["z"]), h=h)
    K, B = case["K"], case["B"]
    x, f, z = t["x"], t["f"], t["z"]
    ends = torch.full((B,), K, device="cuda") if t["lengths"] is None else t["lengths"]
    h = h.clone()
    y, states = torch.zeros_like(x), []
    for k in range(K):
        on = (k < ends)[:, None]
        states.append(h)
        a = _logistic(f[k] + bias)
        h = torch.where(on, x[k] + a * (h - x[k]), h)
        y[k] = torch.where(on, h * swish(None if z is None else z[k]), 0.0)
    out = dict(y=y, h=h)
    if not case["train"]:
        return out
    if case["keep"]:
        x, f, z = _exact_held8(x), _exact_held8(f), None if z is None else _exact_held8(z)
        again = torch.zeros_like(x)
        for k in range(K):
            if k % PERIOD == 0:
                h = states[k]
            states[k] = h
            a = _logistic(f[k] + bias)
            h = torch.where((k < ends)[:, None], x[k] + a * (h - x[k]), h)
            again[k] = torch.where((k < ends)[:, None], h * swish(None if z is None else z[k]), 0.0)
        out["y_again"] = again
    dx, df, dz = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    carry = torch.zeros_like(h)
    for k in reversed(range(K)):
        on = (k < ends)[:, None]
        a = _logistic(f[k] + bias)
        g = carry + t["dy"][k] * swish(None if z is None else z[k])
        dx[k] = torch.where(on, g * (1.0 - a), 0.0)
        df[k] = torch.where(on, g * (states[k] - x[k]) * a * (1.0 - a), 0.0)
        if z is not None:
            s = _logistic(z[k])
            now = x[k] + a * (states[k] - x[k])
            dz[k] = torch.where(on, t["dy"][k] * now * (s + z[k] * s * (1.0 - s)), 0.0)
        carry = torch.where(on, g * a, carry)
    if z is not None:
        out["dz"] = dz
    out.update(dx=dx, df=df, dbias=df.sum((0, 1)), dh0=carry)
    return out
