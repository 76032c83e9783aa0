"""The trunk of gated blocks (the gated block's operators and the cell together): its gradients
against float64 autograd of the same trunk, with what is kept in 8 bits against the float64 oracle on
the kept values, and serving on 4-bit weights token by token against the prompt and against float64."""
import numpy as np
import pytest

import oracle.gated as og

pytestmark = pytest.mark.gpu

# A layer is four operators in a row, each within 1e-5 of its exact result in fp32 (the single
# operators' tests); two layers, the last norm and the cell are ten.  Gradients are 1e-4 each way, as
# the single operators', over twice as many.
OUT_TOL, GRAD_TOL = 1e-4, 1e-3
K, B, D, E, C = 19, 3, 24, 40, 32


@pytest.fixture(scope="module", autouse=True)
def built():
    import torch

    from recurrent_cfc_cell_gb300 import build

    build.build()
    torch.backends.cuda.matmul.allow_tf32 = False


def close(x, y, tol, name=""):
    import torch

    y = torch.as_tensor(y, dtype=torch.float64)
    err = (x.double().cpu() - y).abs().max()
    assert err <= tol * y.abs().max(), f"{name}: {err:.3g} of {y.abs().max():.3g}"


def rms(v, w):
    import torch

    return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + 1e-5) * w


def trunk64(P, s, ends):
    """The trunk up to the last norm in float64 torch operations, for autograd."""
    import torch

    on = (torch.arange(s.shape[0])[:, None] < torch.as_tensor(ends))[..., None]
    o = None
    for p in P["layers"]:
        s = s if o is None else s + o
        x, f, z = (rms(s, p["w"]) @ p["W_in"].T).chunk(3, -1)
        h, ys = torch.zeros(x.shape[1:], dtype=s.dtype), []
        for t in range(s.shape[0]):
            g = torch.sigmoid(f[t] + p["bias"])
            h = torch.where(on[t], g * h + (1 - g) * x[t], h)
            ys.append(torch.where(on[t], h * torch.nn.functional.silu(z[t]), 0.0))
        o = torch.stack(ys) @ p["W_out"].T
    return rms(s + o, P["w"])


def cell64(P, n, h, ts):
    import torch

    H = []
    for t in range(n.shape[0]):
        pre = torch.einsum("gcn,bn->gbc", P["cell_W"], torch.cat([n[t], h], -1)) + P["cell_b"][:, None]
        gate = torch.sigmoid(pre[2] * ts[t][:, None] + pre[3])
        h = torch.tanh(pre[0]) * (1 - gate) + gate * torch.tanh(pre[1])
        H.append(h)
    return torch.stack(H)


def inputs(seed=3):
    import torch

    g = torch.Generator().manual_seed(seed)
    r = lambda *n: torch.randn(*n, generator=g)  # noqa: E731
    return dict(s=r(K, B, D), h0=r(B, C) * 0.1, ts=torch.rand(K, B, generator=g) + 0.5, dH=r(K, B, C))


def double(P, grad=False):
    f = lambda v: v.double().cpu().requires_grad_(grad)  # noqa: E731
    return {k: [{n: f(t) for n, t in p.items()} for p in v] if k == "layers" else f(v)
            for k, v in P.items()}


def test_trunk_gradients():
    import torch

    from recurrent_cfc_cell_gb300.gated_block import GatedTrunk, make_gated_params

    P = make_gated_params(2, D, E, C, seed=1)
    i, ends = inputs(), [19, 4, 0]
    trunk = GatedTrunk(K, B, P)
    H = trunk.forward(i["s"].cuda(), i["h0"].cuda(), i["ts"].cuda(),
                      torch.tensor(ends, dtype=torch.int32).cuda())
    R = double(P, True)
    s, h0 = i["s"].double().requires_grad_(True), i["h0"].double().requires_grad_(True)
    want = cell64(R, trunk64(R, s, ends), h0, i["ts"].double())
    close(H, want.detach(), OUT_TOL, "H")
    got = trunk.backward(i["dH"].cuda())
    (want * i["dH"].double()).sum().backward()
    for name in ("w", "cell_W", "cell_b"):
        close(got[name], R[name].grad, GRAD_TOL, name)
    close(got["ds"], s.grad, GRAD_TOL, "ds")
    close(got["dh0"], h0.grad, GRAD_TOL, "dh0")
    for k, (a, b) in enumerate(zip(got["layers"], R["layers"])):
        for name in ("w", "W_in", "bias", "W_out"):
            close(a[name], b[name].grad, GRAD_TOL, f"{name} of layer {k}")


def test_trunk_kept_in_8_bits():
    """The forward pass is the same, bit by bit; the gradients are the oracle's on the kept values,
    from the activations that the trunk that keeps everything has."""
    import torch

    from recurrent_cfc_cell_gb300.gated_block import GatedTrunk, make_gated_params

    P = make_gated_params(2, D, E, C, seed=2)
    i = inputs(4)
    args = (i["s"].cuda(), i["h0"].cuda(), i["ts"].cuda())
    full, kept = GatedTrunk(K, B, P), GatedTrunk(K, B, P, keep8=True)
    H = full.forward(*args)
    before = args[0].clone()
    assert torch.equal(kept.forward(*args), H) and torch.equal(args[0], before)
    got = kept.backward(i["dH"].cuda())
    full.backward(i["dH"].cuda())
    n64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    g = n64(full.last.dx)  # from the cell and the last norm, which keep all they need
    close(kept.last.dx, g, GRAD_TOL, "last norm")
    rows, ends = K * B, np.full(B, K)
    for k in (1, 0):
        p = {n: n64(t) for n, t in P["layers"][k].items()}
        x, f, z = np.split(n64(full.xfz[k]), 3, axis=-1)
        dy = (g @ p["W_out"]).reshape(K, B, E)
        out, y = og.gated_backward(dy, x, f, p["bias"], z, np.zeros((B, E)), ends, kept=True)
        close(got["layers"][k]["W_out"], g.T @ y.reshape(rows, E), GRAD_TOL, f"W_out {k}")
        close(got["layers"][k]["bias"], out["dbias"], GRAD_TOL, f"bias {k}")
        dxfz = np.concatenate([out[n] for n in ("dx", "df", "dz")], -1).reshape(rows, 3 * E)
        norm = full.norms[k]
        stream = n64(norm.inputs["x"] if k == 0 else norm.s)
        g, dw, n = og.rmsnorm_backward(dxfz @ p["W_in"], stream, p["w"], 1e-5, og.held8(stream), g)
        close(got["layers"][k]["W_in"], dxfz.T @ n, GRAD_TOL, f"W_in {k}")
        close(got["layers"][k]["w"], dw, GRAD_TOL, f"w {k}")
    close(got["ds"], g.reshape(K, B, D), GRAD_TOL, "ds")


def test_serving():
    """A prompt in two parts and tokens behind it, against float64 on the weights that 4 bits hold."""
    import torch

    from recurrent_cfc_cell_gb300.gated_block import GatedServe, make_gated_params
    from recurrent_cfc_cell_gb300.trunk import Weights4

    P = make_gated_params(2, D, E, C, seed=5)
    s = inputs(6)["s"].cuda()
    serve = GatedServe(B, P, group=32)
    parts = [serve.prompt(s[:9]), serve.prompt(s[9:12])]
    parts += [serve.token(s[t])[None] for t in range(12, K)]
    R = double(P)
    for p, q in zip(R["layers"], P["layers"]):
        for n in ("W_in", "W_out"):
            codes, scales = Weights4.quantized(q[n], 32)
            p[n] = torch.from_numpy(og.weights4(codes.cpu().numpy(), scales.double().cpu().numpy(),
                                                q[n].shape[1], 32))
    close(torch.cat(parts), trunk64(R, s.double().cpu(), [K] * B), OUT_TOL)
    first = parts[3].clone()
    serve.token(s[0])
    assert torch.equal(parts[3], first)  # a token's result is its own
