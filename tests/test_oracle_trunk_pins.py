"""The trunk operators' fp64 oracle pinned to facts outside it: published vectors of the counter-
based generator, central differences of its own forward passes, torch's layer norm, convolution
and autograd, and identities of the scan."""
import numpy as np
import pytest
import torch

import oracle.trunk as ot
from trunk_cases import conv_inputs, norm_inputs, scan_inputs

# Central differences in fp64 with step h: truncation ~ h^2 |f'''| / 6 and rounding ~ 2^-53 |f| / h;
# h = 1e-5 leaves both near 1e-10 for sums of a few hundred terms of order one.
H, FD_TOL = 1e-5, 1e-7


def differences(f, x):
    g = np.zeros_like(x)
    flat, out = x.reshape(-1), g.reshape(-1)
    for i in range(flat.size):
        v = flat[i]
        flat[i] = v + H
        up = f()
        flat[i] = v - H
        out[i] = (up - f()) / (2 * H)
        flat[i] = v
    return g


def close(a, b):
    assert np.max(np.abs(a - b)) <= FD_TOL * max(1.0, np.max(np.abs(b)))


def test_philox_known_answers():
    """Known-answer vectors published with the generator (philox4x32-10)."""
    f = 0xFFFFFFFF
    assert ot.philox4x32((0, 0, 0, 0), (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert ot.philox4x32((f, f, f, f), (f, f)) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]


def test_dropout_rate_and_expectation():
    kept, scale = ot.dropout_mask(200, 300, 0.25, 7, 11)
    q = 1.0 - 1.0 / scale
    assert abs(q - 0.25) <= 2.0 ** -17
    # 60000 independent draws: 5 standard deviations
    assert abs(kept.mean() - (1 - q)) <= 5 * np.sqrt(q * (1 - q) / kept.size)
    assert ot.dropout_mask(3, 5, 0.0, 1, 2)[0].all()
    assert not ot.dropout_mask(3, 5, 1.0, 1, 2)[0].any()


def test_layernorm_against_torch_and_differences():
    i = norm_inputs(4, 7, "f32", 1)
    t = {k: torch.tensor(v, requires_grad=k in "xwb") for k, v in i.items()}
    y = torch.nn.functional.layer_norm(t["x"], (7,), t["w"], t["b"], 1e-5)
    y.backward(t["dy"])
    close(ot.layernorm(i["x"], i["w"], i["b"], 1e-5), y.detach().numpy())
    dx, dw, db = ot.layernorm_backward(i["dy"], i["x"], i["w"], 1e-5)
    for got, k in ((dx, "x"), (dw, "w"), (db, "b")):
        close(got, t[k].grad.numpy())
        close(got, differences(lambda: (ot.layernorm(i["x"], i["w"], i["b"], 1e-5) * i["dy"]).sum(), i[k]))


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("silu", [True, False])
def test_conv_against_torch_and_differences(W, silu):
    K, B, D = 5, 2, 3
    i = conv_inputs(K, B, D, W, "f32", W)
    ends = [K, K]
    u, last = ot.conv(i["x"], i["w"], i["bias"], i["x0"], ends, silu)
    line = torch.tensor(np.concatenate([i["x0"].transpose(1, 0, 2), i["x"]])).permute(1, 2, 0)
    p = torch.nn.functional.conv1d(line, torch.tensor(i["w"])[:, None], torch.tensor(i["bias"]), groups=D)
    want = (torch.nn.functional.silu(p) if silu else p).permute(2, 0, 1).numpy()
    close(u, want)
    assert np.array_equal(last, line[:, :, K:].permute(0, 2, 1).numpy())
    ends = [K, 3]
    grads = ot.conv_backward(i["du"], i["x"], i["w"], i["bias"], i["x0"], ends, silu)
    for got, k in zip(grads, ("x", "x0", "w", "bias")):
        close(got, differences(
            lambda: (ot.conv(i["x"], i["w"], i["bias"], i["x0"], ends, silu)[0] * i["du"]).sum(), i[k]))


@pytest.mark.parametrize("softplus,gated", [(True, True), (False, True), (True, False)])
def test_scan_backward_against_differences(softplus, gated):
    K, B, D, N, G = 4, 2, 4, 3, 2
    i = scan_inputs(K, B, D, N, G, "f32", 5)
    if not softplus:
        i["dt"], i["dt_bias"] = np.abs(i["dt"]), np.abs(i["dt_bias"])
    if not gated:
        i["z"] = None
    ends = [K, 3]
    dy, dh = i["dy"], i["dh_last"]

    def loss():
        y, h, _ = ot.scan(i, ends, softplus)
        return (y * dy).sum() + (h * dh).sum()

    g = ot.scan_backward(i, ends, dy, dh, softplus)
    for k, name in (("x", "dx"), ("dt", "ddt"), ("A", "dA"), ("Bm", "dB"), ("Cm", "dC"),
                    ("skip", "dskip"), ("dt_bias", "ddt_bias"), ("h0", "dh0"), ("z", "dz")):
        if i[k] is not None:
            close(g[name], differences(loss, i[k]))


def test_scan_identities():
    """With A = 0 the state is a running sum; a prompt in two pieces is the prompt; a sequence of
    length zero keeps its state and gives nothing."""
    K, B, D, N, G = 6, 2, 4, 3, 1
    i = scan_inputs(K, B, D, N, G, "f32", 9)
    i["z"] = None
    y, h, _ = ot.scan(i, [K, 0])
    assert np.array_equal(h[1], i["h0"][1]) and not y[:, 1].any()
    one = {k: (v[:2] if k in ("x", "dt", "Bm", "Cm") else v) for k, v in i.items()}
    y1, h1, _ = ot.scan(one, [2, 2])
    two = {k: (v[2:] if k in ("x", "dt", "Bm", "Cm") else v) for k, v in i.items()}
    two["h0"] = h1
    y2, h2, _ = ot.scan(two, [K - 2, K - 2])
    full = ot.scan(i, [K, K])
    assert np.allclose(np.concatenate([y1, y2]), full[0], atol=1e-13)
    assert np.allclose(h2, full[1], atol=1e-13)
    i["A"] = np.zeros_like(i["A"])
    d = np.logaddexp(0.0, i["dt"] + i["dt_bias"])
    want = i["h0"] + np.einsum("tbd,tbn->bdn", d * i["x"], i["Bm"][:, :, 0])
    assert np.allclose(ot.scan(i, [K, K])[1], want, atol=1e-12)
