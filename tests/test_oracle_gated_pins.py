"""The gated block's fp64 oracle against facts outside it: torch's own 8-bit type and autograd,
differences, and cases that can be done by hand."""
import numpy as np
import pytest
import torch

import oracle.gated as og
from gated_cases import gated_inputs, rms_inputs


def test_e4m3_codes_are_torchs():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    for c in range(256):
        v = og.e4m3_value(c)
        assert (np.isnan(v) and np.isnan(codes[c])) or v == codes[c]
    r = np.random.default_rng(0)
    u = np.concatenate([r.normal(size=500) * 2.0 ** r.integers(-12, 7, size=500), og.E4M3,
                        (og.E4M3[1:] + og.E4M3[:-1]) / 2, [448.0, -448.0, 0.0]])
    u = u[np.abs(u) <= 448].astype(np.float32)
    want = torch.from_numpy(u).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal([og.e4m3_value(og.e4m3_code(v)) for v in u], want)


@pytest.mark.parametrize("top,byte", [(448.0, 127), (448.1, 128), (449.0, 128), (224.0, 126),
                                      (1.0, 119), (1.75, 119), (1.7500001, 120), (0.0, 1),
                                      (1e-45, 1), (3.4e38, 247)])
def test_scale_is_the_smallest_power_of_two(top, byte):
    v = np.zeros(40)
    v[3] = -top
    codes, scales = og.pack8(v)
    assert scales[0] == byte and scales[1] == 1 and not codes[32:].any()
    assert np.max(np.abs(v)) <= 448 * 2.0 ** (byte - 127)


def test_held_values_are_within_half_a_step():
    r = np.random.default_rng(1)
    v = r.normal(size=(50, 77)) * 2.0 ** r.integers(-30, 30, size=(50, 1))
    h = og.held8(v)
    for c in range(0, 77, 32):
        scale = 2.0 ** np.ceil(np.log2(np.abs(v[:, c:c + 32]).max(axis=1, keepdims=True) / 448))
        assert np.all(np.abs(h - v)[:, c:c + 32] <= np.maximum(2.0 ** -4 * np.abs(v[:, c:c + 32]),
                                                              2.0 ** -10 * scale))
    assert np.array_equal(og.held8(h), h)
    v[7, 40] = np.inf
    h = og.held8(v)
    assert np.isnan(h[7, 32:64]).all() and np.isfinite(h[7, :32]).all()


def test_rmsnorm_against_autograd():
    i = rms_inputs(7, 13, "f32", 3)
    x, res, w = (torch.tensor(i[k], requires_grad=True) for k in ("x", "residual", "w"))
    s = x + res
    y = s / torch.sqrt((s * s).mean(1, keepdim=True) + 1e-5) * w
    (y * torch.tensor(i["dy"])).sum().add((s * torch.tensor(i["ds"])).sum()).backward()
    s = i["x"] + i["residual"]
    dx, dw, again = og.rmsnorm_backward(i["dy"], s, i["w"], 1e-5, ds=i["ds"])
    assert np.allclose(og.rmsnorm(s, i["w"], 1e-5), y.detach().numpy(), rtol=1e-12)
    assert np.allclose(again, y.detach().numpy(), rtol=1e-12)
    assert np.allclose(dx, x.grad.numpy(), rtol=1e-10) and np.allclose(dx, res.grad.numpy(), rtol=1e-10)
    assert np.allclose(dw, w.grad.numpy(), rtol=1e-10)


@pytest.mark.parametrize("gate", [True, False])
def test_gated_against_autograd(gate):
    i = gated_inputs(11, 3, 4, "f32", 5, [11, 0, 7])
    t = {k: torch.tensor(i[k], requires_grad=True) for k in ("x", "f", "z", "bias", "h0")}
    y, h, _ = og.gated(i["x"], i["f"], i["bias"], i["z"] if gate else None, i["h0"], i["ends"])
    states, total = t["h0"], 0.0
    for k in range(11):
        on = torch.tensor(k < i["ends"])[:, None]
        g = 1 / (1 + torch.exp(-(t["f"][k] + t["bias"])))
        states = torch.where(on, g * states + (1 - g) * t["x"][k], states)
        yk = states * (t["z"][k] / (1 + torch.exp(-t["z"][k])) if gate else 1.0)
        assert np.allclose(torch.where(on, yk, 0.0).detach().numpy(), y[k], atol=1e-13)
        total = total + (torch.where(on, yk, 0.0) * torch.tensor(i["dy"][k])).sum()
    assert np.allclose(states.detach().numpy(), h, atol=1e-13)
    (total + (states * torch.tensor(i["dh_last"])).sum()).backward()
    out, again = og.gated_backward(i["dy"], i["x"], i["f"], i["bias"], i["z"] if gate else None,
                                   i["h0"], i["ends"], i["dh_last"])
    assert np.allclose(again, y, atol=1e-13)
    for name, want in (("dx", "x"), ("df", "f"), ("dbias", "bias"), ("dh0", "h0")):
        assert np.allclose(out[name], t[want].grad.numpy(), atol=1e-12), name
    if gate:
        assert np.allclose(out["dz"], t["z"].grad.numpy(), atol=1e-12)


def test_gated_by_differences():
    i = gated_inputs(9, 1, 2, "f32", 6)

    def loss(**over):
        j = {**i, **over}
        y, h, _ = og.gated(j["x"], j["f"], j["bias"], j["z"], j["h0"], j["ends"])
        return (y * i["dy"]).sum() + (h * i["dh_last"]).sum()

    out, _ = og.gated_backward(i["dy"], i["x"], i["f"], i["bias"], i["z"], i["h0"], i["ends"],
                               i["dh_last"])
    for name, of in (("x", "dx"), ("f", "df"), ("z", "dz"), ("bias", "dbias"), ("h0", "dh0")):
        for at in np.ndindex(i[name].shape):
            up, down = i[name].copy(), i[name].copy()
            up[at] += 1e-6
            down[at] -= 1e-6
            diff = (loss(**{name: up}) - loss(**{name: down})) / 2e-6
            assert abs(diff - out[of][at]) <= 1e-8 * (1 + abs(diff)), (name, at)


def test_kept_gradients_are_the_periods_on_held_values():
    """What holds its values exactly gives the unheld gradients; and one period at a time, the
    gradients of the recurrence on the held values from the kept state."""
    i = gated_inputs(8, 2, 3, "f32", 8)
    for k in ("x", "f", "z"):
        i[k] = og.held8(i[k])
    a, ya = og.gated_backward(i["dy"], i["x"], i["f"], i["bias"], i["z"], i["h0"], i["ends"])
    b, yb = og.gated_backward(i["dy"], i["x"], i["f"], i["bias"], i["z"], i["h0"], i["ends"],
                              kept=True)
    assert np.array_equal(ya, yb) and all(np.array_equal(a[k], b[k]) for k in a)
    i = gated_inputs(8, 2, 3, "f32", 9)
    b, yb = og.gated_backward(i["dy"], i["x"], i["f"], i["bias"], i["z"], i["h0"], i["ends"],
                              kept=True)
    h = {k: og.held8(i[k]) for k in ("x", "f", "z")}
    a, ya = og.gated_backward(i["dy"], h["x"], h["f"], i["bias"], h["z"], i["h0"], i["ends"])
    assert np.allclose(ya, yb) and all(np.allclose(a[k], b[k]) for k in a)


def test_weights4_by_hand():
    codes = np.array([[0x80, 0x0f], [0x98, 0xf7]], dtype=np.uint8)
    W = og.weights4(codes, np.array([[2.0], [0.5]]), 3, 32)
    assert np.array_equal(W, [[-16.0, 0.0, 14.0], [0.0, 0.5, -0.5]])
