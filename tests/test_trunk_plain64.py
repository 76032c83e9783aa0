"""The batched float64 forms of the trunk operators (trunk_plain64.py) against the oracle."""
import numpy as np
import pytest
import torch

import oracle.trunk as ot
import trunk_plain64 as p64
from trunk_cases import conv_inputs, norm_inputs, scan_inputs

# Both sides are the same formulas in float64: what a few hundred roundings leave.
TOL = 1e-12


def near(got, want, name=""):
    want = np.asarray(want)
    assert tuple(got.shape) == want.shape, name
    assert np.abs(got.numpy() - want).max() <= TOL * max(1.0, np.abs(want).max()), name


def tensors(i):
    return {k: torch.from_numpy(np.ascontiguousarray(v)) for k, v in i.items()}


def test_norm():
    i = norm_inputs(7, 13, "f32", 1)
    t = tensors(i)
    near(p64.norm(t["x"], t["w"], t["b"]), ot.layernorm(i["x"], i["w"], i["b"], 1e-5))
    for got, want in zip(p64.norm_backward(t["dy"], t["x"], t["w"]),
                         ot.layernorm_backward(i["dy"], i["x"], i["w"], 1e-5)):
        near(got, want)


@pytest.mark.parametrize("rows,n,p", [(1, 1, 0.5), (9, 21, 0.2), (4, 40, 0.0), (4, 40, 1.0)])
def test_dropout_mask(rows, n, p):
    seed, offset = 0xFEDCBA9876543210, 0x8000000500000003
    got, scale = p64.dropout_mask(rows, n, p, seed, offset)
    want, want_scale = ot.dropout_mask(rows, n, p, seed, offset)
    assert np.array_equal(got.numpy(), want) and scale == want_scale


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("K,B,D,W,ends", [(1, 1, 1, 2, [1]), (11, 5, 6, 4, [11, 0, 1, 2, 7]),
                                          (2, 3, 4, 4, [0, 1, 2])])
def test_conv(K, B, D, W, ends, silu):
    i = conv_inputs(K, B, D, W, "f32", 2)
    t = tensors(i)
    out = p64.conv(t["x"], t["w"], t["bias"], t["x0"], torch.tensor(ends), silu, t["du"])
    u, last = ot.conv(i["x"], i["w"], i["bias"], i["x0"], ends, silu)
    dx, dx0, dw, dbias = ot.conv_backward(i["du"], i["x"], i["w"], i["bias"], i["x0"], ends, silu)
    for k, want in dict(u=u, last=last, dx=dx, dx0=dx0, dw=dw, dbias=dbias).items():
        near(out[k], want, k)


@pytest.mark.parametrize("K,B,D,N,G,ends,gate,softplus", [
    (1, 1, 1, 1, 1, [1], True, True), (9, 4, 6, 5, 3, [9, 0, 1, 4], True, True),
    (5, 2, 4, 2, 1, [5, 3], False, False)])
def test_scan(K, B, D, N, G, ends, gate, softplus):
    i = scan_inputs(K, B, D, N, G, "f32", 3)
    if not softplus:
        i["dt"] = np.abs(i["dt"]) * 0.125
    if not gate:
        i.pop("z")
    t = tensors(i)
    i.setdefault("z", None)
    t.setdefault("z", None)
    out = p64.scan(t, torch.tensor(ends), softplus)
    y, h, _ = ot.scan(i, ends, softplus)
    near(out["y"], y, "y")
    near(out["h"], h, "h")
    want = ot.scan_backward(i, ends, i["dy"], i["dh_last"], softplus)
    want["dD"] = want.pop("dskip")
    for k, v in want.items():
        if k in out:
            near(out[k], v, k)
    assert ("dz" in out) == gate
