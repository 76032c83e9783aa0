"""The trunk operators' C entry points on the host: bad arguments are refused with the documented
status codes before a GPU is touched (no kernel runs), and workspace sizes are what the kernels'
plans need."""
import ctypes

import pytest

from recurrent_cfc_cell_gb300 import _lib, build

OK, INVALID_DIM, NULL_PTR, MISALIGNED, WS_TOO_SMALL, INVALID_ARG = 0, -1, -2, -3, -4, -8
F, ODD = 0x10000, 0x10001  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def change(args, **at):
    out = list(args)
    for k, v in at.items():
        out[int(k[1:])] = v
    return out


# x, ldx, w, b, rows, n, eps, dtype, y, ldy, stats, stream
NORM = [F, 8, F, F, 4, 8, 1e-5, 0, F, 8, F, None]


@pytest.mark.parametrize("at,code", [
    (dict(a0=None), NULL_PTR), (dict(a2=None), NULL_PTR), (dict(a3=None), NULL_PTR),
    (dict(a8=None), NULL_PTR), (dict(a10=None), NULL_PTR), (dict(a4=0), INVALID_DIM),
    (dict(a5=0), INVALID_DIM), (dict(a5=-3), INVALID_DIM), (dict(a9=7), INVALID_DIM),
    (dict(a1=-1), INVALID_DIM), (dict(a6=float("nan")), INVALID_ARG), (dict(a6=-1.0), INVALID_ARG),
    (dict(a6=float("inf")), INVALID_ARG), (dict(a7=2), INVALID_ARG), (dict(a0=ODD), MISALIGNED),
    (dict(a0=ODD + 1), MISALIGNED), (dict(a2=ODD), MISALIGNED), (dict(a10=F + 4), MISALIGNED),
    (dict(a0=ODD, a7=1), MISALIGNED)])
def test_layernorm_refusals(lib, at, code):
    assert lib.cfc_layernorm_forward(*change(NORM, **at)) == code


def test_layernorm_backward_workspace(lib):
    need = _lib.layernorm_workspace_bytes(5000, 300)
    assert need > 0
    args = [F, 300, F, 300, F, F, 5000, 300, 0, F, 300, F, F, F, need - 1, None]
    assert lib.cfc_layernorm_backward(*args) == WS_TOO_SMALL
    assert lib.cfc_layernorm_backward(*change(args, a13=None)) == NULL_PTR
    assert lib.cfc_layernorm_backward(*change(args, a13=F + 8, a14=need)) == MISALIGNED
    assert _lib.layernorm_workspace_bytes(1, 64) == 0  # one CTA writes the gradients itself
    assert lib.cfc_layernorm_workspace_bytes(4, 8, None) == NULL_PTR
    assert lib.cfc_layernorm_workspace_bytes(0, 8, ctypes.byref(ctypes.c_size_t())) == INVALID_DIM


# x, ldx, residual, ldr, rng, p, rows, n, dtype, y, ldy, stream
DROP = [F, 8, None, 0, F, 0.5, 4, 8, 0, F, 8, None]


@pytest.mark.parametrize("at,code", [
    (dict(a0=None), NULL_PTR), (dict(a4=None), NULL_PTR), (dict(a9=None), NULL_PTR),
    (dict(a5=-0.1), INVALID_ARG), (dict(a5=1.1), INVALID_ARG), (dict(a5=float("nan")), INVALID_ARG),
    (dict(a4=F + 4), MISALIGNED), (dict(a6=0), INVALID_DIM), (dict(a10=4), INVALID_DIM),
    (dict(a2=F, a3=-8), INVALID_DIM), (dict(a8=7), INVALID_ARG)])
def test_dropout_refusals(lib, at, code):
    assert lib.cfc_dropout_forward(*change(DROP, **at)) == code


def test_dropout_layernorm_refusals(lib):
    fwd = [F, 8, None, 0, F, 0.5, F, F, 4, 8, 1e-5, 0, F, 8, F, 8, F, None]
    for k in (0, 4, 6, 7, 12, 14, 16):
        assert lib.cfc_dropout_layernorm_forward(*change(fwd, **{f"a{k}": None})) == NULL_PTR
    assert lib.cfc_dropout_layernorm_forward(*change(fwd, a5=2.0)) == INVALID_ARG
    bwd = [F, 8, None, 0, F, 8, F, 0.5, F, F, 4, 8, 0, F, 8, None, 0, F, F, F, 1 << 20, None]
    for k in (0, 4, 6, 8, 9, 13, 17, 18):
        assert lib.cfc_dropout_layernorm_backward(*change(bwd, **{f"a{k}": None})) == NULL_PTR
    assert lib.cfc_dropout_layernorm_backward(*change(bwd, a15=F, a16=7)) == INVALID_DIM


def conv_args(**over):
    a = dict(B=2, K=4, D=8, W=4, dtype=0, silu=1, lengths=None, x=F, x_t=16, x_b=8, w=F, bias=None,
             x0=None)
    a.update(over)
    return ctypes.byref(_lib.ConvArgs(**a))


@pytest.mark.parametrize("over,code", [
    (dict(B=0), INVALID_DIM), (dict(B=65536), INVALID_DIM), (dict(K=0), INVALID_DIM),
    (dict(D=0), INVALID_DIM), (dict(W=1), INVALID_DIM), (dict(W=5), INVALID_DIM),
    (dict(x_t=-1), INVALID_DIM), (dict(dtype=5), INVALID_ARG), (dict(x=None), NULL_PTR),
    (dict(w=None), NULL_PTR), (dict(x=ODD), MISALIGNED), (dict(x0=ODD), MISALIGNED),
    (dict(lengths=F + 2), MISALIGNED)])
def test_conv_refusals(lib, over, code):
    assert lib.cfc_conv_forward(conv_args(**over), F, 16, 8, None, None) == code
    assert lib.cfc_conv_backward(conv_args(**over), F, 16, 8, F, 16, 8, F, F, None, F, 1 << 30,
                                 None) == code


def test_conv_outputs_and_step_refusals(lib):
    assert lib.cfc_conv_forward(None, F, 16, 8, None, None) == NULL_PTR
    assert lib.cfc_conv_forward(conv_args(), None, 16, 8, None, None) == NULL_PTR
    assert lib.cfc_conv_forward(conv_args(), F, 0, 8, None, None) == INVALID_DIM
    need = _lib.conv_workspace_bytes(2, 4000, 8, 4, 0)
    args = [conv_args(K=4000), F, 16, 8, F, 16, 8, F, F, None, F, need - 1, None]
    assert lib.cfc_conv_backward(*args) == WS_TOO_SMALL
    step = [F, 8, F, None, F, 2, 8, 4, 0, 1, F, 8, F, None]
    for k in (0, 2, 4, 10, 12):
        assert lib.cfc_conv_step(*change(step, **{f"a{k}": None})) == NULL_PTR
    assert lib.cfc_conv_step(*change(step, a7=9)) == INVALID_DIM


def scan_args(**over):
    a = dict(B=2, K=4, D=8, N=4, G=2, dtype=0, softplus=1, lengths=None, x=F, dt=F, z=None, x_t=16,
             x_b=8, dt_t=16, dt_b=8, z_t=0, z_b=0, Bm=F, Cm=F, Bm_t=16, Bm_b=8, Cm_t=16, Cm_b=8,
             A=F, skip=None, dt_bias=None, h0=None)
    a.update(over)
    return ctypes.byref(_lib.ScanArgs(**a))


def grads(**over):
    g = dict(dx=F, ddt=F, dz=None, dx_t=16, dx_b=8, ddt_t=16, ddt_b=8, dz_t=0, dz_b=0, dB=F, dC=F,
             dA=F, dskip=None, ddt_bias=None, dh0=None)
    g.update(over)
    return ctypes.byref(_lib.ScanGrads(**g))


@pytest.mark.parametrize("over,code", [
    (dict(B=0), INVALID_DIM), (dict(K=0), INVALID_DIM), (dict(D=0), INVALID_DIM),
    (dict(N=0), INVALID_DIM), (dict(N=129), INVALID_DIM), (dict(G=3), INVALID_DIM),
    (dict(G=0), INVALID_DIM), (dict(x_b=-8), INVALID_DIM), (dict(dtype=2), INVALID_ARG),
    (dict(x=None), NULL_PTR), (dict(dt=None), NULL_PTR), (dict(Bm=None), NULL_PTR),
    (dict(Cm=None), NULL_PTR), (dict(A=None), NULL_PTR), (dict(h0=F + 4), MISALIGNED),
    (dict(A=ODD), MISALIGNED), (dict(z=ODD), MISALIGNED)])
def test_scan_refusals(lib, over, code):
    assert lib.cfc_scan_forward(scan_args(**over), F, 16, 8, None, None, F, 1 << 30, None) == code
    assert lib.cfc_scan_backward(scan_args(**over), F, F, 16, 8, None, grads(), F, 1 << 30,
                                 None) == code


def test_scan_outputs_refusals(lib):
    assert lib.cfc_scan_forward(scan_args(), None, 16, 8, None, None, None, 0, None) == NULL_PTR
    assert lib.cfc_scan_forward(scan_args(), F, 16, 0, None, None, None, 0, None) == INVALID_DIM
    assert lib.cfc_scan_forward(scan_args(), F, 16, 8, F + 8, None, None, 0, None) == MISALIGNED
    for name in ("dx", "ddt", "dB", "dC", "dA"):
        assert lib.cfc_scan_backward(scan_args(), F, F, 16, 8, None, grads(**{name: None}), F,
                                     1 << 30, None) == NULL_PTR
    assert lib.cfc_scan_backward(scan_args(z=F), F, F, 16, 8, None, grads(), F, 1 << 30,
                                 None) == NULL_PTR  # a gate's gradient is wanted
    assert lib.cfc_scan_backward(scan_args(), None, F, 16, 8, None, grads(), F, 1 << 30,
                                 None) == NULL_PTR
    assert lib.cfc_scan_backward(scan_args(), F, F, 16, 8, None, grads(), F, 16, None) == WS_TOO_SMALL
    step = scan_args(K=0)
    assert lib.cfc_scan_step(step, F, 8, F, None) == NULL_PTR  # no state
    assert lib.cfc_scan_step(scan_args(K=0, h0=F), F, 8, None, None) == NULL_PTR


def test_scan_sizes(lib):
    assert _lib.scan_states_bytes(17, 2, 8, 4, 1, 0) == 3 * 2 * 8 * 4 * 4
    assert _lib.scan_workspace_bytes(64, 32, 256, 32, 1, 0, False) == 0  # no split of the steps
    assert _lib.scan_workspace_bytes(8192, 1, 256, 16, 1, 0, False) > 0
    assert _lib.scan_workspace_bytes(64, 32, 256, 32, 1, 0, True) >= 32 * 256 * 34 * 4


def test_ctypes_structures_match_the_header(lib):
    """Sizes that a C compiler gives the structures."""
    import os
    import subprocess
    import tempfile

    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "s.c"), os.path.join(d, "s")
        with open(src, "w") as fh:
            fh.write('#include <stdio.h>\n#include "cfc.h"\nint main(void) { printf("%zu %zu %zu", '
                     "sizeof(cfc_conv_args), sizeof(cfc_scan_args), sizeof(cfc_scan_grads)); return 0; }")
        subprocess.run(["gcc", "-I", inc, src, "-o", exe], check=True)
        sizes = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in sizes] == [ctypes.sizeof(c) for c in
                                       (_lib.ConvArgs, _lib.ScanArgs, _lib.ScanGrads)]
