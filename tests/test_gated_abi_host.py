"""The gated block's C entry points on the host: bad arguments are refused with the documented status
codes before a GPU is touched (no kernel runs), and sizes are what the header says."""
import ctypes
import os
import subprocess
import tempfile

import pytest

from recurrent_cfc_cell_gb300 import _lib, build

INVALID_DIM, NULL_PTR, MISALIGNED, WS_TOO_SMALL, INVALID_ARG = -1, -2, -3, -4, -8
F, ODD = 0x10000, 0x10001  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def held(codes=F, scales=F):
    return ctypes.byref(_lib.Held8Ptrs(codes, scales))


def change(args, **at):
    out = list(args)
    for k, v in at.items():
        out[int(k[1:])] = v
    return out


@pytest.mark.parametrize("at,code", [
    (dict(a0=None), NULL_PTR), (dict(a1=-1), INVALID_DIM), (dict(a2=0), INVALID_DIM),
    (dict(a3=0), INVALID_DIM), (dict(a3=(1 << 24) + 1), INVALID_DIM), (dict(a4=3), INVALID_ARG),
    (dict(a0=ODD), MISALIGNED), (dict(a0=ODD, a4=1), MISALIGNED), (dict(a5=None), NULL_PTR),
    (dict(a5=held(None)), NULL_PTR), (dict(a5=held(F, None)), NULL_PTR)])
def test_pack8_refusals(lib, at, code):
    args = change([F, 8, 4, 8, 0, held(), None], **at)
    assert lib.cfc_pack8(*args) == code
    if "a1" not in at:
        assert lib.cfc_unpack8(args[5], args[2], args[3], args[4], args[0], args[1], None) == code
    assert lib.cfc_unpack8(held(), 4, 8, 0, F, 7, None) == INVALID_DIM


def rms(**over):
    a = dict(rows=4, n=8, dtype=0, eps=1e-5, x=F, residual=None, ldx=8, ldr=0, w=F)
    a.update(over)
    return ctypes.byref(_lib.RmsnormArgs(**a))


@pytest.mark.parametrize("over,code", [
    (dict(rows=0), INVALID_DIM), (dict(n=0), INVALID_DIM), (dict(ldx=-1), INVALID_DIM),
    (dict(dtype=2), INVALID_ARG), (dict(x=None), NULL_PTR), (dict(w=None), NULL_PTR),
    (dict(x=ODD), MISALIGNED), (dict(w=ODD), MISALIGNED)])
def test_rmsnorm_refusals(lib, over, code):
    assert lib.cfc_rmsnorm_forward(rms(**over), F, 8, F, 8, None, None, F, None) == code
    assert lib.cfc_rmsnorm_backward(rms(**over), None, F, F, 8, None, 0, F, 8, None, 0, F, F,
                                    1 << 30, None) == code


def test_rmsnorm_output_refusals(lib):
    fwd = [rms(), F, 8, F, 8, None, None, F, None]
    for eps in (-1.0, float("nan"), float("inf")):
        assert lib.cfc_rmsnorm_forward(*change(fwd, a0=rms(eps=eps))) == INVALID_ARG
    assert lib.cfc_rmsnorm_forward(*change(fwd, a0=None)) == NULL_PTR
    assert lib.cfc_rmsnorm_forward(*change(fwd, a0=rms(residual=F, ldr=-8))) == INVALID_DIM
    assert lib.cfc_rmsnorm_forward(*change(fwd, a2=7)) == INVALID_DIM
    assert lib.cfc_rmsnorm_forward(*change(fwd, a4=7)) == INVALID_DIM
    assert lib.cfc_rmsnorm_forward(*change(fwd, a5=held(None))) == NULL_PTR
    assert lib.cfc_rmsnorm_forward(*change(fwd, a6=held(F, None))) == NULL_PTR
    assert lib.cfc_rmsnorm_forward(*change(fwd, a7=ODD)) == MISALIGNED
    need = _lib.rmsnorm_workspace_bytes(5000, 300)
    bwd = [rms(rows=5000, n=300, ldx=300), None, F, F, 300, None, 0, F, 300, None, 0, F, F, need,
           None]
    for k in (2, 3, 7, 11, 12):
        assert lib.cfc_rmsnorm_backward(*change(bwd, **{f"a{k}": None})) == NULL_PTR
    assert lib.cfc_rmsnorm_backward(*change(bwd, a13=need - 1)) == WS_TOO_SMALL
    assert lib.cfc_rmsnorm_backward(*change(bwd, a12=F + 8)) == MISALIGNED
    assert lib.cfc_rmsnorm_backward(*change(bwd, a1=held(None))) == NULL_PTR
    assert lib.cfc_rmsnorm_backward(*change(bwd, a9=F, a10=299)) == INVALID_DIM
    assert _lib.rmsnorm_workspace_bytes(1, 64) == 0
    assert lib.cfc_rmsnorm_workspace_bytes(4, 8, None) == NULL_PTR


def gated(**over):
    a = dict(B=2, K=4, D=8, dtype=0, lengths=None, x=F, f=F, z=None, x_t=16, x_b=8, f_t=16, f_b=8,
             z_t=0, z_b=0, bias=None, h0=None)
    a.update(over)
    return ctypes.byref(_lib.GatedArgs(**a))


def kept(x=(F, F), f=(F, F), z=(None, None)):
    return ctypes.byref(_lib.GatedKept(*(_lib.Held8Ptrs(*v) for v in (x, f, z))))


def grads(**over):
    g = dict(dx=F, df=F, dz=None, y=None, dx_t=16, dx_b=8, df_t=16, df_b=8, dz_t=16, dz_b=8, y_t=16,
             y_b=8, dbias=None, dh0=None)
    g.update(over)
    return ctypes.byref(_lib.GatedGrads(**g))


@pytest.mark.parametrize("over,code", [
    (dict(B=0), INVALID_DIM), (dict(B=65536), INVALID_DIM), (dict(K=0), INVALID_DIM),
    (dict(K=(1 << 24) + 1), INVALID_DIM), (dict(D=0), INVALID_DIM), (dict(x_t=-1), INVALID_DIM),
    (dict(f_b=-8), INVALID_DIM), (dict(dtype=5), INVALID_ARG), (dict(x=None), NULL_PTR),
    (dict(f=None), NULL_PTR), (dict(x=ODD), MISALIGNED), (dict(z=ODD), MISALIGNED),
    (dict(bias=ODD), MISALIGNED), (dict(h0=ODD), MISALIGNED), (dict(lengths=F + 2), MISALIGNED)])
def test_gated_refusals(lib, over, code):
    assert lib.cfc_gated_forward(gated(**over), F, 16, 8, None, None, None, F, 1 << 30, None) == code
    assert lib.cfc_gated_backward(gated(**over), None, F, F, 16, 8, None, grads(dz=F), F, 1 << 30,
                                  None) == code
    if "K" not in over and "x_t" not in over:
        assert lib.cfc_gated_step(gated(**{"h0": F, "K": 0, **over}), F, 8, F, None) == code


def test_gated_output_refusals(lib):
    fwd = [gated(), F, 16, 8, None, None, None, None, 0, None]
    assert lib.cfc_gated_forward(*change(fwd, a0=None)) == NULL_PTR
    assert lib.cfc_gated_forward(*change(fwd, a1=None)) == NULL_PTR
    assert lib.cfc_gated_forward(*change(fwd, a2=0)) == INVALID_DIM
    assert lib.cfc_gated_forward(*change(fwd, a4=ODD)) == MISALIGNED
    assert lib.cfc_gated_forward(*change(fwd, a5=ODD)) == MISALIGNED
    assert lib.cfc_gated_forward(*change(fwd, a6=kept(x=(None, F)))) == NULL_PTR
    assert lib.cfc_gated_forward(*change(fwd, a6=kept(f=(F, None)))) == NULL_PTR
    assert lib.cfc_gated_forward(*change(fwd, a0=gated(z=F), a6=kept())) == NULL_PTR
    need = _lib.gated_workspace_bytes(4096, 2, 8, False)  # few channels, many steps: segments
    long = [gated(K=4096), F, 16, 8, None, None, None, F, need - 1, None]
    assert lib.cfc_gated_forward(*long) == WS_TOO_SMALL
    assert lib.cfc_gated_forward(*change(long, a7=None)) == NULL_PTR
    assert lib.cfc_gated_forward(*change(long, a7=F + 8)) == MISALIGNED
    need = _lib.gated_workspace_bytes(4, 2, 8, True)
    bwd = [gated(), None, F, F, 16, 8, None, grads(), F, need, None]
    for k in (2, 3, 7):
        assert lib.cfc_gated_backward(*change(bwd, **{f"a{k}": None})) == NULL_PTR
    for name in ("dx", "df"):
        assert lib.cfc_gated_backward(*change(bwd, a7=grads(**{name: None}))) == NULL_PTR
    assert lib.cfc_gated_backward(*change(bwd, a0=gated(z=F))) == NULL_PTR  # a gate's gradient
    assert lib.cfc_gated_backward(*change(bwd, a1=kept(z=(F, F)))) == NULL_PTR
    assert lib.cfc_gated_backward(*change(bwd, a1=kept(z=(F, None)), a7=grads(dz=F))) == NULL_PTR
    assert lib.cfc_gated_backward(*change(bwd, a7=grads(y=F, y_t=0))) == INVALID_DIM
    assert lib.cfc_gated_backward(*change(bwd, a7=grads(dbias=ODD))) == MISALIGNED
    assert lib.cfc_gated_backward(*change(bwd, a9=need - 1)) == WS_TOO_SMALL
    step = [gated(K=0, h0=F), F, 8, F, None]
    assert lib.cfc_gated_step(*change(step, a0=gated(K=0))) == NULL_PTR
    assert lib.cfc_gated_step(*change(step, a1=None)) == NULL_PTR
    assert lib.cfc_gated_step(*change(step, a3=None)) == NULL_PTR
    assert lib.cfc_gated_step(*change(step, a3=ODD)) == MISALIGNED
    assert lib.cfc_gated_workspace_bytes(0, 4, 8, 1, ctypes.byref(ctypes.c_size_t())) == INVALID_DIM
    assert lib.cfc_gated_workspace_bytes(2, 4, 8, 0, None) == NULL_PTR


def test_weights4_refusals(lib):
    out = ctypes.c_size_t()
    for N, K, group, code in ((0, 8, 32, INVALID_DIM), (8, 0, 32, INVALID_DIM),
                              (8, 8, 16, INVALID_ARG), (8, 8, 0, INVALID_ARG),
                              (1 << 24, 1 << 24, 32, INVALID_DIM)):
        assert lib.cfc_weights4_bytes(N, K, group, ctypes.byref(out)) == code
        assert lib.cfc_weights4_quantize(F, 1 << 24, N, K, group, 0, F, F, None) == code
        assert lib.cfc_weights4_lay_out(F, F, N, K, group, F, 1 << 62, None) == code
        assert lib.cfc_matvec4(F, 1 << 24, F, 1, N, K, group, 0, F, 1 << 24, None) == code
    assert lib.cfc_weights4_bytes(8, 8, 32, None) == NULL_PTR
    quant = [F, 8, 4, 8, 32, 0, F, F, None]
    for at, code in ((dict(a0=None), NULL_PTR), (dict(a1=-1), INVALID_DIM), (dict(a5=2), INVALID_ARG),
                     (dict(a6=None), NULL_PTR), (dict(a7=None), NULL_PTR), (dict(a7=ODD), MISALIGNED),
                     (dict(a0=ODD), MISALIGNED)):
        assert lib.cfc_weights4_quantize(*change(quant, **at)) == code
    need = _lib.weights4_bytes(4, 8, 32)
    lay = [F, F, 4, 8, 32, F, need, None]
    for at, code in ((dict(a0=None), NULL_PTR), (dict(a1=None), NULL_PTR), (dict(a5=None), NULL_PTR),
                     (dict(a6=need - 1), WS_TOO_SMALL), (dict(a5=F + 8), MISALIGNED)):
        assert lib.cfc_weights4_lay_out(*change(lay, **at)) == code
    vec = [F, 8, F, 2, 4, 8, 32, 0, F, 4, None]
    for at, code in ((dict(a0=None), NULL_PTR), (dict(a2=None), NULL_PTR), (dict(a8=None), NULL_PTR),
                     (dict(a3=0), INVALID_DIM), (dict(a3=(1 << 19) + 1), INVALID_DIM),
                     (dict(a9=3), INVALID_DIM), (dict(a1=-1), INVALID_DIM), (dict(a7=4), INVALID_ARG),
                     (dict(a0=ODD), MISALIGNED), (dict(a2=F + 8), MISALIGNED)):
        assert lib.cfc_matvec4(*change(vec, **at)) == code


def test_weights4_sizes(lib):
    assert _lib.weights4_bytes(16, 128, 128) == 1024 + 32
    assert _lib.weights4_bytes(17, 129, 32) == 4 * 1024 + 2 * 8 * 32
    assert _lib.weights4_bytes(1, 1, 64) == 1024 + 2 * 32


def test_ctypes_structures_match_the_header(lib):
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    names = ("cfc_held8", "cfc_rmsnorm_args", "cfc_gated_args", "cfc_gated_kept", "cfc_gated_grads")
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "s.c"), os.path.join(d, "s")
        with open(src, "w") as fh:
            fh.write('#include <stdio.h>\n#include "cfc.h"\nint main(void) {' + "".join(
                f'printf("%zu ", sizeof({n}));' for n in names) +
                'printf("%d %d", CFC_GATED_PERIOD, CFC_HELD8_BLOCK); return 0; }')
        subprocess.run(["gcc", "-I", inc, src, "-o", exe], check=True)
        sizes = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in sizes] == [ctypes.sizeof(c) for c in (
        _lib.Held8Ptrs, _lib.RmsnormArgs, _lib.GatedArgs, _lib.GatedKept, _lib.GatedGrads)] + [
        _lib.GATED_PERIOD, _lib.HELD8_BLOCK]
