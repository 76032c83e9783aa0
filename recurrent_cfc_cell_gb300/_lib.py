"""ctypes binding of libcfc.so (include/cfc.h): argument marshalling only.

Every function takes torch tensors that already live on the current CUDA device, checks
dtype / contiguity / shape on the host, passes raw pointers and the current stream to the C
entry point of the same name and raises ``CfcError`` on a non-zero status.  All computation
happens in the library's CUDA kernels.  If the library has not been built (or fails to load)
importing it raises, so nothing can silently run elsewhere.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_build", "libcfc.so")

CFC_OK = 0
CFC_DW_ACCURATE = 0   # tensor cores, two bf16 terms per operand (three products per step)
CFC_DW_BF16 = 1       # tensor cores, one bf16 product per step
CFC_DW_TF32 = 2       # tensor cores, one tf32 product per step
CFC_DW_SIMT_FP32 = 3  # CUDA-core fp32
DW_MODES = (CFC_DW_ACCURATE, CFC_DW_BF16, CFC_DW_TF32, CFC_DW_SIMT_FP32)


def dpre_operand_pitch(C: int, dw_mode: int) -> int:
    """bf16 values per term in a d_pre row of the workspace head (modes ACCURATE and BF16), as
    include/cfc.h documents: 4C rounded up to a multiple of 8."""
    return (4 * C + 7) // 8 * 8

# Public C symbols declared in include/cfc.h (checked by the test suite).
EXPORTED = ("cfc_workspace_bytes", "cfc_forward", "cfc_backward", "cfc_backward_recurrence",
            "cfc_weight_grad", "reduce_axis0", "cfc_error_string", "cfc_device_status",
            "cfc_backward_noalloc", "cfc_input_projection", "cfc_forward_recurrence",
            "cfc_step_launches", "cfc_forward_backward", "cfc_bptt_workspace_bytes",
            "cfc_backward_recurrence_ws", "cfc_wait_self_test", "cfc_probe_fma",
            "cfc_probe_l2_read", "cfc_forward_bf16_workspace_bytes", "cfc_forward_bf16",
            "cfc_backward_bf16", "cfc_decay_forward", "cfc_decay_workspace_bytes",
            "cfc_decay_backward", "cfc_forward_workspace_bytes", "cfc_copy",
            "cfc_layernorm_forward", "cfc_layernorm_workspace_bytes", "cfc_layernorm_backward",
            "cfc_dropout_forward", "cfc_dropout_backward", "cfc_dropout_layernorm_forward",
            "cfc_dropout_layernorm_backward", "cfc_conv_forward", "cfc_conv_workspace_bytes",
            "cfc_conv_backward", "cfc_conv_step", "cfc_scan_workspace_bytes",
            "cfc_scan_states_bytes", "cfc_scan_forward", "cfc_scan_backward", "cfc_scan_step",
            "cfc_pack8", "cfc_unpack8", "cfc_rmsnorm_forward", "cfc_rmsnorm_workspace_bytes",
            "cfc_rmsnorm_backward", "cfc_gated_forward", "cfc_gated_workspace_bytes",
            "cfc_gated_backward", "cfc_gated_step", "cfc_weights4_quantize", "cfc_weights4_bytes",
            "cfc_weights4_lay_out", "cfc_matvec4")
CFC_F32, CFC_BF16 = 0, 1          # activation types of the trunk operators
SCAN_PERIOD = 8                   # steps between the states a training scan keeps
GATED_PERIOD = 8                  # and a training gated recurrence
HELD8_BLOCK = 32                  # columns that share a scale in 8 bits
MATVEC4_ROWS = 1 << 19            # most rows of one call of cfc_matvec4
CFC_ERR_SCRATCH_LIMIT = -10
NOALLOC_SCRATCH_BYTES = 32 << 20  # size of cfc_backward_noalloc's built-in device scratch


class ConvArgs(ctypes.Structure):
    """cfc_conv_args of include/cfc.h."""
    _fields_ = [(k, ctypes.c_int) for k in ("B", "K", "D", "W", "dtype", "silu")] + [
        ("lengths", ctypes.c_void_p), ("x", ctypes.c_void_p), ("x_t", ctypes.c_longlong),
        ("x_b", ctypes.c_longlong), ("w", ctypes.c_void_p), ("bias", ctypes.c_void_p),
        ("x0", ctypes.c_void_p)]


class ScanArgs(ctypes.Structure):
    """cfc_scan_args of include/cfc.h."""
    _fields_ = [(k, ctypes.c_int) for k in ("B", "K", "D", "N", "G", "dtype", "softplus")] + [
        (k, ctypes.c_void_p) for k in ("lengths", "x", "dt", "z")] + [
        (k, ctypes.c_longlong) for k in ("x_t", "x_b", "dt_t", "dt_b", "z_t", "z_b")] + [
        (k, ctypes.c_void_p) for k in ("Bm", "Cm")] + [
        (k, ctypes.c_longlong) for k in ("Bm_t", "Bm_b", "Cm_t", "Cm_b")] + [
        (k, ctypes.c_void_p) for k in ("A", "skip", "dt_bias", "h0")]


class ScanGrads(ctypes.Structure):
    """cfc_scan_grads of include/cfc.h."""
    _fields_ = [(k, ctypes.c_void_p) for k in ("dx", "ddt", "dz")] + [
        (k, ctypes.c_longlong) for k in ("dx_t", "dx_b", "ddt_t", "ddt_b", "dz_t", "dz_b")] + [
        (k, ctypes.c_void_p) for k in ("dB", "dC", "dA", "dskip", "ddt_bias", "dh0")]


class Held8Ptrs(ctypes.Structure):
    """cfc_held8 of include/cfc.h."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class RmsnormArgs(ctypes.Structure):
    """cfc_rmsnorm_args of include/cfc.h."""
    _fields_ = [(k, ctypes.c_int) for k in ("rows", "n", "dtype")] + [
        ("eps", ctypes.c_float), ("x", ctypes.c_void_p), ("residual", ctypes.c_void_p),
        ("ldx", ctypes.c_longlong), ("ldr", ctypes.c_longlong), ("w", ctypes.c_void_p)]


class GatedArgs(ctypes.Structure):
    """cfc_gated_args of include/cfc.h."""
    _fields_ = [(k, ctypes.c_int) for k in ("B", "K", "D", "dtype")] + [
        (k, ctypes.c_void_p) for k in ("lengths", "x", "f", "z")] + [
        (k, ctypes.c_longlong) for k in ("x_t", "x_b", "f_t", "f_b", "z_t", "z_b")] + [
        (k, ctypes.c_void_p) for k in ("bias", "h0")]


class GatedKept(ctypes.Structure):
    """cfc_gated_kept of include/cfc.h."""
    _fields_ = [(k, Held8Ptrs) for k in ("x", "f", "z")]


class GatedGrads(ctypes.Structure):
    """cfc_gated_grads of include/cfc.h."""
    _fields_ = [(k, ctypes.c_void_p) for k in ("dx", "df", "dz", "y")] + [
        (k, ctypes.c_longlong) for k in ("dx_t", "dx_b", "df_t", "df_b", "dz_t", "dz_b", "y_t",
                                         "y_b")] + [
        (k, ctypes.c_void_p) for k in ("dbias", "dh0")]


class CfcError(RuntimeError):
    def __init__(self, func: str, code: int, text: str):
        super().__init__(f"{func} failed: {code} ({text})")
        self.code = code


_lib = None


def load(path: str | None = None) -> ctypes.CDLL:
    """Load libcfc.so (raises if it is missing: build it with recurrent_cfc_cell_gb300.build)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise ImportError(f"libcfc.so not built ({p}); run python -m recurrent_cfc_cell_gb300.build")
    lib = ctypes.CDLL(p)
    vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.cfc_workspace_bytes.argtypes = [i, i, i, i, i, ctypes.POINTER(sz)]
    lib.cfc_workspace_bytes.restype = i
    lib.cfc_forward.argtypes = [vp] * 5 + [i] * 4 + [vp, vp, vp, sz, vp]
    lib.cfc_forward.restype = i
    lib.cfc_backward.argtypes = [vp] * 7 + [i] * 4 + [vp] * 5 + [sz, i, vp]
    lib.cfc_backward.restype = i
    lib.cfc_forward_backward.argtypes = [vp] * 6 + [i] * 4 + [vp] * 7 + [sz, i, vp]
    lib.cfc_forward_backward.restype = i
    lib.cfc_backward_recurrence.argtypes = [vp] * 4 + [i] * 4 + [vp, vp, vp]
    lib.cfc_backward_recurrence.restype = i
    lib.cfc_bptt_workspace_bytes.argtypes = [i] * 4 + [vp]
    lib.cfc_bptt_workspace_bytes.restype = i
    lib.cfc_backward_recurrence_ws.argtypes = [vp] * 4 + [i] * 4 + [vp, vp, vp, sz, vp]
    lib.cfc_backward_recurrence_ws.restype = i
    lib.cfc_weight_grad.argtypes = [vp] * 5 + [i] * 4 + [vp] * 4 + [sz, i, vp]
    lib.cfc_weight_grad.restype = i
    lib.reduce_axis0.argtypes = [vp, i, i, vp, vp]
    lib.reduce_axis0.restype = i
    lib.cfc_input_projection.argtypes = [vp] * 3 + [i] * 4 + [vp, vp, vp]
    lib.cfc_input_projection.restype = i
    lib.cfc_forward_recurrence.argtypes = [vp] * 3 + [i] * 4 + [vp, vp, vp, sz, vp]
    lib.cfc_forward_recurrence.restype = i
    lib.cfc_step_launches.argtypes = [i] * 6 + [ctypes.POINTER(i)]
    lib.cfc_step_launches.restype = i
    lib.cfc_backward_noalloc.argtypes = [vp] * 7 + [i] * 4 + [vp] * 4 + [i, vp]
    lib.cfc_backward_noalloc.restype = i
    lib.cfc_error_string.argtypes = [i]
    lib.cfc_error_string.restype = ctypes.c_char_p
    lib.cfc_device_status.argtypes = [ctypes.POINTER(i)]
    lib.cfc_device_status.restype = i
    lib.cfc_wait_self_test.argtypes = [vp]
    lib.cfc_wait_self_test.restype = i
    dptr = ctypes.POINTER(ctypes.c_double)
    lib.cfc_probe_fma.argtypes = [vp, i, i, dptr, vp]
    lib.cfc_probe_fma.restype = i
    lib.cfc_probe_l2_read.argtypes = [vp, sz, i, vp, i, dptr, vp]
    lib.cfc_probe_l2_read.restype = i
    lib.cfc_forward_bf16_workspace_bytes.argtypes = [i] * 4 + [ctypes.POINTER(sz)]
    lib.cfc_forward_workspace_bytes.argtypes = [i] * 4 + [ctypes.POINTER(sz)]
    lib.cfc_forward_workspace_bytes.restype = i
    lib.cfc_forward_bf16_workspace_bytes.restype = i
    lib.cfc_forward_bf16.argtypes = [vp] * 5 + [i] * 4 + [vp, vp, vp, sz, vp]
    lib.cfc_forward_bf16.restype = i
    lib.cfc_backward_bf16.argtypes = [vp] * 7 + [i] * 4 + [vp] * 5 + [sz, vp]
    lib.cfc_backward_bf16.restype = i
    lib.cfc_decay_forward.argtypes = [vp] * 6 + [i] * 4 + [vp, vp, vp]
    lib.cfc_decay_forward.restype = i
    lib.cfc_decay_workspace_bytes.argtypes = [i] * 4 + [ctypes.POINTER(sz)]
    lib.cfc_decay_workspace_bytes.restype = i
    lib.cfc_decay_backward.argtypes = [vp] * 8 + [i] * 4 + [vp] * 6 + [sz, vp]
    lib.cfc_decay_backward.restype = i
    lib.cfc_copy.argtypes = [vp, vp, sz, vp]
    lib.cfc_copy.restype = i
    ll, fl, szp = ctypes.c_longlong, ctypes.c_float, ctypes.POINTER(sz)
    conv, scan, grads = (ctypes.POINTER(c) for c in (ConvArgs, ScanArgs, ScanGrads))
    held, rms, gated, kept, ggrads = (ctypes.POINTER(c) for c in (
        Held8Ptrs, RmsnormArgs, GatedArgs, GatedKept, GatedGrads))
    for name, args in {
        "cfc_layernorm_forward": [vp, ll, vp, vp, i, i, fl, i, vp, ll, vp, vp],
        "cfc_layernorm_workspace_bytes": [i, i, szp],
        "cfc_layernorm_backward": [vp, ll, vp, ll, vp, vp, i, i, i, vp, ll, vp, vp, vp, sz, vp],
        "cfc_dropout_forward": [vp, ll, vp, ll, vp, fl, i, i, i, vp, ll, vp],
        "cfc_dropout_backward": [vp, ll, vp, fl, i, i, i, vp, ll, vp],
        "cfc_dropout_layernorm_forward": [vp, ll, vp, ll, vp, fl, vp, vp, i, i, fl, i, vp, ll, vp,
                                          ll, vp, vp],
        "cfc_dropout_layernorm_backward": [vp, ll, vp, ll, vp, ll, vp, fl, vp, vp, i, i, i, vp, ll,
                                           vp, ll, vp, vp, vp, sz, vp],
        "cfc_conv_forward": [conv, vp, ll, ll, vp, vp],
        "cfc_conv_workspace_bytes": [i] * 5 + [szp],
        "cfc_conv_backward": [conv, vp, ll, ll, vp, ll, ll, vp, vp, vp, vp, sz, vp],
        "cfc_conv_step": [vp, ll, vp, vp, vp, i, i, i, i, i, vp, ll, vp, vp],
        "cfc_scan_workspace_bytes": [scan, i, szp],
        "cfc_scan_states_bytes": [scan, szp],
        "cfc_scan_forward": [scan, vp, ll, ll, vp, vp, vp, sz, vp],
        "cfc_scan_backward": [scan, vp, vp, ll, ll, vp, grads, vp, sz, vp],
        "cfc_scan_step": [scan, vp, ll, vp, vp],
        "cfc_pack8": [vp, ll, i, i, i, held, vp],
        "cfc_unpack8": [held, i, i, i, vp, ll, vp],
        "cfc_rmsnorm_forward": [rms, vp, ll, vp, ll, held, held, vp, vp],
        "cfc_rmsnorm_workspace_bytes": [i, i, szp],
        "cfc_rmsnorm_backward": [rms, held, vp, vp, ll, vp, ll, vp, ll, vp, ll, vp, vp, sz, vp],
        "cfc_gated_forward": [gated, vp, ll, ll, vp, vp, kept, vp, sz, vp],
        "cfc_gated_workspace_bytes": [i] * 4 + [szp],
        "cfc_gated_backward": [gated, kept, vp, vp, ll, ll, vp, ggrads, vp, sz, vp],
        "cfc_gated_step": [gated, vp, ll, vp, vp],
        "cfc_weights4_quantize": [vp, ll, i, i, i, i, vp, vp, vp],
        "cfc_weights4_bytes": [i, i, i, szp],
        "cfc_weights4_lay_out": [vp, vp, i, i, i, vp, sz, vp],
        "cfc_matvec4": [vp, ll, vp, i, i, i, i, i, vp, ll, vp],
    }.items():
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = i
    if path is None:
        _lib = lib
    return lib


def error_string(code: int) -> str:
    return load().cfc_error_string(int(code)).decode()


def _check(func: str, rc: int) -> None:
    if rc != CFC_OK:
        raise CfcError(func, rc, error_string(rc))


def _ptr(t, name: str, shape=None):
    import torch

    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 CUDA tensor")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return ctypes.c_void_p(t.data_ptr())


def _ptr16(t, name: str, shape):
    """A contiguous bfloat16 CUDA tensor of the given shape (bf16 H / cache)."""
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous bfloat16 CUDA tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return ctypes.c_void_p(t.data_ptr())


def _ws(ws):
    import torch

    if ws.dtype != torch.uint8 or not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous uint8 CUDA tensor")
    return ctypes.c_void_p(ws.data_ptr()), ws.numel()


def _stream(stream):
    import torch

    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def workspace_bytes(B: int, K: int, C: int, n_x: int, dw_mode: int = CFC_DW_ACCURATE) -> int:
    out = ctypes.c_size_t(0)
    _check("cfc_workspace_bytes",
           load().cfc_workspace_bytes(B, K, C, n_x, dw_mode, ctypes.byref(out)))
    return out.value


def forward_workspace_bytes(B: int, K: int, C: int, n_x: int) -> int:
    out = ctypes.c_size_t(0)
    _check("cfc_forward_workspace_bytes",
           load().cfc_forward_workspace_bytes(B, K, C, n_x, ctypes.byref(out)))
    return out.value


def _fwd_ws(ws, B, K, C, n_x, like):
    """(pointer, bytes) of the forward's workspace: `ws`, or a fresh device buffer when the
    caller gave none and the sizes need one."""
    if ws is None:
        need = forward_workspace_bytes(B, K, C, n_x)
        if need == 0:
            return None, 0, None
        import torch

        ws = torch.empty(need, dtype=torch.uint8, device=like.device)
    p, n = _ws(ws)
    return p, n, ws


def cfc_forward(u, h0, W, b, ts, H, cache, ws=None, stream=None) -> None:
    """H [K,B,C] and cache [K,B,3,C] <- forward recurrence over K steps.  `ws`: a uint8
    device buffer of forward_workspace_bytes() bytes (allocated here when None and needed)."""
    K, B, n_x = u.shape
    C = h0.shape[1]
    n_in = n_x + C
    wp, wn, _keep = _fwd_ws(ws, B, K, C, n_x, H)
    rc = load().cfc_forward(
        _ptr(u, "u", (K, B, n_x)), _ptr(h0, "h0", (B, C)), _ptr(W, "W", (4, C, n_in)),
        _ptr(b, "b", (4, C)), _ptr(ts, "ts", (K, B)), B, K, C, n_x,
        _ptr(H, "H", (K, B, C)), _ptr(cache, "cache", (K, B, 3, C)), wp, wn, _stream(stream))
    _check("cfc_forward", rc)


def cfc_input_projection(u, W, b, H, cache, stream=None) -> None:
    """X = W_u u + b for all steps, written in place into H (ff1) and cache (ff2, ta, tb)."""
    K, B, n_x = u.shape
    C = H.shape[2]
    rc = load().cfc_input_projection(
        _ptr(u, "u", (K, B, n_x)), _ptr(W, "W", (4, C, n_x + C)), _ptr(b, "b", (4, C)),
        B, K, C, n_x, _ptr(H, "H", (K, B, C)), _ptr(cache, "cache", (K, B, 3, C)),
        _stream(stream))
    _check("cfc_input_projection", rc)


def cfc_forward_recurrence(h0, W, ts, H, cache, ws=None, stream=None) -> None:
    """The K-step recurrence on top of the projection left in H / cache (`ws` as for
    cfc_forward)."""
    K, B, C = H.shape
    n_x = W.shape[2] - C
    wp, wn, _keep = _fwd_ws(ws, B, K, C, n_x, H)
    rc = load().cfc_forward_recurrence(
        _ptr(h0, "h0", (B, C)), _ptr(W, "W", (4, C, n_x + C)), _ptr(ts, "ts", (K, B)),
        B, K, C, n_x, _ptr(H, "H", (K, B, C)), _ptr(cache, "cache", (K, B, 3, C)), wp, wn,
        _stream(stream))
    _check("cfc_forward_recurrence", rc)


def step_launches(B: int, K: int, C: int, n_x: int, dw_mode: int = CFC_DW_ACCURATE,
                  with_du: bool = True) -> int:
    """Kernel launches of one cfc_forward + cfc_backward for these sizes."""
    out = ctypes.c_int(0)
    _check("cfc_step_launches",
           load().cfc_step_launches(B, K, C, n_x, dw_mode, int(with_du), ctypes.byref(out)))
    return out.value


def cfc_backward(dH, u, h0, W, ts, H, cache, dW, db, du, dh0, ws,
                 dw_mode: int = CFC_DW_ACCURATE, stream=None) -> None:
    """dW, db, du (optional), dh0 and d_pre (at the head of ws) <- BPTT + contractions."""
    K, B, n_x = u.shape
    C = h0.shape[1]
    n_in = n_x + C
    import torch

    if ws.dtype != torch.uint8 or not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous uint8 CUDA tensor")
    rc = load().cfc_backward(
        _ptr(dH, "dH", (K, B, C)), _ptr(u, "u", (K, B, n_x)), _ptr(h0, "h0", (B, C)),
        _ptr(W, "W", (4, C, n_in)), _ptr(ts, "ts", (K, B)), _ptr(H, "H", (K, B, C)),
        _ptr(cache, "cache", (K, B, 3, C)), B, K, C, n_x, _ptr(dW, "dW", (4, C, n_in)),
        _ptr(db, "db", (4, C)), _ptr(du, "du", (K, B, n_x)), _ptr(dh0, "dh0", (B, C)),
        ctypes.c_void_p(ws.data_ptr()), ws.numel(), dw_mode, _stream(stream))
    _check("cfc_backward", rc)


def cfc_forward_backward(u, h0, W, b, ts, dH, H, cache, dW, db, du, dh0, ws,
                         dw_mode: int = CFC_DW_ACCURATE, stream=None) -> None:
    """One training step: cfc_forward then cfc_backward in one call (the backward recurrence
    launched as a dependent of the forward)."""
    K, B, n_x = u.shape
    C = h0.shape[1]
    n_in = n_x + C
    import torch

    if ws.dtype != torch.uint8 or not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous uint8 CUDA tensor")
    rc = load().cfc_forward_backward(
        _ptr(u, "u", (K, B, n_x)), _ptr(h0, "h0", (B, C)), _ptr(W, "W", (4, C, n_in)),
        _ptr(b, "b", (4, C)), _ptr(ts, "ts", (K, B)), _ptr(dH, "dH", (K, B, C)), B, K, C, n_x,
        _ptr(H, "H", (K, B, C)), _ptr(cache, "cache", (K, B, 3, C)),
        _ptr(dW, "dW", (4, C, n_in)), _ptr(db, "db", (4, C)), _ptr(du, "du", (K, B, n_x)),
        _ptr(dh0, "dh0", (B, C)), ctypes.c_void_p(ws.data_ptr()), ws.numel(), dw_mode,
        _stream(stream))
    _check("cfc_forward_backward", rc)


def cfc_backward_recurrence(dH, W, ts, cache, d_pre, dh0, stream=None) -> None:
    """d_pre [K,B,4,C] and dh0 [B,C] <- reverse-time recurrence only."""
    K, B, C = dH.shape
    n_x = W.shape[2] - C
    rc = load().cfc_backward_recurrence(
        _ptr(dH, "dH", (K, B, C)), _ptr(W, "W", (4, C, n_x + C)), _ptr(ts, "ts", (K, B)),
        _ptr(cache, "cache", (K, B, 3, C)), B, K, C, n_x, _ptr(d_pre, "d_pre", (K, B, 4, C)),
        _ptr(dh0, "dh0", (B, C)), _stream(stream))
    _check("cfc_backward_recurrence", rc)


def bptt_workspace_bytes(B: int, K: int, C: int, n_x: int) -> int:
    """Workspace bytes cfc_backward_recurrence_ws takes (0: the CUDA-core recurrence runs)."""
    out = ctypes.c_size_t(0)
    _check("cfc_bptt_workspace_bytes",
           load().cfc_bptt_workspace_bytes(B, K, C, n_x, ctypes.byref(out)))
    return int(out.value)


def cfc_backward_recurrence_ws(dH, W, ts, cache, d_pre, dh0, ws=None, stream=None) -> None:
    """As cfc_backward_recurrence, with a workspace (a uint8 CUDA tensor of at least
    bptt_workspace_bytes(B, K, C, n_x) bytes, or None when that is 0) so that large batches
    take the tensor-core recurrence."""
    import torch

    K, B, C = dH.shape
    n_x = W.shape[2] - C
    if ws is None:
        wp, wn = None, 0
    else:
        if ws.dtype != torch.uint8 or not ws.is_cuda or not ws.is_contiguous():
            raise ValueError("ws must be a contiguous uint8 CUDA tensor")
        wp, wn = ctypes.c_void_p(ws.data_ptr()), ws.numel()
    rc = load().cfc_backward_recurrence_ws(
        _ptr(dH, "dH", (K, B, C)), _ptr(W, "W", (4, C, n_x + C)), _ptr(ts, "ts", (K, B)),
        _ptr(cache, "cache", (K, B, 3, C)), B, K, C, n_x, _ptr(d_pre, "d_pre", (K, B, 4, C)),
        _ptr(dh0, "dh0", (B, C)), wp, wn, _stream(stream))
    _check("cfc_backward_recurrence_ws", rc)


def cfc_weight_grad(d_pre, u, h0, W, H, dW, db, du, ws, dw_mode: int = CFC_DW_ACCURATE,
                    stream=None) -> None:
    """dW, db, du (optional) <- contractions of d_pre (second stage of cfc_backward)."""
    K, B, n_x = u.shape
    C = h0.shape[1]
    n_in = n_x + C
    rc = load().cfc_weight_grad(
        _ptr(d_pre, "d_pre", (K, B, 4, C)), _ptr(u, "u", (K, B, n_x)), _ptr(h0, "h0", (B, C)),
        _ptr(W, "W", (4, C, n_in)), _ptr(H, "H", (K, B, C)), B, K, C, n_x,
        _ptr(dW, "dW", (4, C, n_in)), _ptr(db, "db", (4, C)), _ptr(du, "du", (K, B, n_x)),
        ctypes.c_void_p(ws.data_ptr()), ws.numel(), dw_mode, _stream(stream))
    _check("cfc_weight_grad", rc)


def reduce_axis0(per_batch, out, stream=None) -> None:
    """out[n] <- sum_r per_batch[r, n] (overwrite, deterministic order)."""
    n_batch, n_tail = per_batch.shape
    rc = load().reduce_axis0(_ptr(per_batch, "per_batch"), n_batch, n_tail,
                             _ptr(out, "out", (n_tail,)), _stream(stream))
    _check("reduce_axis0", rc)


def cfc_wait_self_test(stream=None) -> None:
    """Enqueue the self-test kernel whose bounded wait runs out (read the result with
    device_status(): 1 after about 2 s)."""
    _check("cfc_wait_self_test", load().cfc_wait_self_test(_stream(stream)))


def probe_fma(out, blocks: int, iters: int, stream=None) -> float:
    """Enqueue the fp32 FMA throughput probe; returns the flops it performs."""
    flop = ctypes.c_double(0)
    _check("cfc_probe_fma", load().cfc_probe_fma(_ptr(out, "out"), blocks, iters,
                                                 ctypes.byref(flop), _stream(stream)))
    return flop.value


def probe_l2_read(buf, passes: int, out, blocks: int, stream=None) -> float:
    """Enqueue the L2 read-bandwidth probe over ``buf``; returns the bytes it reads."""
    nbytes = ctypes.c_double(0)
    _check("cfc_probe_l2_read",
           load().cfc_probe_l2_read(_ptr(buf, "buf"), buf.numel(), passes, _ptr(out, "out"), blocks,
                                    ctypes.byref(nbytes), _stream(stream)))
    return nbytes.value


def copy(src, dst, stream=None) -> None:
    """dst <- src by the library's copy kernel.  Both are contiguous tensors of the same size in
    bytes (a multiple of 16, 16-byte aligned); each is on the device or in pinned host memory."""
    import torch

    for t, name in ((src, "src"), (dst, "dst")):
        if not isinstance(t, torch.Tensor) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous torch.Tensor")
        if not t.is_cuda and not t.is_pinned():
            raise ValueError(f"{name} must be a CUDA tensor or in pinned host memory")
    nbytes = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != nbytes:
        raise ValueError("src and dst differ in size")
    _check("cfc_copy", load().cfc_copy(ctypes.c_void_p(src.data_ptr()),
                                       ctypes.c_void_p(dst.data_ptr()), nbytes, _stream(stream)))


def device_status() -> int:
    """Synchronise, then read and clear the device status word (0 = no kernel gave up)."""
    v = ctypes.c_int(0)
    _check("cfc_device_status", load().cfc_device_status(ctypes.byref(v)))
    return v.value


def forward_bf16_workspace_bytes(B: int, K: int, C: int, n_x: int) -> int:
    """Workspace of cfc_forward_bf16 (X = W_u u + b in fp32)."""
    out = ctypes.c_size_t(0)
    _check("cfc_forward_bf16_workspace_bytes",
           load().cfc_forward_bf16_workspace_bytes(B, K, C, n_x, ctypes.byref(out)))
    return out.value


def cfc_forward_bf16(u, h0, W, b, ts, H, cache, ws, stream=None) -> None:
    """bf16 H [K,B,C] and cache [K,B,3,C] <- the forward with fp32 arithmetic."""
    K, B, n_x = u.shape
    C = h0.shape[1]
    n_in = n_x + C
    wp, wn = _ws(ws)
    rc = load().cfc_forward_bf16(
        _ptr(u, "u", (K, B, n_x)), _ptr(h0, "h0", (B, C)), _ptr(W, "W", (4, C, n_in)),
        _ptr(b, "b", (4, C)), _ptr(ts, "ts", (K, B)), B, K, C, n_x,
        _ptr16(H, "H", (K, B, C)), _ptr16(cache, "cache", (K, B, 3, C)), wp, wn,
        _stream(stream))
    _check("cfc_forward_bf16", rc)


def cfc_backward_bf16(dH, u, h0, W, ts, H, cache, dW, db, du, dh0, ws, stream=None) -> None:
    """dW, db, du (optional), dh0 <- the backward of the bf16 H / cache of cfc_forward_bf16."""
    K, B, n_x = u.shape
    C = h0.shape[1]
    n_in = n_x + C
    wp, wn = _ws(ws)
    rc = load().cfc_backward_bf16(
        _ptr(dH, "dH", (K, B, C)), _ptr(u, "u", (K, B, n_x)), _ptr(h0, "h0", (B, C)),
        _ptr(W, "W", (4, C, n_in)), _ptr(ts, "ts", (K, B)), _ptr16(H, "H", (K, B, C)),
        _ptr16(cache, "cache", (K, B, 3, C)), B, K, C, n_x, _ptr(dW, "dW", (4, C, n_in)),
        _ptr(db, "db", (4, C)), _ptr(du, "du", (K, B, n_x)), _ptr(dh0, "dh0", (B, C)),
        wp, wn, _stream(stream))
    _check("cfc_backward_bf16", rc)


# ---- the pages' tau-decay cell ----

def decay_workspace_bytes(B: int, K: int, C: int, n_x: int) -> int:
    out = ctypes.c_size_t(0)
    _check("cfc_decay_workspace_bytes",
           load().cfc_decay_workspace_bytes(B, K, C, n_x, ctypes.byref(out)))
    return out.value


def cfc_decay_forward(x, h0, W, b, tau, ts, H, E, stream=None) -> None:
    """H [K,B,C] and E = tanh(a) [K,B,C] <- the tau-decay cell over K steps."""
    K, B, n_x = x.shape
    C = h0.shape[1]
    rc = load().cfc_decay_forward(
        _ptr(x, "x", (K, B, n_x)), _ptr(h0, "h0", (B, C)), _ptr(W, "W", (C, n_x + C)),
        _ptr(b, "b", (C,)), _ptr(tau, "tau", (C,)), _ptr(ts, "ts", (K, B)), B, K, C, n_x,
        _ptr(H, "H", (K, B, C)), _ptr(E, "E", (K, B, C)), _stream(stream))
    _check("cfc_decay_forward", rc)


def cfc_decay_backward(dH, x, h0, W, tau, ts, H, E, dW, db, dtau, dx, dh0, ws,
                       stream=None) -> None:
    """dW, db, dtau, dx (optional), dh0 <- BPTT of the tau-decay cell."""
    K, B, n_x = x.shape
    C = h0.shape[1]
    wp, wn = _ws(ws)
    rc = load().cfc_decay_backward(
        _ptr(dH, "dH", (K, B, C)), _ptr(x, "x", (K, B, n_x)), _ptr(h0, "h0", (B, C)),
        _ptr(W, "W", (C, n_x + C)), _ptr(tau, "tau", (C,)), _ptr(ts, "ts", (K, B)),
        _ptr(H, "H", (K, B, C)), _ptr(E, "E", (K, B, C)), B, K, C, n_x,
        _ptr(dW, "dW", (C, n_x + C)), _ptr(db, "db", (C,)), _ptr(dtau, "dtau", (C,)),
        _ptr(dx, "dx", (K, B, n_x)), _ptr(dh0, "dh0", (B, C)), wp, wn, _stream(stream))
    _check("cfc_decay_backward", rc)


# ---- trunk operators: layer norm, dropout, causal convolution, selective scan ----

class Prepared:
    """A checked call of an entry point on given tensors (kept by reference): calling it enqueues
    the work on ``stream`` (default: the current stream)."""

    __slots__ = ("name", "fn", "args", "kept", "device")

    def __init__(self, name, fn, args, kept, device):
        self.name, self.fn, self.args, self.kept, self.device = name, fn, args, kept, device

    def __call__(self, stream=None) -> None:
        import torch

        s = (torch._C._cuda_getCurrentRawStream(self.device) if stream is None
             else stream.cuda_stream)
        rc = self.fn(*self.args, s)
        if rc != CFC_OK:
            _check(self.name, rc)


def _entry(f):
    """An entry point from the function that checks its tensors and marshals its arguments:
    f(...) enqueues, f.prepare(...) returns the Prepared call."""
    import functools

    name = f.__name__

    @functools.wraps(f)
    def call(*a, stream=None, **k):
        prepare(*a, **k)(stream)

    def prepare(*a, **k) -> Prepared:
        import torch

        args, kept = f(*a, **k)
        dev = torch.cuda.current_device()
        for t in kept:
            if isinstance(t, torch.Tensor) and t.device.index != dev:
                raise ValueError(f"{name}: a tensor is not on the current device")
        return Prepared(name, getattr(load(), name), args, kept, dev)

    call.prepare = prepare
    return call


def _dims(*sizes):
    """The sizes, which the C entry points take as ints (a conversion would keep the low bits)."""
    if max(sizes) > 0x7FFFFFFF or min(sizes) < -0x80000000:
        raise ValueError(f"sizes {tuple(sizes)} do not fit the entry points' 32-bit integers")
    return sizes


def _act(t, name: str, shape, dtype=None):
    """(pointer, dtype code) of an activation: fp32 or bf16, the last dimension contiguous."""
    import torch

    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in (torch.float32, torch.bfloat16) or not t.is_cuda:
        raise ValueError(f"{name} must be a float32 or bfloat16 CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} has type {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return t.data_ptr()


def _code(t) -> int:
    import torch

    return CFC_BF16 if t.dtype == torch.bfloat16 else CFC_F32


def _par(t, name: str, shape):
    """Address of a contiguous fp32 tensor (None stays None)."""
    p = _ptr(t, name, shape)
    return None if p is None else p.value


def _con(t, name: str, shape, dtype):
    """Address of a contiguous activation-typed tensor (None stays None)."""
    p = _act(t, name, shape, dtype)
    if p is not None and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return p


def _ld(t) -> int:
    """Elements from a row to the next (of a single row, whose stride may be anything, its length)."""
    return 0 if t is None else t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _tb(t) -> tuple[int, int]:
    return (0, 0) if t is None else (t.stride(0), t.stride(1))


def _rng(rng):
    import torch

    if (not isinstance(rng, torch.Tensor) or rng.dtype not in (torch.int64, torch.uint64)
            or not rng.is_cuda or tuple(rng.shape) != (2,) or not rng.is_contiguous()):
        raise ValueError("rng must be a contiguous 64-bit integer CUDA tensor {seed, offset}")
    return rng.data_ptr()


def _lengths(lengths, B):
    import torch

    if lengths is None:
        return None
    if (not isinstance(lengths, torch.Tensor) or lengths.dtype != torch.int32
            or not lengths.is_cuda or tuple(lengths.shape) != (B,) or not lengths.is_contiguous()):
        raise ValueError("lengths must be a contiguous int32 CUDA tensor, one per sequence")
    return lengths.data_ptr()


def _work(ws):
    if ws is None:
        return None, 0
    p, n = _ws(ws)
    return p.value, n


def layernorm_workspace_bytes(rows: int, n: int) -> int:
    out = ctypes.c_size_t(0)
    _check("cfc_layernorm_workspace_bytes",
           load().cfc_layernorm_workspace_bytes(*_dims(rows, n), ctypes.byref(out)))
    return out.value


@_entry
def cfc_layernorm_forward(x, w, b, y, stats, eps: float = 1e-5):
    """y [rows, n] and stats [rows, 2] (mean, rstd) <- layer norm of x's rows."""
    rows, n = _dims(*x.shape)
    return ((_act(x, "x", (rows, n)), _ld(x), _par(w, "w", (n,)), _par(b, "b", (n,)), rows, n, eps,
             _code(x), _act(y, "y", (rows, n), x.dtype), _ld(y), _par(stats, "stats", (rows, 2))),
            (x, w, b, y, stats))


@_entry
def cfc_layernorm_backward(dy, x, w, stats, dx, dw, db, ws=None):
    """dx [rows, n], dw [n], db [n] <- gradient of the layer norm."""
    rows, n = _dims(*x.shape)
    wp, wn = _work(ws)
    return ((_act(dy, "dy", (rows, n), x.dtype), _ld(dy), _act(x, "x", (rows, n)), _ld(x),
             _par(w, "w", (n,)), _par(stats, "stats", (rows, 2)), rows, n, _code(x),
             _act(dx, "dx", (rows, n), x.dtype), _ld(dx), _par(dw, "dw", (n,)),
             _par(db, "db", (n,)), wp, wn), (dy, x, w, stats, dx, dw, db, ws))


@_entry
def cfc_dropout_forward(x, residual, rng, p: float, y):
    """y [rows, n] <- residual (or None) + dropout of x, drawn from rng = {seed, offset}."""
    rows, n = _dims(*x.shape)
    return ((_act(x, "x", (rows, n)), _ld(x), _act(residual, "residual", (rows, n), x.dtype),
             _ld(residual), _rng(rng), p, rows, n, _code(x), _act(y, "y", (rows, n), x.dtype),
             _ld(y)), (x, residual, rng, y))


@_entry
def cfc_dropout_backward(dy, rng, p: float, dx):
    """dx [rows, n] <- dy through the mask of the forward call with the same rng and p."""
    rows, n = _dims(*dy.shape)
    return ((_act(dy, "dy", (rows, n)), _ld(dy), _rng(rng), p, rows, n, _code(dy),
             _act(dx, "dx", (rows, n), dy.dtype), _ld(dx)), (dy, rng, dx))


@_entry
def cfc_dropout_layernorm_forward(x, residual, rng, p: float, w, b, s, y, stats,
                                  eps: float = 1e-5):
    """s <- residual (or None) + dropout of x; y, stats <- layer norm of s."""
    rows, n = _dims(*x.shape)
    return ((_act(x, "x", (rows, n)), _ld(x), _act(residual, "residual", (rows, n), x.dtype),
             _ld(residual), _rng(rng), p, _par(w, "w", (n,)), _par(b, "b", (n,)), rows, n, eps,
             _code(x), _act(s, "s", (rows, n), x.dtype), _ld(s),
             _act(y, "y", (rows, n), x.dtype), _ld(y), _par(stats, "stats", (rows, 2))),
            (x, residual, rng, w, b, s, y, stats))


@_entry
def cfc_dropout_layernorm_backward(dy, ds, s, rng, p: float, w, stats, dx, dres, dw, db, ws=None):
    """dres (or None) <- ds (or None) + the norm's gradient; dx <- dres through the mask; dw, db."""
    rows, n = _dims(*s.shape)
    wp, wn = _work(ws)
    return ((_act(dy, "dy", (rows, n), s.dtype), _ld(dy), _act(ds, "ds", (rows, n), s.dtype),
             _ld(ds), _act(s, "s", (rows, n)), _ld(s), _rng(rng), p, _par(w, "w", (n,)),
             _par(stats, "stats", (rows, 2)), rows, n, _code(s),
             _act(dx, "dx", (rows, n), s.dtype), _ld(dx),
             _act(dres, "dres", (rows, n), s.dtype), _ld(dres), _par(dw, "dw", (n,)),
             _par(db, "db", (n,)), wp, wn), (dy, ds, s, rng, w, stats, dx, dres, dw, db, ws))


def conv_workspace_bytes(B: int, K: int, D: int, W: int, dtype: int) -> int:
    out = ctypes.c_size_t(0)
    _check("cfc_conv_workspace_bytes",
           load().cfc_conv_workspace_bytes(*_dims(B, K, D, W), dtype, ctypes.byref(out)))
    return out.value


def _conv_args(x, w, bias, x0, lengths, silu):
    K, B, D = _dims(*x.shape)
    W = _dims(w.shape[1])[0]
    return ConvArgs(B, K, D, W, _code(x), int(silu), _lengths(lengths, B), _act(x, "x", (K, B, D)),
                    *_tb(x), _par(w, "w", (D, W)), _par(bias, "bias", (D,)),
                    _con(x0, "x0", (B, W - 1, D), x.dtype))


@_entry
def cfc_conv_forward(x, w, u, bias=None, x0=None, lengths=None, last=None, silu: bool = True):
    """u [K, B, D] and last [B, W-1, D] (or None) <- causal convolution of x [K, B, D]."""
    K, B, D = x.shape
    a = _conv_args(x, w, bias, x0, lengths, silu)
    return ((ctypes.byref(a), _act(u, "u", (K, B, D), x.dtype), *_tb(u),
             _con(last, "last", (B, w.shape[1] - 1, D), x.dtype)),
            (x, w, u, bias, x0, lengths, last, a))


@_entry
def cfc_conv_backward(du, x, w, dx, dw, dbias, bias=None, x0=None, lengths=None, dx0=None, ws=None,
                      silu: bool = True):
    """dx, dw [D, W], dbias [D], dx0 (or None) <- gradient of the causal convolution."""
    K, B, D = x.shape
    W = w.shape[1]
    a = _conv_args(x, w, bias, x0, lengths, silu)
    wp, wn = _work(ws)
    return ((ctypes.byref(a), _act(du, "du", (K, B, D), x.dtype), *_tb(du),
             _act(dx, "dx", (K, B, D), x.dtype), *_tb(dx), _par(dw, "dw", (D, W)),
             _par(dbias, "dbias", (D,)), _con(dx0, "dx0", (B, W - 1, D), x.dtype), wp, wn),
            (du, x, w, dx, dw, dbias, bias, x0, lengths, dx0, ws, a))


@_entry
def cfc_conv_step(x, w, state, new_state, u, bias=None, silu: bool = True):
    """u [B, D], new_state [B, W-1, D] (may be state) <- one token of the causal convolution."""
    B, D = _dims(*x.shape)
    W = _dims(w.shape[1])[0]
    return ((_act(x, "x", (B, D)), _ld(x), _par(w, "w", (D, W)), _par(bias, "bias", (D,)),
             _con(state, "state", (B, W - 1, D), x.dtype), B, D, W, _code(x), int(silu),
             _act(u, "u", (B, D), x.dtype), _ld(u),
             _con(new_state, "new_state", (B, W - 1, D), x.dtype)),
            (x, w, bias, state, new_state, u))


def _scan_sizes(K, B, D, N, G, dtype):
    _dims(B, K, D, N, G)
    return ScanArgs(B=B, K=K, D=D, N=N, G=G, dtype=dtype)


def scan_workspace_bytes(K: int, B: int, D: int, N: int, G: int, dtype: int, backward: bool) -> int:
    out, a = ctypes.c_size_t(0), _scan_sizes(K, B, D, N, G, dtype)
    _check("cfc_scan_workspace_bytes",
           load().cfc_scan_workspace_bytes(ctypes.byref(a), int(backward), ctypes.byref(out)))
    return out.value


def scan_states_bytes(K: int, B: int, D: int, N: int, G: int, dtype: int) -> int:
    out, a = ctypes.c_size_t(0), _scan_sizes(K, B, D, N, G, dtype)
    _check("cfc_scan_states_bytes",
           load().cfc_scan_states_bytes(ctypes.byref(a), ctypes.byref(out)))
    return out.value


def _groups(t, name, shape, dtype):
    p = _act(t, name, shape, dtype)
    if t.shape[-2] > 1 and t.stride(-2) != t.shape[-1]:
        raise ValueError(f"{name} must be contiguous in its last two dimensions")
    return p


def _scan_args(x, dt, A, Bm, Cm, D, dt_bias, z, h0, lengths, softplus):
    K, B, Dn = _dims(*x.shape)
    G, N = _dims(*Bm.shape[-2:])
    rows, bc = (K, B, Dn), (K, B, G, N)
    return ScanArgs(B, K, Dn, N, G, _code(x), int(softplus), _lengths(lengths, B),
                    _act(x, "x", rows), _act(dt, "dt", rows, x.dtype), _act(z, "z", rows, x.dtype),
                    *_tb(x), *_tb(dt), *_tb(z), _groups(Bm, "Bm", bc, x.dtype),
                    _groups(Cm, "Cm", bc, x.dtype), *_tb(Bm), *_tb(Cm), _par(A, "A", (Dn, N)),
                    _par(D, "D", (Dn,)), _par(dt_bias, "dt_bias", (Dn,)),
                    _par(h0, "h0", (B, Dn, N)))


@_entry
def cfc_scan_forward(x, dt, A, Bm, Cm, y, D=None, dt_bias=None, z=None, h0=None, lengths=None,
                     h_last=None, states=None, ws=None, softplus: bool = True):
    """y [K, B, D], h_last [B, D, N] (or None) and, for training, states (a float32 tensor of
    scan_states_bytes() bytes, or None) <- selective scan."""
    K, B, Dn = x.shape
    N = A.shape[1]
    a = _scan_args(x, dt, A, Bm, Cm, D, dt_bias, z, h0, lengths, softplus)
    wp, wn = _work(ws)
    kept = (-(-K // SCAN_PERIOD), B, Dn, N)
    return ((ctypes.byref(a), _act(y, "y", (K, B, Dn), x.dtype), *_tb(y),
             _par(h_last, "h_last", (B, Dn, N)), _par(states, "states", kept), wp, wn),
            (x, dt, A, Bm, Cm, y, D, dt_bias, z, h0, lengths, h_last, states, ws, a))


@_entry
def cfc_scan_backward(dy, x, dt, A, Bm, Cm, states, dx, ddt, dA, dB, dC, D=None, dt_bias=None,
                      z=None, h0=None, lengths=None, dh_last=None, dD=None, ddt_bias=None, dz=None,
                      dh0=None, ws=None, softplus: bool = True):
    """The selective scan's gradients from dy and dh_last (or None)."""
    K, B, Dn = x.shape
    G, N = Bm.shape[-2:]
    a = _scan_args(x, dt, A, Bm, Cm, D, dt_bias, z, h0, lengths, softplus)
    rows = (K, B, Dn)
    g = ScanGrads(_act(dx, "dx", rows, x.dtype), _act(ddt, "ddt", rows, x.dtype),
                  _act(dz, "dz", rows, x.dtype), *_tb(dx), *_tb(ddt), *_tb(dz),
                  _con(dB, "dB", (K, B, G, N), x.dtype), _con(dC, "dC", (K, B, G, N), x.dtype),
                  _par(dA, "dA", (Dn, N)), _par(dD, "dD", (Dn,)),
                  _par(ddt_bias, "ddt_bias", (Dn,)), _par(dh0, "dh0", (B, Dn, N)))
    wp, wn = _work(ws)
    return ((ctypes.byref(a), _par(states, "states", (-(-K // SCAN_PERIOD), B, Dn, N)),
             _act(dy, "dy", rows, x.dtype), *_tb(dy), _par(dh_last, "dh_last", (B, Dn, N)),
             ctypes.byref(g), wp, wn),
            (dy, x, dt, A, Bm, Cm, states, dx, ddt, dA, dB, dC, D, dt_bias, z, h0, lengths,
             dh_last, dD, ddt_bias, dz, dh0, ws, a, g))


@_entry
def cfc_scan_step(x, dt, A, Bm, Cm, state, new_state, y, D=None, dt_bias=None, z=None,
                  softplus: bool = True):
    """y [B, D], new_state [B, D, N] (may be state) <- one token of the selective scan; x, dt, z
    [B, D], Bm, Cm [B, G, N]."""
    def steps(t):
        return None if t is None else t[None]

    a = _scan_args(x[None], steps(dt), A, steps(Bm), steps(Cm), D, dt_bias, steps(z), state, None,
                   softplus)
    B, Dn = x.shape
    return ((ctypes.byref(a), _act(y, "y", (B, Dn), x.dtype), _ld(y),
             _par(new_state, "new_state", (B, Dn, A.shape[1]))),
            (x, dt, A, Bm, Cm, state, new_state, y, D, dt_bias, z, a))


# ---- the gated block's operators: values in 8 bits, root-mean-square norm, gated linear
# recurrence, products with 4-bit weights ----

class Held8:
    """Rows held in 8 bits: `codes` [.., n] (e4m3) and `scales` [.., ceil(n / HELD8_BLOCK)] (e8m0),
    contiguous uint8 CUDA tensors of their own unless they are given."""

    __slots__ = ("codes", "scales")

    def __init__(self, shape, device=None, codes=None, scales=None):
        import torch

        blocks = (*shape[:-1], -(-shape[-1] // HELD8_BLOCK))
        new = dict(dtype=torch.uint8, device=device or "cuda")
        self.codes = torch.empty(shape, **new) if codes is None else codes
        self.scales = torch.empty(blocks, **new) if scales is None else scales


def _bytes8(t, name: str, shape):
    """Address of a contiguous uint8 tensor."""
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.uint8 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous uint8 CUDA tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr()


def _held8(h, name: str, shape):
    """The pointers of rows in 8 bits (None stays None)."""
    if h is None:
        return None
    if not isinstance(h, Held8):
        raise TypeError(f"{name} must be a Held8")
    return Held8Ptrs(_bytes8(h.codes, name + ".codes", shape),
                     _bytes8(h.scales, name + ".scales",
                             (*shape[:-1], -(-shape[-1] // HELD8_BLOCK))))


def _by(s):
    return None if s is None else ctypes.byref(s)


def _parts8(*held):
    """The tensors of the rows in 8 bits that there are."""
    return tuple(t for h in held if h is not None for t in (h.codes, h.scales))


@_entry
def cfc_pack8(x, held):
    """held (Held8) <- the rows of x [rows, n] in 8 bits."""
    rows, n = _dims(*x.shape)
    h = _held8(held, "held", (rows, n))
    if h is None:
        raise TypeError("held must be a Held8")
    return ((_act(x, "x", (rows, n)), _ld(x), rows, n, _code(x), ctypes.byref(h)),
            (x, *_parts8(held), h))


@_entry
def cfc_unpack8(held, y):
    """y [rows, n] <- what the rows in 8 bits stand for."""
    rows, n = _dims(*y.shape)
    h = _held8(held, "held", (rows, n))
    if h is None:
        raise TypeError("held must be a Held8")
    return ((ctypes.byref(h), rows, n, _code(y), _act(y, "y", (rows, n)), _ld(y)),
            (y, *_parts8(held), h))


def rmsnorm_workspace_bytes(rows: int, n: int) -> int:
    out = ctypes.c_size_t(0)
    _check("cfc_rmsnorm_workspace_bytes",
           load().cfc_rmsnorm_workspace_bytes(*_dims(rows, n), ctypes.byref(out)))
    return out.value


@_entry
def cfc_rmsnorm_forward(x, w, residual=None, s=None, y=None, s8=None, y8=None, rstd=None,
                        eps: float = 1e-5):
    """s <- x + residual (or None); y <- its root-mean-square norm; s8, y8 <- both in 8 bits; rstd
    [rows].  Each output may be None; s may be x or residual."""
    rows, n = _dims(*x.shape)
    a = RmsnormArgs(rows, n, _code(x), eps, _act(x, "x", (rows, n)),
                    _act(residual, "residual", (rows, n), x.dtype), _ld(x), _ld(residual),
                    _par(w, "w", (n,)))
    h, k = _held8(s8, "s8", (rows, n)), _held8(y8, "y8", (rows, n))
    return ((ctypes.byref(a), _act(s, "s", (rows, n), x.dtype), _ld(s),
             _act(y, "y", (rows, n), x.dtype), _ld(y), _by(h), _by(k),
             _par(rstd, "rstd", (rows,))),
            (x, w, residual, s, y, rstd, *_parts8(s8, y8), a, h, k))


@_entry
def cfc_rmsnorm_backward(dy, s, w, rstd, dx, dw, ds=None, y=None, ws=None):
    """dx [rows, n] (plus ds, or None), dw [n] and y formed again (or None) from the stream s, a
    tensor or a Held8."""
    rows, n = _dims(*dy.shape)
    held = isinstance(s, Held8)
    h = _held8(s, "s", (rows, n)) if held else None
    a = RmsnormArgs(rows, n, _code(dy), 0.0, None if held else _act(s, "s", (rows, n), dy.dtype),
                    None, 0 if held else _ld(s), 0, _par(w, "w", (n,)))
    wp, wn = _work(ws)
    return ((ctypes.byref(a), _by(h), _par(rstd, "rstd", (rows,)), _act(dy, "dy", (rows, n)),
             _ld(dy), _act(ds, "ds", (rows, n), dy.dtype), _ld(ds),
             _act(dx, "dx", (rows, n), dy.dtype), _ld(dx), _act(y, "y", (rows, n), dy.dtype),
             _ld(y), _par(dw, "dw", (n,)), wp, wn),
            (dy, w, rstd, dx, dw, ds, y, ws, *(_parts8(s) if held else (s,)), a, h))


def gated_workspace_bytes(K: int, B: int, D: int, backward: bool) -> int:
    out = ctypes.c_size_t(0)
    _check("cfc_gated_workspace_bytes",
           load().cfc_gated_workspace_bytes(*_dims(B, K, D), int(backward), ctypes.byref(out)))
    return out.value


def _gated_args(shape, dtype, x, f, bias, z, h0, lengths):
    K, B, D = _dims(*shape)
    code = CFC_BF16 if "bfloat16" in str(dtype) else CFC_F32
    return GatedArgs(B, K, D, code, _lengths(lengths, B), _act(x, "x", shape, dtype),
                     _act(f, "f", shape, dtype), _act(z, "z", shape, dtype), *_tb(x), *_tb(f),
                     *_tb(z), _par(bias, "bias", (D,)), _par(h0, "h0", (B, D)))


def _gated_kept(kept, shape):
    """cfc_gated_kept of a tuple (x, f, z) of Held8, z None where there is none; None stays None."""
    if kept is None:
        return None
    if len(kept) != 3 or kept[0] is None or kept[1] is None:
        raise ValueError("kept must be (x, f, z) as Held8, z None where the recurrence has none")
    return GatedKept(*(_held8(h, "kept", shape) or Held8Ptrs() for h in kept))


@_entry
def cfc_gated_forward(x, f, y, bias=None, z=None, h0=None, lengths=None, h_last=None, states=None,
                      kept=None, ws=None):
    """y [K, B, D], h_last [B, D] (or None; may be h0) and, for training, states
    [ceil(K / GATED_PERIOD), B, D] and kept, a tuple (x, f, z) of Held8 (or None) <- gated linear
    recurrence."""
    K, B, D = x.shape
    a = _gated_args((K, B, D), x.dtype, x, f, bias, z, h0, lengths)
    k = _gated_kept(kept, (K, B, D))
    if kept is not None and (kept[2] is None) != (z is None):
        raise ValueError("kept holds a z where the recurrence has one")
    return ((ctypes.byref(a), _act(y, "y", (K, B, D), x.dtype), *_tb(y),
             _par(h_last, "h_last", (B, D)),
             _par(states, "states", (-(-K // GATED_PERIOD), B, D)), _by(k), *_work(ws)),
            (x, f, y, bias, z, h0, lengths, h_last, states, ws, *_parts8(*(kept or ())), a, k))


@_entry
def cfc_gated_backward(dy, x, f, states, dx, df, bias=None, z=None, lengths=None, dh_last=None,
                       dz=None, dbias=None, dh0=None, y=None, kept=None, ws=None):
    """The gated linear recurrence's gradients from dy and dh_last (or None), and y formed again (or
    None).  With kept, what it holds takes the place of x, f and z, which are None then."""
    K, B, D = dy.shape
    rows, act = (K, B, D), dy.dtype
    if (kept is None) == (x is None) or (kept is None) == (f is None):
        raise ValueError("the backward pass reads either x and f or what was kept of them")
    if kept is not None and z is not None:
        raise ValueError("z is read from what was kept")
    a = _gated_args(rows, act, x, f, bias, z, None, lengths)
    k = _gated_kept(kept, rows)
    g = GatedGrads(_act(dx, "dx", rows, act), _act(df, "df", rows, act),
                   _act(dz, "dz", rows, act), _act(y, "y", rows, act), *_tb(dx), *_tb(df),
                   *_tb(dz), *_tb(y), _par(dbias, "dbias", (D,)), _par(dh0, "dh0", (B, D)))
    wp, wn = _work(ws)
    return ((ctypes.byref(a), _by(k), _par(states, "states", (-(-K // GATED_PERIOD), B, D)),
             _act(dy, "dy", rows), *_tb(dy), _par(dh_last, "dh_last", (B, D)),
             ctypes.byref(g), wp, wn),
            (dy, x, f, states, dx, df, bias, z, lengths, dh_last, dz, dbias, dh0, y, ws,
             *_parts8(*(kept or ())), a, k, g))


@_entry
def cfc_gated_step(x, f, state, new_state, y, bias=None, z=None):
    """y [B, D], new_state [B, D] (may be state) <- one token of the gated linear recurrence."""
    def steps(t):
        return None if t is None else t[None]

    B, D = x.shape
    a = _gated_args((1, B, D), x.dtype, x[None], steps(f), bias, steps(z), state, None)
    return ((ctypes.byref(a), _act(y, "y", (B, D), x.dtype), _ld(y),
             _par(new_state, "new_state", (B, D))),
            (x, f, state, new_state, y, bias, z, a))


def _scales4(t, shape):
    """Address of the bf16 scales of 4-bit weights."""
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError("scales must be a torch.Tensor")
    if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
        raise ValueError("scales must be a contiguous bfloat16 CUDA tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"scales has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr()


def weights4_bytes(N: int, K: int, group: int) -> int:
    out = ctypes.c_size_t(0)
    _check("cfc_weights4_bytes",
           load().cfc_weights4_bytes(*_dims(N, K), group, ctypes.byref(out)))
    return out.value


@_entry
def cfc_weights4_quantize(W, codes, scales, group: int):
    """codes [N, ceil(K / 2)], scales [N, ceil(K / group)] (bf16) <- the nearest 4-bit weights."""
    N, K = _dims(*W.shape)
    group = max(int(group), 1)
    return ((_act(W, "W", (N, K)), _ld(W), N, K, group, _code(W),
             _bytes8(codes, "codes", (N, (K + 1) // 2)), _scales4(scales, (N, -(-K // group)))),
            (W, codes, scales))


@_entry
def cfc_weights4_lay_out(codes, scales, K: int, group: int, weights):
    """weights (uint8, weights4_bytes() of them) <- codes and scales in the order of cfc_matvec4."""
    N = _dims(codes.shape[0], K)[0]
    group = max(int(group), 1)
    wp, wn = _work(weights)
    return ((_bytes8(codes, "codes", (N, (K + 1) // 2)), _scales4(scales, (N, -(-K // group))), N,
             K, group, wp, wn), (codes, scales, weights))


@_entry
def cfc_matvec4(x, weights, N: int, group: int, y):
    """y [M, N] <- x [M, K] times the transposed 4-bit weights of cfc_weights4_lay_out."""
    M, K = _dims(*x.shape)
    wp, wn = _work(weights)
    if wn < weights4_bytes(N, K, group):
        raise ValueError("weights are shorter than weights4_bytes() of these sizes")
    return ((_act(x, "x", (M, K)), _ld(x), wp, M, N, K, group, _code(x),
             _act(y, "y", (M, N), x.dtype), _ld(y)), (x, weights, y))
