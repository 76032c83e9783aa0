"""The trunk operators as steps that own their outputs and workspaces, in the manner of
``step.KLoopStep``: bind the inputs once (their types and shapes are checked then; they are kept
by reference), run them any number of times on the current stream, or capture a run into a CUDA
graph.

Sequences are time-major [K, B, D]; views whose last dimension is contiguous are used in place
(a slice of a packed projection, batch-first memory transposed).  Activations are float32 or
bfloat16, parameters and states float32.
"""
from __future__ import annotations

import torch

from . import _lib


def _device(device):
    return (torch.device(device) if device is not None
            else torch.device("cuda", torch.cuda.current_device()))


def _workspace(nbytes: int, device):
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


class _Step:
    """Prepared calls, run in order."""

    def __init__(self, device):
        self.device = _device(device)
        self._unbind()

    def _act(self, *shape):
        return torch.empty(shape, dtype=self.dtype, device=self.device)

    def _f32(self, *shape):
        return torch.empty(shape, dtype=torch.float32, device=self.device)

    def _unbind(self):
        """What every bind begins with, so that one that is refused leaves nothing bound."""
        self.inputs, self.graph = None, None
        self._forward, self._backward = (), ()

    def forward(self, stream=None) -> None:
        if not self._forward:
            raise ValueError("no inputs are bound")
        for call in self._forward:
            call(stream)

    def backward(self, stream=None) -> None:
        if not self._backward:
            raise ValueError("no gradient is bound")
        for call in self._backward:
            call(stream)

    def run(self, stream=None) -> None:
        """The forward pass and, where a gradient is bound, the backward pass, enqueued on
        ``stream`` (default: the current stream)."""
        self.forward(stream)
        for call in self._backward:
            call(stream)

    def capture(self) -> torch.cuda.CUDAGraph:
        """Capture run() into a CUDA graph (after one eager run)."""
        self.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self.run()
        self.graph = g
        return g

    def replay(self) -> None:
        if self.graph is None:
            self.capture()
        self.graph.replay()


class LayerNormStep(_Step):
    """Layer norm over `rows` rows of n columns: y; with dy bound also dx, dw, db."""

    def __init__(self, rows: int, n: int, dtype=torch.float32, eps: float = 1e-5, device=None):
        super().__init__(device)
        self.rows, self.n, self.dtype, self.eps = rows, n, dtype, eps
        self.y, self.stats = self._act(rows, n), self._f32(rows, 2)
        self.dx = self.dw = self.db = self.ws = None

    def _alloc_grads(self):
        if self.dx is None:
            self.dx = self._act(self.rows, self.n)
            self.dw, self.db = self._f32(self.n), self._f32(self.n)
            self.ws = _workspace(_lib.layernorm_workspace_bytes(self.rows, self.n), self.device)

    def bind(self, x, w, b, dy=None) -> "LayerNormStep":
        self._unbind()
        forward = (_lib.cfc_layernorm_forward.prepare(x, w, b, self.y, self.stats, self.eps),)
        backward = ()
        if dy is not None:
            self._alloc_grads()
            backward = (_lib.cfc_layernorm_backward.prepare(
                dy, x, w, self.stats, self.dx, self.dw, self.db, self.ws),)
        self.inputs = dict(x=x, w=w, b=b, dy=dy)
        self._forward, self._backward = forward, backward
        return self

    def outputs(self) -> dict:
        out = {"y": self.y}
        if self._backward:
            out.update(dx=self.dx, dw=self.dw, db=self.db)
        return out


class DropoutNormStep(_Step):
    """s = residual + dropout(x), y = layer norm of s; with dy (and the stream's gradient ds)
    bound also dx, dres, dw, db.  ``rng`` is a device tensor {seed, offset} that the caller
    advances between steps."""

    def __init__(self, rows: int, n: int, p: float, dtype=torch.float32, eps: float = 1e-5,
                 device=None):
        super().__init__(device)
        self.rows, self.n, self.p, self.dtype, self.eps = rows, n, p, dtype, eps
        self.s, self.y, self.stats = self._act(rows, n), self._act(rows, n), self._f32(rows, 2)
        self.dx = self.dres = self.dw = self.db = self.ws = None

    def bind(self, x, residual, rng, w, b, dy=None, ds=None) -> "DropoutNormStep":
        self._unbind()
        forward = (_lib.cfc_dropout_layernorm_forward.prepare(
            x, residual, rng, self.p, w, b, self.s, self.y, self.stats, self.eps),)
        backward = ()
        if dy is not None:
            if self.dx is None:
                self.dx, self.dres = self._act(self.rows, self.n), self._act(self.rows, self.n)
                self.dw, self.db = self._f32(self.n), self._f32(self.n)
                self.ws = _workspace(_lib.layernorm_workspace_bytes(self.rows, self.n),
                                     self.device)
            backward = (_lib.cfc_dropout_layernorm_backward.prepare(
                dy, ds, self.s, rng, self.p, w, self.stats, self.dx, self.dres, self.dw, self.db,
                self.ws),)
        self.inputs = dict(x=x, residual=residual, rng=rng, w=w, b=b, dy=dy, ds=ds)
        self._forward, self._backward = forward, backward
        return self

    def outputs(self) -> dict:
        out = {"s": self.s, "y": self.y}
        if self._backward:
            out.update(dx=self.dx, dres=self.dres, dw=self.dw, db=self.db)
        return out


class ConvStep(_Step):
    """Causal convolution of W taps over [K, B, D]: u and the last W - 1 inputs; with dy bound
    also dx, dx0, dw, dbias."""

    def __init__(self, K: int, B: int, D: int, W: int, dtype=torch.float32, silu: bool = True,
                 device=None):
        super().__init__(device)
        self.K, self.B, self.D, self.W, self.dtype, self.silu = K, B, D, W, dtype, silu
        self.u, self.last = self._act(K, B, D), self._act(B, W - 1, D)
        self.dx = self.dx0 = self.dw = self.dbias = self.ws = None

    def bind(self, x, w, bias=None, x0=None, lengths=None, dy=None) -> "ConvStep":
        self._unbind()
        forward = (_lib.cfc_conv_forward.prepare(x, w, self.u, bias, x0, lengths, self.last,
                                                 self.silu),)
        backward = ()
        if dy is not None:
            if self.dx is None:
                self.dx, self.dx0 = self._act(self.K, self.B, self.D), torch.empty_like(self.last)
                self.dw, self.dbias = self._f32(self.D, self.W), self._f32(self.D)
                code = _lib.CFC_BF16 if self.dtype == torch.bfloat16 else _lib.CFC_F32
                self.ws = _workspace(_lib.conv_workspace_bytes(self.B, self.K, self.D, self.W,
                                                               code), self.device)
            backward = (_lib.cfc_conv_backward.prepare(
                dy, x, w, self.dx, self.dw, self.dbias, bias, x0, lengths, self.dx0, self.ws,
                self.silu),)
        self.inputs = dict(x=x, w=w, bias=bias, x0=x0, lengths=lengths, dy=dy)
        self._forward, self._backward = forward, backward
        return self

    def outputs(self) -> dict:
        out = {"u": self.u, "last": self.last}
        if self._backward:
            out.update(dx=self.dx, dx0=self.dx0, dw=self.dw, dbias=self.dbias)
        return out


class ScanStep(_Step):
    """Selective scan over [K, B, D] with N states per channel and G groups of B / C: y and the
    last state h.  With ``train`` it keeps the states that the backward pass reads, and a bound
    dy (and dh_last) gives every gradient."""

    def __init__(self, K: int, B: int, D: int, N: int, G: int = 1, dtype=torch.float32,
                 train: bool = False, softplus: bool = True, device=None):
        super().__init__(device)
        self.K, self.B, self.D, self.N, self.G = K, B, D, N, G
        self.dtype, self.train, self.softplus = dtype, train, softplus
        code = _lib.CFC_BF16 if dtype == torch.bfloat16 else _lib.CFC_F32
        self.y, self.h = self._act(K, B, D), self._f32(B, D, N)
        self.ws = _workspace(_lib.scan_workspace_bytes(K, B, D, N, G, code, False), self.device)
        self.states = None
        if train:
            self.states = self._f32(-(-K // _lib.SCAN_PERIOD), B, D, N)
            self.bws = _workspace(_lib.scan_workspace_bytes(K, B, D, N, G, code, True), self.device)
            self.dx, self.ddt, self.dz = (self._act(K, B, D) for _ in range(3))
            self.dB, self.dC = self._act(K, B, G, N), self._act(K, B, G, N)
            self.dA, self.dD, self.ddt_bias = self._f32(D, N), self._f32(D), self._f32(D)
            self.dh0 = self._f32(B, D, N)

    def bind(self, x, dt, A, Bm, Cm, D=None, dt_bias=None, z=None, h0=None, lengths=None, dy=None,
             dh_last=None) -> "ScanStep":
        self._unbind()
        opt = dict(D=D, dt_bias=dt_bias, z=z, h0=h0, lengths=lengths, softplus=self.softplus)
        forward = (_lib.cfc_scan_forward.prepare(x, dt, A, Bm, Cm, self.y, h_last=self.h,
                                                 states=self.states, ws=self.ws, **opt),)
        backward = ()
        if dy is not None:
            if not self.train:
                raise ValueError("a ScanStep made without train keeps no states to go back through")
            backward = (_lib.cfc_scan_backward.prepare(
                dy, x, dt, A, Bm, Cm, self.states, self.dx, self.ddt, self.dA, self.dB, self.dC,
                dh_last=dh_last, dD=self.dD if D is not None else None,
                ddt_bias=self.ddt_bias if dt_bias is not None else None,
                dz=self.dz if z is not None else None, dh0=self.dh0, ws=self.bws, **opt),)
        self.inputs = dict(x=x, dt=dt, A=A, Bm=Bm, Cm=Cm, D=D, dt_bias=dt_bias, z=z, h0=h0,
                           lengths=lengths, dy=dy, dh_last=dh_last)
        self._forward, self._backward = forward, backward
        return self

    def outputs(self) -> dict:
        out = {"y": self.y, "h": self.h}
        if self._backward:
            i = self.inputs
            if i["z"] is not None:
                out["dz"] = self.dz
            out.update(dx=self.dx, ddt=self.ddt, dA=self.dA, dB=self.dB, dC=self.dC)
            if i["D"] is not None:
                out["dD"] = self.dD
            if i["dt_bias"] is not None:
                out["ddt_bias"] = self.ddt_bias
            out["dh0"] = self.dh0
        return out


class ConvToken:
    """One token per sequence of the causal convolution: u [B, D] and the moved-on state."""

    def __init__(self, B: int, D: int, W: int, dtype=torch.float32, silu: bool = True, device=None):
        self.silu = silu
        self.u = torch.empty((B, D), dtype=dtype, device=_device(device))

    def bind(self, x, w, state, bias=None, new_state=None) -> "ConvToken":
        """new_state None: the state moves on in place."""
        new_state = state if new_state is None else new_state
        self._call = _lib.cfc_conv_step.prepare(x, w, state, new_state, self.u, bias, self.silu)
        self.state = new_state
        return self

    def run(self, stream=None):
        self._call(stream)
        return self.u, self.state


class ScanToken:
    """One token per sequence of the selective scan: y [B, D] and the new state [B, D, N]."""

    def __init__(self, B: int, D: int, N: int, G: int = 1, dtype=torch.float32,
                 softplus: bool = True, device=None):
        self.softplus = softplus
        self.y = torch.empty((B, D), dtype=dtype, device=_device(device))

    def bind(self, x, dt, A, Bm, Cm, state, D=None, dt_bias=None, z=None,
             new_state=None) -> "ScanToken":
        """new_state None: the state is updated in place."""
        new_state = state if new_state is None else new_state
        self._call = _lib.cfc_scan_step.prepare(x, dt, A, Bm, Cm, state, new_state, self.y, D,
                                                dt_bias, z, self.softplus)
        self.state = new_state
        return self

    def run(self, stream=None):
        self._call(stream)
        return self.y, self.state
