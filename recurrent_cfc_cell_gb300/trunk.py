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


def _expect(t, name: str, shape, dtype):
    """The sizes and the type that a step was made for (the binding checks the rest against them)."""
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype:
        raise ValueError(f"{name} is {tuple(t.shape)} of {t.dtype}, but the step was made for "
                         f"{tuple(shape)} of {dtype}")


class _Step:
    """Prepared calls, run in order."""

    _into = ()  # names of the outputs for which a step takes tensors

    def __init__(self, device, into: dict | None = None):
        self.device, self.into = _device(device), into or {}
        if not set(self.into) <= set(self._into):
            raise ValueError(f"into names {sorted(self.into)}, but the step takes {self._into}")
        self._unbind()

    def _act(self, *shape):
        return torch.empty(shape, dtype=self.dtype, device=self.device)

    def _out(self, name: str, *shape):
        """The output `name`: the tensor that the step was given for it, or one of its own."""
        return self.into[name] if name in self.into else self._act(*shape)

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


class _Call:
    """One prepared call.  A bind that is refused leaves the one before as it was."""

    _call = None

    def _enqueue(self, stream) -> None:
        if self._call is None:
            raise ValueError("no inputs are bound")
        self._call(stream)


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


class ConvToken(_Call):
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
        self._enqueue(stream)
        return self.u, self.state


class ScanToken(_Call):
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
        self._enqueue(stream)
        return self.y, self.state


class Pack8Step(_Call):
    """The rows of x [rows, n] in 8 bits: `held`, a Held8."""

    def __init__(self, rows: int, n: int, dtype=torch.float32, device=None):
        self.rows, self.n, self.dtype = rows, n, dtype
        self.held = _lib.Held8((rows, n), _device(device))

    def bind(self, x) -> "Pack8Step":
        _expect(x, "x", (self.rows, self.n), self.dtype)
        self._call = _lib.cfc_pack8.prepare(x, self.held)
        return self

    def run(self, stream=None):
        self._enqueue(stream)
        return self.held


class Unpack8Step(_Call):
    """What rows in 8 bits stand for: y [rows, n]."""

    def __init__(self, rows: int, n: int, dtype=torch.float32, device=None):
        self.y = torch.empty((rows, n), dtype=dtype, device=_device(device))

    def bind(self, held) -> "Unpack8Step":
        self._call = _lib.cfc_unpack8.prepare(held, self.y)
        return self

    def run(self, stream=None):
        self._enqueue(stream)
        return self.y


class RMSNormStep(_Step):
    """s = x + residual (without one s is x) and its root-mean-square norm y over `rows` rows of n
    columns; with dy (and the stream's gradient ds) bound also dx (of x and of the residual) and dw.
    With ``out8`` y is held in 8 bits (``y8``, a Held8).  With ``keep8`` the stream is kept in 8 bits
    (``s8``) and the backward pass reads that in its place and forms y again (``y_again``).  ``into``
    gives tensors for y, s, dx and y_again, by these names, which steps that take turns may share; dx
    may be ds."""

    _into = ("y", "s", "dx", "y_again")

    def __init__(self, rows: int, n: int, dtype=torch.float32, eps: float = 1e-5,
                 out8: bool = False, keep8: bool = False, device=None, into: dict | None = None):
        super().__init__(device, into)
        self.rows, self.n, self.dtype, self.eps = rows, n, dtype, eps
        self.out8, self.keep8 = out8, keep8
        self.y = None if out8 else self._out("y", rows, n)
        self.y8 = _lib.Held8((rows, n), self.device) if out8 else None
        self.s8 = _lib.Held8((rows, n), self.device) if keep8 else None
        self.rstd = self._f32(rows)
        self.s = self.dx = self.dw = self.y_again = self.ws = None

    def _alloc_grads(self):
        if self.dx is None:
            self.dx, self.dw = self._out("dx", self.rows, self.n), self._f32(self.n)
            self.y_again = self._out("y_again", self.rows, self.n) if self.keep8 else None
            self.ws = _workspace(_lib.rmsnorm_workspace_bytes(self.rows, self.n), self.device)

    def bind(self, x, w, residual=None, dy=None, ds=None) -> "RMSNormStep":
        self._unbind()
        _expect(x, "x", (self.rows, self.n), self.dtype)
        if residual is not None and self.s is None:
            self.s = self._out("s", self.rows, self.n)
        s = None if residual is None else self.s
        forward = (_lib.cfc_rmsnorm_forward.prepare(
            x, w, residual, s, self.y, self.s8, self.y8, self.rstd, self.eps),)
        backward = ()
        if dy is not None:
            self._alloc_grads()
            stream = self.s8 if self.keep8 else x if residual is None else self.s
            backward = (_lib.cfc_rmsnorm_backward.prepare(
                dy, stream, w, self.rstd, self.dx, self.dw, ds, self.y_again, self.ws),)
        self.inputs = dict(x=x, w=w, residual=residual, dy=dy, ds=ds)
        self._forward, self._backward = forward, backward
        return self

    def outputs(self) -> dict:
        out = {"y8": self.y8} if self.out8 else {"y": self.y}
        if self.inputs is not None and self.inputs["residual"] is not None:
            out["s"] = self.s
        if self._backward:
            out.update(dx=self.dx, dw=self.dw)
            if self.keep8:
                out["y_again"] = self.y_again
        return out


class GatedStep(_Step):
    """Gated linear recurrence over [K, B, D]: y and the last state h.  With ``train`` it keeps the
    states that the backward pass starts from, and a bound dy (and dh_last) gives every gradient.
    With ``keep8`` it keeps x, f and z in 8 bits (``kept``), and the backward pass reads those in
    their place, so that the inputs may be gone by then, and forms y again (``y_again``).  ``into``
    gives tensors for y, dx, df, dz and y_again, by these names, which steps that take turns may
    share."""

    _into = ("y", "dx", "df", "dz", "y_again")

    def __init__(self, K: int, B: int, D: int, dtype=torch.float32, train: bool = False,
                 keep8: bool = False, device=None, into: dict | None = None):
        super().__init__(device, into)
        if keep8 and not train:
            raise ValueError("a GatedStep made without train keeps nothing")
        self.K, self.B, self.D, self.dtype = K, B, D, dtype
        self.train, self.keep8 = train, keep8
        self.y, self.h = self._out("y", K, B, D), self._f32(B, D)
        self.states = self.kept = self.y_again = None
        # One workspace for both passes, which follow one another.
        self.ws = _workspace(max(_lib.gated_workspace_bytes(K, B, D, back)
                                for back in (False, train)), self.device)
        if train:
            self.states = self._f32(-(-K // _lib.GATED_PERIOD), B, D)
            self.dx, self.df = self._out("dx", K, B, D), self._out("df", K, B, D)
            self.dz = None
            self.dbias, self.dh0 = self._f32(D), self._f32(B, D)

    def _keep(self, z):
        if not self.keep8:
            return None
        shape = (self.K, self.B, self.D)
        if self.kept is None:
            self.kept = (_lib.Held8(shape, self.device), _lib.Held8(shape, self.device), None)
        if z is not None and self.kept[2] is None:
            self.kept = (*self.kept[:2], _lib.Held8(shape, self.device))
        return self.kept if z is not None else (*self.kept[:2], None)

    def bind(self, x, f, bias=None, z=None, h0=None, lengths=None, dy=None,
             dh_last=None) -> "GatedStep":
        self._unbind()
        _expect(x, "x", (self.K, self.B, self.D), self.dtype)
        kept = self._keep(z)
        forward = (_lib.cfc_gated_forward.prepare(x, f, self.y, bias, z, h0, lengths, self.h,
                                                  self.states, kept, self.ws),)
        backward = ()
        if dy is not None:
            if not self.train:
                raise ValueError("a GatedStep made without train keeps no states to go back from")
            if z is not None and self.dz is None:
                self.dz = self._out("dz", self.K, self.B, self.D)
            if self.keep8 and self.y_again is None:
                self.y_again = self._out("y_again", self.K, self.B, self.D)
            read = (None, None) if kept else (x, f)
            backward = (_lib.cfc_gated_backward.prepare(
                dy, *read, self.states, self.dx, self.df, bias, None if kept else z, lengths, dh_last,
                None if z is None else self.dz, None if bias is None else self.dbias, self.dh0,
                self.y_again, kept, self.ws),)
        self.inputs = dict(x=x, f=f, bias=bias, z=z, h0=h0, lengths=lengths, dy=dy,
                           dh_last=dh_last)
        self._forward, self._backward = forward, backward
        return self

    def outputs(self) -> dict:
        out = {"y": self.y, "h": self.h}
        if self._backward:
            out.update(dx=self.dx, df=self.df)
            if self.inputs["z"] is not None:
                out["dz"] = self.dz
            if self.inputs["bias"] is not None:
                out["dbias"] = self.dbias
            out["dh0"] = self.dh0
            if self.keep8:
                out["y_again"] = self.y_again
        return out


class GatedToken(_Call):
    """One token per sequence of the gated linear recurrence: y [B, D] and the new state [B, D]."""

    def __init__(self, B: int, D: int, dtype=torch.float32, device=None):
        self.y = torch.empty((B, D), dtype=dtype, device=_device(device))

    def bind(self, x, f, state, bias=None, z=None, new_state=None) -> "GatedToken":
        """new_state None: the state is updated in place."""
        new_state = state if new_state is None else new_state
        self._call = _lib.cfc_gated_step.prepare(x, f, state, new_state, self.y, bias, z)
        self.state = new_state
        return self

    def run(self, stream=None):
        self._enqueue(stream)
        return self.y, self.state


class Weights4:
    """A matrix [N, K] of 4-bit weights in the order in which the products read them, laid out once
    (on the current stream) from codes [N, ceil(K / 2)] (uint8, two to a byte, the even column in
    the low half) and scales [N, ceil(K / group)] (bfloat16)."""

    def __init__(self, codes, scales, K: int, group: int):
        self.N, self.K, self.group = codes.shape[0], K, group
        self.data = torch.empty(_lib.weights4_bytes(self.N, K, group), dtype=torch.uint8,
                                device=codes.device)
        _lib.cfc_weights4_lay_out(codes, scales, K, group, self.data)

    @staticmethod
    def quantized(W, group: int):
        """(codes, scales) of the 4-bit weights nearest to W [N, K]."""
        N, K = W.shape
        codes = torch.empty((N, (K + 1) // 2), dtype=torch.uint8, device=W.device)
        scales = torch.empty((N, -(-K // max(group, 1))), dtype=torch.bfloat16, device=W.device)
        _lib.cfc_weights4_quantize(W, codes, scales, group)
        return codes, scales

    @classmethod
    def of(cls, W, group: int = 128) -> "Weights4":
        """The 4-bit weights nearest to W [N, K] (float32 or bfloat16), laid out."""
        return cls(*cls.quantized(W, group), W.shape[1], group)


class MatvecStep(_Step):
    """y [M, N] = x W^T for M rows and a matrix of 4-bit weights; more rows than a call of the product
    takes go in several."""

    def __init__(self, M: int, weights: Weights4, dtype=torch.float32, device=None):
        super().__init__(device)
        self.M, self.weights, self.dtype = M, weights, dtype
        self.y = self._act(M, weights.N)

    def bind(self, x) -> "MatvecStep":
        self._unbind()
        w = self.weights
        _expect(x, "x", (self.M, w.K), self.dtype)
        most = _lib.MATVEC4_ROWS
        self._forward = tuple(_lib.cfc_matvec4.prepare(x[m:m + most], w.data, w.N, w.group,
                                                       self.y[m:m + most])
                              for m in range(0, max(self.M, 1), most))
        self.inputs = dict(x=x)
        return self

    def outputs(self) -> dict:
        return {"y": self.y}
