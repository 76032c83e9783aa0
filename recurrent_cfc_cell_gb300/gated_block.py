"""A trunk of gated blocks in front of the cell, made of the gated block's operators: per layer a
root-mean-square norm with the residual's addition, one product for the mixer's inputs, the gated
linear recurrence, and the product back into the stream; then the last norm and the CfC K-loop.

    s' = s + o;  n = norm(s')                     [K, B, D]   (o: of the layer before; none at first)
    x, f, z = n W_in^T                            [K, B, E] each
    o' = gated(x, f, bias, z) W_out^T             [K, B, D]
    H = cell(norm(s' + o'))                       [K, B, C]   behind the last layer

``GatedTrunk`` trains it.  With ``keep8`` a layer keeps the stream and x, f and z in 8 bits for its
backward pass, 3 E + D bytes a step and sequence (and a scale's byte for every 32) beside the
recurrence's states, and what the products' weight gradients need (n and the recurrence's y) is
formed again by the backward passes, so that those buffers are the same ones for all layers.
``GatedServe`` runs prompts and then single tokens with carried states on 4-bit weights, a token as
one CUDA graph, up to the last norm.  The training products are torch's; everything else is this
library's kernels.  All float32, as the cell.
"""
from __future__ import annotations

import torch

from . import _lib
from .step import KLoopStep
from .trunk import GatedStep, GatedToken, MatvecStep, RMSNormStep, Weights4, _expect


def make_gated_params(layers: int, D: int, E: int, C: int, seed: int = 0, device=None) -> dict:
    """Random parameters: `layers` dicts of w, W_in [3 E, D], bias, W_out [D, E] under "layers", the
    last norm's w and the cell's cell_W [4, C, D + C] and cell_b [4, C]."""
    g = torch.Generator().manual_seed(seed)
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(*shape, generator=g) * std + mean).to(dev).contiguous()

    return dict(
        layers=[dict(w=normal(D, std=0.1, mean=1.0), W_in=normal(3 * E, D, std=D ** -0.5),
                     bias=normal(E, std=1.0, mean=2.0), W_out=normal(D, E, std=E ** -0.5))
                for _ in range(layers)],
        w=normal(D, std=0.1, mean=1.0), cell_W=normal(4, C, D + C, std=(D + C) ** -0.5),
        cell_b=normal(4, C, std=0.1))


class GatedTrunk:
    """One training step of the trunk for K steps of B sequences.  Like the steps it is made of, it
    owns its results: what forward and backward return is valid until they are called again."""

    def __init__(self, K: int, B: int, params: dict, keep8: bool = False):
        self.K, self.B, self.params, self.keep8 = K, B, params, keep8
        self.D, self.E = params["layers"][0]["W_out"].shape
        rows, D, E = K * B, self.D, self.E
        layers = len(params["layers"])
        self.last = RMSNormStep(rows, D)
        self.cell = KLoopStep(B, K, params["cell_b"].shape[1], D)

        def new(*shape):
            return torch.empty(*shape, device=self.last.device)

        self.xfz = [new(K, B, 3 * E) for _ in range(1 if keep8 else layers)]
        self.o = new(rows, D)
        # Gradients on their way back, the same buffers for all layers; a norm's dx takes the place of
        # the stream's gradient that it is added to.
        self.dy, self.dn, self.dxfz = new(K, B, E), new(rows, D), new(K, B, 3 * E)
        norm, mix = dict(dx=new(rows, D)), {
            k: self.dxfz[..., n * E:(n + 1) * E] for n, k in enumerate(("dx", "df", "dz"))}
        if keep8:  # y is formed again, and wanted no longer than its product; the sum is in place
            self.stream = new(rows, D)
            norm.update(y=new(rows, D), y_again=new(rows, D), s=self.stream)
            mix.update(y=new(K, B, E), y_again=new(K, B, E))
        self.norms = [RMSNormStep(rows, D, keep8=keep8, into=norm) for _ in range(layers)]
        self.mixers = [GatedStep(K, B, E, train=True, keep8=keep8, into=mix) for _ in range(layers)]

    def forward(self, s, h0, ts, lengths=None) -> torch.Tensor:
        """H [K, B, C] from the stream s [K, B, D], the cell's h0 [B, C] and time scales ts [K, B].  With
        lengths the recurrences end at them; norms, products and the cell have none, so that s is finite
        behind a length too, and dH is 0 there where H is not wanted."""
        P, K, B, E, rows = self.params, self.K, self.B, self.E, self.K * self.B
        _expect(s, "s", (K, B, self.D), torch.float32)  # as many elements in another order would do
        stream, o = s.reshape(rows, self.D), None
        for i, (p, norm, mix) in enumerate(zip(P["layers"], self.norms, self.mixers)):
            norm.bind(stream, p["w"], o).forward()
            stream = stream if o is None else norm.s
            xfz = self.xfz[0 if self.keep8 else i]
            torch.mm(norm.y, p["W_in"].T, out=xfz.view(rows, 3 * E))
            mix.bind(xfz[..., :E], xfz[..., E:2 * E], p["bias"], xfz[..., 2 * E:], None, lengths,
                     self.dy).forward()
            o = torch.mm(mix.y.view(rows, E), p["W_out"].T, out=self.o) if self.keep8 else (
                mix.y.view(rows, E) @ p["W_out"].T)
        self.last.bind(stream, P["w"], o).forward()
        self.h0, self.ts, self.lengths = h0, ts, lengths
        self.u_cell = self.last.y.view(K, B, self.D)
        _lib.cfc_forward(self.u_cell, h0, P["cell_W"], P["cell_b"], ts, self.cell.H,
                         self.cell.cache, ws=self.cell.fws)
        return self.cell.H

    def backward(self, dH) -> dict:
        """Gradients of sum dH . H: of every parameter (by its name), of the stream (ds) and of the
        cell's initial state (dh0)."""
        P, K, B, E, rows = self.params, self.K, self.B, self.E, self.K * self.B
        c = self.cell
        c.bind(self.u_cell, self.h0, P["cell_W"], P["cell_b"], self.ts, dH).backward()
        g, w = self._norm_back(self.last, P["w"], c.du.view(rows, self.D), None)
        layers = []
        for p, norm, mix in zip(reversed(P["layers"]), reversed(self.norms), reversed(self.mixers)):
            # g: of the layer's output and of the stream beside it.
            torch.mm(g, p["W_out"], out=self.dy.view(rows, E))
            mix.backward()
            y = mix.y_again if self.keep8 else mix.y
            dxfz = self.dxfz.view(rows, 3 * E)
            grads = dict(W_out=g.T @ y.view(rows, E), bias=mix.dbias)
            torch.mm(dxfz, p["W_in"], out=self.dn)
            g, grads["w"] = self._norm_back(norm, p["w"], self.dn, g)
            grads["W_in"] = dxfz.T @ (norm.y_again if self.keep8 else norm.y)
            layers.append(grads)
        return dict(layers=layers[::-1], w=w, cell_W=c.dW, cell_b=c.db, dh0=c.dh0,
                    ds=g.view(K, B, self.D))

    def _norm_back(self, norm, w, dy, ds):
        i = norm.inputs
        stream = norm.s8 if norm.keep8 else i["x"] if i["residual"] is None else norm.s
        if norm.dx is None:
            norm._alloc_grads()
        _lib.cfc_rmsnorm_backward(dy, stream, w, norm.rstd, norm.dx, norm.dw, ds, norm.y_again,
                                  norm.ws)
        return norm.dx, norm.dw


class GatedServe:
    """The trunk up to the last norm for serving, its products on 4-bit weights: a prompt (of at most
    2^24 steps, the recurrence's limit, and 2^31 - 1 rows), then single tokens, with the recurrences'
    states carried in place.  A prompt's products are the tokens' kernels, ten rows at a time."""

    def __init__(self, B: int, params: dict, group: int = 128):
        self.B, self.params = B, params
        self.D, self.E = params["layers"][0]["W_out"].shape
        self.W_in = [Weights4.of(p["W_in"], group) for p in params["layers"]]
        self.W_out = [Weights4.of(p["W_out"], group) for p in params["layers"]]
        dev = params["w"].device
        self.states = [torch.zeros(B, self.E, device=dev) for _ in params["layers"]]
        self._token = None

    def _calls(self, s, mixers, rows):
        """The steps of one pass over `rows` rows s, and its result."""
        E, calls, stream, o = self.E, [], s, None
        for p, w_in, w_out, mix in zip(self.params["layers"], self.W_in, self.W_out, mixers):
            norm = RMSNormStep(rows, self.D).bind(stream, p["w"], o)
            stream = stream if o is None else norm.s
            inner = MatvecStep(rows, w_in).bind(norm.y)
            step = mix(inner.y, p["bias"])
            outer = MatvecStep(rows, w_out).bind(step.y.view(rows, E))
            o = outer.y
            calls += [norm, inner, step, outer]
        last = RMSNormStep(rows, self.D).bind(stream, self.params["w"], o)
        return calls + [last], last.y

    def prompt(self, s, lengths=None) -> torch.Tensor:
        """The last norm's output [K, B, D] of a prompt s [K, B, D], continuing from the carried
        states."""
        _expect(s, "s", (*s.shape[:1], self.B, self.D), torch.float32)
        K, B, E = s.shape[0], self.B, self.E

        def mixer(state):
            def make(xfz, bias):
                v = xfz.view(K, B, 3 * E)
                step = GatedStep(K, B, E)
                step.h = state  # moves on in place
                return step.bind(v[..., :E], v[..., E:2 * E], bias, v[..., 2 * E:], state, lengths)
            return make

        calls, y = self._calls(s.reshape(K * B, self.D), [mixer(t) for t in self.states], K * B)
        for c in calls:
            c.run()
        return y.view(K, B, self.D)

    def token(self, s) -> torch.Tensor:
        """The last norm's output [B, D] of one token s [B, D] per sequence, a tensor of its own."""
        _expect(s, "s", (self.B, self.D), torch.float32)  # a copy would repeat one row for all
        if self._token is None:
            B, E = self.B, self.E
            self.s = torch.empty(B, self.D, device=s.device)

            def mixer(state):
                def make(xfz, bias):
                    return GatedToken(B, E).bind(xfz[:, :E], xfz[:, E:2 * E], state, bias,
                                                 xfz[:, 2 * E:])
                return make

            calls, self.y = self._calls(self.s, [mixer(t) for t in self.states], B)
            before = [t.clone() for t in self.states]
            self.s.copy_(s)
            try:
                for c in calls:  # eagerly once, before the capture
                    c.run()
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    for c in calls:
                        c.run()
            finally:  # the states move on with the replay, and not where the capture fails
                for t, b in zip(self.states, before):
                    t.copy_(b)
            self._token = (graph, calls)
        self.s.copy_(s)
        self._token[0].replay()
        return self.y.clone()
